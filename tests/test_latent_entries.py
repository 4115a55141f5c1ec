"""Entries of the second pass of absorbed attention: the host side of the check that the kernel makes, since
no kernel is made to give a wait up."""
import os
import subprocess

from causal_gqa_attention_rope_gb300 import _build

PROGRAM = r"""
#include <climits>
#include <cstdio>
#include "latent.cuh"

int main()
{
    // what a workspace may hold where no entry was written, and entries of runs that there are
    const int odd[] = {INT_MIN, -1, 0, 1, 5, 75, 76, 151, 152, INT_MAX, (int)0xffffffff, 0x7fc00000, 0x3f800000};
    const int grid = 152;
    int named = 0;
    for (int z : odd)
        for (int w : odd) {
            const bool there = z >= 0 && z < grid && w >= z && w < grid;
            if (names_runs(make_int4(INT_MAX, INT_MIN, z, w), grid) != there)
                return 1;
            named += there;
        }
    printf("%d\n", named);
    return 0;
}
"""


def test_only_runs_of_the_call_are_joined(tmp_path):
    src = tmp_path / "entries.cu"
    src.write_text(PROGRAM)
    exe = str(tmp_path / "entries")
    subprocess.run([_build.nvcc(), *_build.ARCH, *_build.NVCC_FLAGS, str(src), "-o", exe], check=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True).stdout
    assert int(out) == 21  # z <= w of {0, 1, 5, 75, 76, 151}


def test_the_second_pass_looks_before_it_addresses():
    """Between reading an entry and the first address that depends on it stands the check."""
    with open(os.path.join(_build.CSRC, "latent_attn.cu")) as f:
        kernel = f.read().split("latent_merge_kernel(const", 1)[1]
    read, check, use = (kernel.index(x) for x in ("p.cut[blockIdx.x]", "names_runs(cut, p.grid)", "cut.z + i"))
    assert read < check < use
    assert kernel.index("cut.x = s.tok0") < check
