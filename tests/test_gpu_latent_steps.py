"""Absorbed latent attention as a server's steps meet it: loose bounds, one workspace for steps of many
sizes, many rows, the same step again."""
import os
import subprocess
import sys

import pytest
import torch

from latent_ref import make_latent
from paged_ref import bits
from test_gpu_latent import absorbed, check_absorbed, ints, packed, randn

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("H,R,rd,most", [(32, 512, 64, 4), (16, 256, 64, 8), (40, 128, 32, 100)])
def test_a_bound_above_the_call_s_tokens(H, R, rd, most):
    """The workspace that the query names for the same arguments is enough."""
    check_absorbed(H, R, rd, 64, [8000, 10], [1, 1], bounds=(most, 8064))


@pytest.mark.parametrize("R,rd", [(512, 64), (128, 32)])
def test_one_workspace_for_steps_of_many_sizes(R, rd):
    """Sized for the largest step, dirty with what the step before left in it."""
    import causal_gqa_attention_rope_gb300 as na
    H, prior = 32, [4000, 70, 900]
    cfg = na.LatentConfig(H, R, rd)
    pool, table = make_latent([n + 8 for n in prior], R + rd, 32, 21)
    need = na.na_latent_paged_workspace_size(cfg, 3, 24, 8, 4008)
    shared = na.workspace(need, DEV)
    for step, new in enumerate(([8, 8, 8], [1, 1, 1], [2, 0, 3], [0, 1, 0])):
        q = randn(22 + step, sum(new), H, R + rd)
        alone, status = absorbed(cfg, pool, table, prior, new, q)
        assert status == 0
        got, status = absorbed(cfg, pool, table, prior, new, q, workspace=shared)
        assert status == 0 and torch.equal(bits(got), bits(alone))


@pytest.mark.parametrize("R,H,new", [(512, 32, 8), (512, 128, 1), (256, 40, 5), (128, 32, 8)])
def test_many_rows_again_and_again(R, H, new):
    """Units of two CTAs: the same bits from every call, next to the 64-bit statement once."""
    import causal_gqa_attention_rope_gb300 as na
    prior = [3000, 129, 1, 6000, 64, 777]
    check_absorbed(H, R, 64, 64, prior, [new] * 6, seed=31)
    cfg = na.LatentConfig(H, R, 64)
    pool, table = make_latent([n + new for n in prior], R + 64, 64, 32)
    q = randn(33, 6 * new, H, R + 64)
    first, status = absorbed(cfg, pool, table, prior, [new] * 6, q)
    assert status == 0
    for _ in range(20):
        got, status = absorbed(cfg, pool, table, prior, [new] * 6, q)
        assert status == 0 and torch.equal(bits(got), bits(first))


@pytest.mark.parametrize("H,R", [(5, 128), (16, 512), (40, 256)])
def test_many_small_pages_in_one_cluster(H, R):
    """Contexts of more than 32 pages that are still joined in a cluster, and of more that are not."""
    check_absorbed(H, R, 32, 16, [900, 513, 511, 40], [1, 1, 1, 1], seed=41)
    check_absorbed(H, R, 32, 16, [2999], [1], seed=42)


def far(pool, table, pages):
    """The same sequences in the last pages of a pool of `pages`, on the GPU."""
    big = torch.empty(pages, *pool.shape[1:], dtype=pool.dtype, device=DEV)
    big[pages - len(pool):] = pool.to(DEV)
    return big, torch.where(table >= 0, table + (pages - len(pool)), table)


@pytest.mark.parametrize("H,new", [(16, [1, 1, 1]), (64, [3, 1, 2])])
def test_pages_beyond_32_bits(H, new):
    """Rows whose elements are past 2^32: appended and read as those of a small pool, and moved from there."""
    import causal_gqa_attention_rope_gb300 as na
    R, rd, page, prior = 512, 64, 128, [300, 4000, 1]
    pool, table = make_latent(prior, R + rd, page, 51, room=3)
    cfg, T, cu = na.LatentConfig(H, R, rd), sum(new), packed(new)
    kv, q, w = randn(52, T, R + rd).to(DEV), randn(53, T, H, R + rd).to(DEV), randn(54, R).to(DEV)
    results = []
    for p, t in ((pool.to(DEV), table), far(pool, table, 60000)):
        cache, status, x = na.PagedLatentCache(p, t.to(DEV)), ints([0]), q.clone()
        na.na_latent_append_paged(cfg, na.RopeConfig(), ints(cu), ints(prior), kv, x[..., R:], x[..., R:], cache,
                                  kv_norm_w=w, status=status)
        out = torch.empty(T, H, R, dtype=torch.bfloat16, device=DEV)
        ws = na.workspace(na.na_latent_paged_workspace_size(cfg, 3, T, 3, 4003), DEV)
        na.na_attn_latent_paged(cfg, ints(cu), ints(prior), 3, 4003, x, cache, out, workspace=ws, status=status)
        near = na.PagedLatentCache(torch.zeros(99, page, R + rd, dtype=torch.bfloat16, device=DEV),
                                   torch.arange(99, dtype=torch.int32, device=DEV).view(3, 33))
        na.na_pages_compact(cache, near, ints([p + n for p, n in zip(prior, new)]), 4003, rope=na.RopeConfig(),
                            rotary_start=R, status=status)
        src, dst = int(t[1, 0]), len(p) - 1 - next(i for i in range(len(pool)) if len(pool) - 1 - i not in table)
        na.na_pages_copy(cache, ints([src]), ints([dst]), status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        assert torch.equal(bits(p[src]), bits(p[dst]))
        results.append((bits(out.cpu()), bits(x.cpu()), bits(near.kv.cpu())))
    for small, big in zip(*results):
        assert torch.equal(small, big)


def test_expanded_keys_beyond_32_bits():
    """Keys and values whose elements are past 2^32, read as those at the beginning."""
    import causal_gqa_attention_rope_gb300 as na
    H, keys, new = 128, 1500, [130, 1]
    cfg = na.LatentConfig(H)
    few, pe = randn(61, keys, H, 256).to(DEV), randn(62, keys, 64).to(DEV)
    q, starts, lens = randn(63, 131, H, 192).to(DEV), [0, 700], [700, 800]
    results = []
    for total in (keys, 135000):
        kv = torch.empty(total, H, 256, dtype=torch.bfloat16, device=DEV)
        rows = torch.empty(total, 64, dtype=torch.bfloat16, device=DEV)
        kv[total - keys:], rows[total - keys:] = few, pe
        out, status = torch.empty(131, H, 128, dtype=torch.bfloat16, device=DEV), ints([0])
        na.na_attn_latent_expanded(cfg, ints([0, 130, 131]), ints([s + total - keys for s in starts]), ints(lens), 130,
                                   800, q, kv, rows, out, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        results.append(bits(out.cpu()))
    assert torch.equal(*results)


def test_captured_without_a_call_before(tmp_path):
    """A process whose first calls are captured: nothing is set up on the side that a capture forbids."""
    code = """
import sys
sys.path[:0] = sys.argv[1:]
import torch
import causal_gqa_attention_rope_gb300 as na
from latent_ref import make_latent
from test_gpu_latent import ints, randn
R, rd, H, prior = 512, 64, 40, [900, 30]
cfg = na.LatentConfig(H, R, rd)
pool, table = make_latent([901, 31], R + rd, 64, 1)
cache, status = na.PagedLatentCache(pool.cuda(), table.cuda()), ints([0])
kv, q = randn(2, 2, R + rd).cuda(), randn(3, 2, H, R + rd).cuda()
out, ws = torch.zeros(2, H, R, dtype=torch.bfloat16, device="cuda"), torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
big_q, big_kv, wide = randn(4, 300, H, 192).cuda(), randn(5, 4096, H, 256).cuda(), torch.zeros(300, H, 128, dtype=torch.bfloat16, device="cuda")
pe = randn(6, 4096, 64).cuda()
w, cu, lens = torch.ones(R, dtype=torch.bfloat16, device="cuda"), ints([0, 1, 2]), ints(prior)
a = [ints(x) for x in ([0, 300], [0], [4096])]
def step():
    na.na_latent_append_paged(cfg, na.RopeConfig(), cu, lens, kv, None, None, cache, kv_norm_w=w, status=status)
    na.na_attn_latent_paged(cfg, cu, lens, 1, 901, q, cache, out, workspace=ws, status=status)
    na.na_attn_latent_expanded(cfg, *a, 300, 4096, big_q, big_kv, pe, wide, status=status)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step()
assert not out.any() and not wide.any()
g.replay()
torch.cuda.synchronize()
got = out.clone(), wide.clone()
assert int(status.item()) == 0 and out.any() and wide.any()
step()
torch.cuda.synchronize()
assert int(status.item()) == 0 and torch.equal(out, got[0]) and torch.equal(wide, got[1])
print("same")
"""
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", code, here, os.path.dirname(here)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
