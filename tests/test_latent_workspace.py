"""The workspace of absorbed latent attention (no kernel is launched): what the query answers is enough
for the call with the same bounds, and for every call with smaller ones."""
import ctypes
import itertools

import pytest
import torch

import causal_gqa_attention_rope_gb300 as na
from causal_gqa_attention_rope_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return na.load_library()


def answer(lib, conf, batch, T, most, top, ws_bytes):
    """What the call says to a workspace of that size.  Only without a GPU: enough of it would be launched
    over these addresses."""
    c = conf.c()
    pages = na.na_paged_latent_cache(kv=16, page_table=16, num_pages=16, page_size=64, batch=batch,
                                     pages_per_seq=1 << 20)
    return lib.na_attn_latent_paged(ctypes.byref(c), batch, 16, 16, T, most, top, 16, ctypes.byref(pages), 16, 16,
                                    ws_bytes, None, None)


RANKS = [(512, 64), (256, 64), (128, 32)]


@pytest.mark.parametrize("R,rd", RANKS)
@pytest.mark.parametrize("H", [16, 32, 33, 64, 128])
def test_a_call_needs_what_the_query_says(lib, H, R, rd):
    """Exactly: with one byte less the call is refused, with that it comes as far as the missing GPU,
    whatever the bounds, new lengths above the call's tokens among them."""
    if torch.cuda.is_available():
        pytest.skip("calls with addresses of nothing")
    conf = na.LatentConfig(H, R, rd)
    for batch, T, most, top in itertools.product((1, 4, 64), (1, 4, 300), (1, 2, 8, 100), (63, 8192)):
        need = na.na_latent_paged_workspace_size(conf, batch, T, most, top)
        assert need == na.na_latent_paged_workspace_size(conf, batch, T, min(most, T), top)
        assert answer(lib, conf, batch, T, most, top, need - 1) == na.NA_ERR_WORKSPACE
        assert answer(lib, conf, batch, T, most, top, need) == na.NA_ERR_CUDA


@pytest.mark.parametrize("R,rd", RANKS)
@pytest.mark.parametrize("H", [5, 16, 32, 40, 128])
def test_more_of_anything_never_needs_less(lib, H, R, rd):
    conf = na.LatentConfig(H, R, rd)
    bounds = [(1, 2, 3, 4, 64, 500), (1, 2, 3, 5, 64, 5000), (0, 1, 2, 3, 4, 5, 8, 13, 64, 500), (1, 64, 65, 640, 8192, 131072)]
    size = {at: na.na_latent_paged_workspace_size(conf, *(b[i] for b, i in zip(bounds, at)))
            for at in itertools.product(*(range(len(b)) for b in bounds))}
    for at, n in size.items():
        for i in range(4):
            if at[i]:
                less = at[:i] + (at[i] - 1,) + at[i + 1:]
                assert size[less] <= n, [b[i] for b, i in zip(bounds, at)]
