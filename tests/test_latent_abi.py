"""Host-side validation of the latent entry points (no kernel is launched)."""
import ctypes

import pytest
import torch

import causal_gqa_attention_rope_gb300 as na
from causal_gqa_attention_rope_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return na.load_library()


def cfg(**kw):
    return na.LatentConfig(**{**dict(num_heads=16, kv_norm=False), **kw}).c()


def pool(**kw):
    base = dict(kv=16, page_table=16, num_pages=16, page_size=64, batch=4, pages_per_seq=8)
    base.update(kw)
    return na.na_paged_latent_cache(**base)


def append(lib, c, kv, rope=None, batch=4, T=4, x=16, xs=576, q=16, qs=64, o=32, os=64, w=None):
    r = (rope or na.RopeConfig()).c()
    return lib.na_latent_append_paged(ctypes.byref(c), ctypes.byref(r), batch, 16, 16, T, x, xs, q, qs, o, os,
                                      w, ctypes.byref(kv), None, None)


def absorbed(lib, c, kv, batch=4, T=8, most=2, top=512, q=16, out=16, ws=16, ws_bytes=1 << 40):
    return lib.na_attn_latent_paged(ctypes.byref(c), batch, 16, 16, T, most, top, q, ctypes.byref(kv), out, ws,
                                    ws_bytes, None, None)


def expanded(lib, c, batch=4, T=8, keys=100, most=2, top=50, q=16, kv=16, pe=16, stride=64, out=16, starts=16):
    return lib.na_attn_latent_expanded(ctypes.byref(c), batch, 16, starts, 16, T, keys, most, top, q, kv, pe,
                                       stride, out, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(num_heads=0), na.NA_ERR_INVALID_ARG), (dict(rms_eps=-1.0), na.NA_ERR_INVALID_ARG),
    (dict(rms_eps=float("nan")), na.NA_ERR_INVALID_ARG), (dict(sm_scale=float("inf")), na.NA_ERR_INVALID_ARG),
    (dict(kv_rank=384), na.NA_ERR_UNSUPPORTED), (dict(kv_rank=0), na.NA_ERR_UNSUPPORTED),
    (dict(rope_dim=0), na.NA_ERR_UNSUPPORTED), (dict(rope_dim=24), na.NA_ERR_UNSUPPORTED),
    (dict(rope_dim=80), na.NA_ERR_UNSUPPORTED), (dict(nope_dim=96), na.NA_ERR_UNSUPPORTED),
    (dict(v_dim=192), na.NA_ERR_UNSUPPORTED),
], ids=str)
def test_bad_configurations(lib, kw, code):
    c, out = cfg(**kw), ctypes.c_size_t(0)
    assert append(lib, c, pool()) == code
    assert absorbed(lib, c, pool()) == code
    assert expanded(lib, c) == code
    assert lib.na_latent_paged_workspace_size(ctypes.byref(c), 1, 1, 1, 1, ctypes.byref(out)) == code


def test_unknown_flags(lib):
    c = cfg()
    c.flags = 4
    assert absorbed(lib, c, pool()) == na.NA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,code", [
    (dict(kv=None), na.NA_ERR_INVALID_ARG), (dict(kv=24), na.NA_ERR_INVALID_ARG),
    (dict(page_table=None), na.NA_ERR_INVALID_ARG), (dict(num_pages=0), na.NA_ERR_INVALID_ARG),
    (dict(pages_per_seq=0), na.NA_ERR_INVALID_ARG), (dict(batch=3), na.NA_ERR_INVALID_ARG),
    (dict(page_size=8), na.NA_ERR_UNSUPPORTED), (dict(page_size=48), na.NA_ERR_UNSUPPORTED),
    (dict(num_pages=1 << 25), na.NA_ERR_UNSUPPORTED), (dict(pages_per_seq=1 << 25), na.NA_ERR_UNSUPPORTED),
], ids=str)
def test_bad_caches(lib, kw, code):
    assert append(lib, cfg(), pool(**kw)) == code
    assert absorbed(lib, cfg(), pool(**kw)) == code


def test_bad_arguments(lib):
    c, bad = cfg(), na.NA_ERR_INVALID_ARG
    for kw in (dict(x=None), dict(x=24), dict(q=None), dict(o=None), dict(q=24), dict(o=24), dict(xs=570),
               dict(xs=560), dict(qs=60), dict(qs=56), dict(os=60), dict(o=16, os=72), dict(batch=0), dict(T=-1),
               dict(rope=na.RopeConfig(base=0.5))):
        assert append(lib, c, pool(), **kw) == bad, kw
    assert append(lib, cfg(kv_norm=True), pool()) == bad          # no weights
    assert append(lib, c, pool(), T=0, x=None, q=None) == na.NA_OK
    for kw in (dict(q=None), dict(q=24), dict(out=None), dict(out=24), dict(most=0), dict(batch=0), dict(T=-1),
               dict(top=-1)):
        assert absorbed(lib, c, pool(), **kw) == bad, kw
    assert absorbed(lib, c, pool(), top=513) == na.NA_ERR_CAPACITY
    assert absorbed(lib, c, pool(), T=1 << 28) == na.NA_ERR_UNSUPPORTED  # 2^32 query rows
    assert absorbed(lib, c, pool(), T=0, q=None) == na.NA_OK
    for kw in (dict(q=None), dict(q=24), dict(kv=None), dict(kv=24), dict(pe=None), dict(pe=24), dict(out=None),
               dict(out=24), dict(starts=None), dict(stride=60), dict(stride=56), dict(keys=0), dict(keys=-1),
               dict(most=0), dict(batch=0), dict(T=-1)):
        assert expanded(lib, c, **kw) == bad, kw
    assert expanded(lib, c, batch=1 << 28, T=1 << 20, most=1 << 20) == na.NA_ERR_UNSUPPORTED
    assert expanded(lib, c, T=0, q=None) == na.NA_OK


def test_workspaces(lib):
    conf = na.LatentConfig(16, kv_norm=False)
    need = na.na_latent_paged_workspace_size(conf, 4, 8, 2, 512)
    c = conf.c()
    assert absorbed(lib, c, pool(), ws=None) == na.NA_ERR_WORKSPACE
    assert absorbed(lib, c, pool(), ws=24) == na.NA_ERR_WORKSPACE
    assert absorbed(lib, c, pool(), ws_bytes=need - 1) == na.NA_ERR_WORKSPACE
    # more of anything never needs less, up to one piece per SM
    sizes = [na.na_latent_paged_workspace_size(conf, b, b * n, n, k)
             for b, n, k in ((1, 1, 1), (1, 1, 64), (1, 1, 65), (2, 1, 65), (2, 5, 65), (64, 5, 8192))]
    assert sizes == sorted(sizes)
    assert na.na_latent_paged_workspace_size(conf, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1) > 0
    with pytest.raises(na.NAError):
        na.na_latent_paged_workspace_size(conf, 0, 1, 1, 1)


def test_binding_checks_shapes_and_types(lib):
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)  # noqa: E731
    i32 = lambda *s: z(*s, t=torch.int32)  # noqa: E731
    conf = na.LatentConfig(4, 128, 32, 64, 64)
    good = dict(cache=na.PagedLatentCache(z(5, 16, 160), i32(2, 2)), kv=z(3, 160), q=z(3, 4, 32), o=z(3, 4, 32),
                w=z(128), lat=z(3, 4, 160), out=z(3, 4, 128), wide=z(3, 4, 96), keys=z(9, 4, 128), pe=z(9, 32),
                dst=z(3, 4, 64), cu=i32(3), lens=i32(2))

    def calls(**kw):
        a = {**good, **kw}
        yield lambda: na.na_latent_append_paged(conf, na.RopeConfig(), a["cu"], a["lens"], a["kv"], a["q"], a["o"],
                                                a["cache"], kv_norm_w=a["w"])
        yield lambda: na.na_attn_latent_paged(conf, a["cu"], a["lens"], 2, 9, a["lat"], a["cache"], a["out"])
        yield lambda: na.na_attn_latent_expanded(conf, a["cu"], a["lens"], a["lens"], 2, 9, a["wide"], a["keys"],
                                                 a["pe"], a["dst"])

    def refuses(which, word, **kw):
        with pytest.raises(ValueError, match=word):
            list(calls(**kw))[which]()

    for which in range(3):
        refuses(which, "CUDA")  # right shapes, but on the host
        refuses(which, "cu_seqlens", cu=i32(3).long())
    for which in range(2):
        refuses(which, "cache.kv", cache=na.PagedLatentCache(z(5, 16, 161), i32(2, 2)))
        refuses(which, "cache.kv", cache=na.PagedLatentCache(z(5, 16, 160).half(), i32(2, 2)))
        refuses(which, "page_table", cache=na.PagedLatentCache(z(5, 16, 160), i32(1, 2)))
        refuses(which, "cache_lens", lens=i32(1))
    refuses(0, "q_out", o=z(3, 4, 33))
    refuses(0, "go together", o=None)
    refuses(0, "kv_norm_w", w=z(127))
    refuses(1, "q_lat", lat=z(3, 4, 128))
    refuses(1, "out", out=z(2, 4, 128))
    refuses(2, "key_", lens=i32(1))
    refuses(2, "kv", keys=z(9, 4, 129))
    refuses(2, "k_pe", pe=z(8, 32))
    refuses(2, "out", dst=z(3, 4, 64).float())
