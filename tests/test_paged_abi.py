"""Host-side validation of the paged entry points (no kernel is launched)."""
import ctypes

import pytest
import torch

import causal_gqa_attention_rope_gb300 as na
from causal_gqa_attention_rope_gb300 import _build
from paged_ref import make_paged


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return na.load_library()


def cfg(**kw):
    base = dict(num_heads=32, num_kv_heads=8, head_dim=128)
    base.update(kw)
    return na.AttnConfig(**base).c()


def paged(**kw):
    """A struct of fake non-null, aligned addresses: 16 pages of 64, 4 sequences of 8 pages."""
    base = dict(k=16, v=16, k_scale=16, v_scale=16, page_table=16, num_pages=16, page_size=64,
                batch=4, pages_per_seq=8, dtype=na.NA_KV_E4M3)
    base.update(kw)
    return na.na_paged_kv_cache(**base)


def append(lib, c, kv, rope=None, batch=4, T=4, q=16, q_out=16):
    r = (rope or na.RopeConfig()).c()
    return lib.na_rope_append_kv_paged(ctypes.byref(c), ctypes.byref(r), batch, 16, 16, T, q, 16, 16,
                                       None, None, q_out, ctypes.byref(kv), None, None)


def prefill(lib, c, kv, batch=4, T=8, most=2, top=512, q=16, gate=None, ws=None, ws_bytes=0):
    return lib.na_attn_prefill_chunk_paged(ctypes.byref(c), batch, 16, 16, T, most, top, q,
                                           ctypes.byref(kv), gate, 16, ws, ws_bytes, None, None)


def decode(lib, c, kv, batch=4, q=16, top=512, gate=None, probs=None, stride=0, splits=0, ws=16,
           ws_bytes=1 << 30):
    return lib.na_attn_decode_paged(ctypes.byref(c), batch, q, ctypes.byref(kv), 16, top, gate, 16,
                                    probs, stride, splits, ws, ws_bytes, None, None)


BAD_CACHES = [
    (dict(k=None), na.NA_ERR_INVALID_ARG),
    (dict(v=None), na.NA_ERR_INVALID_ARG),
    (dict(page_table=None), na.NA_ERR_INVALID_ARG),
    (dict(k=24), na.NA_ERR_INVALID_ARG),  # not 16-byte aligned
    (dict(k_scale=None), na.NA_ERR_INVALID_ARG),
    (dict(v_scale=None), na.NA_ERR_INVALID_ARG),
    (dict(dtype=2), na.NA_ERR_INVALID_ARG),
    (dict(num_pages=0), na.NA_ERR_INVALID_ARG),
    (dict(pages_per_seq=0), na.NA_ERR_INVALID_ARG),
    (dict(batch=3), na.NA_ERR_INVALID_ARG),  # fewer table rows than sequences
    (dict(page_size=0), na.NA_ERR_UNSUPPORTED),
    (dict(page_size=8), na.NA_ERR_UNSUPPORTED),
    (dict(page_size=48), na.NA_ERR_UNSUPPORTED),
    (dict(page_size=256), na.NA_ERR_UNSUPPORTED),
    (dict(num_pages=1 << 22), na.NA_ERR_UNSUPPORTED),       # 2^31 rows
    (dict(pages_per_seq=1 << 25), na.NA_ERR_UNSUPPORTED),   # 2^31 positions
]


@pytest.mark.parametrize("kw,code", BAD_CACHES, ids=lambda x: str(x))
def test_bad_caches(lib, kw, code):
    for call in (append, prefill, decode):
        assert call(lib, cfg(), paged(**kw)) == code


def test_a_ring_is_refused(lib):
    c = cfg(window=64, ring_cache=True)
    for call in (append, prefill, decode):
        assert call(lib, c, paged()) == na.NA_ERR_UNSUPPORTED


def test_bad_arguments(lib):
    c = cfg()
    for call in (append, prefill, decode):
        assert call(lib, cfg(head_dim=96), paged()) == na.NA_ERR_UNSUPPORTED
        assert call(lib, cfg(num_heads=30), paged()) == na.NA_ERR_INVALID_ARG
        assert call(lib, c, paged(), batch=0) == na.NA_ERR_INVALID_ARG
        assert call(lib, c, paged(), q=None) == na.NA_ERR_INVALID_ARG
        assert call(lib, c, paged(), q=18) == na.NA_ERR_INVALID_ARG
    for call in (append, prefill):
        assert call(lib, c, paged(), T=-1) == na.NA_ERR_INVALID_ARG
        assert call(lib, c, paged(), T=0) == na.NA_OK
    assert append(lib, c, paged(), rope=na.RopeConfig(base=1.0)) == na.NA_ERR_INVALID_ARG
    assert append(lib, cfg(qk_norm=True), paged()) == na.NA_ERR_INVALID_ARG  # no weights
    assert prefill(lib, c, paged(), most=0) == na.NA_ERR_INVALID_ARG
    for call in (prefill, decode):
        assert call(lib, c, paged(), top=513) == na.NA_ERR_CAPACITY
        assert call(lib, cfg(out_gate=True), paged()) == na.NA_ERR_INVALID_ARG
    assert decode(lib, c, paged(), probs=16, stride=511) == na.NA_ERR_CAPACITY
    assert decode(lib, c, paged(), splits=-1) == na.NA_ERR_INVALID_ARG


def test_workspaces(lib):
    c, out = cfg(), ctypes.c_size_t(0)
    size = lambda *a: lib.na_decode_paged_workspace_size(ctypes.byref(c), *a, ctypes.byref(out))  # noqa: E731
    assert size(4, 512, 0) == na.NA_OK
    need = out.value
    assert need > 0
    assert decode(lib, c, paged(), ws=None) == na.NA_ERR_WORKSPACE
    assert decode(lib, c, paged(), ws=24) == na.NA_ERR_WORKSPACE
    assert decode(lib, c, paged(), ws_bytes=need - 1) == na.NA_ERR_WORKSPACE
    assert size(0, 512, 0) == na.NA_ERR_INVALID_ARG
    assert size(4, -1, 0) == na.NA_ERR_INVALID_ARG
    assert lib.na_prefill_paged_workspace_size(ctypes.byref(c), 4, 8, 2, 512 * 8, ctypes.byref(out)) == 0
    assert out.value > 0
    big = paged(pages_per_seq=64)
    assert prefill(lib, c, big, top=4096) == na.NA_ERR_WORKSPACE


def test_binding_checks_shapes_and_types(lib):
    """The binding refuses tensors before their pointers cross the C ABI."""
    conf = na.AttnConfig(4, 2, 64)
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)  # noqa: E731
    i32 = lambda *s: z(*s, t=torch.int32)  # noqa: E731
    host = make_paged([5, 9], 2, 64, 16, "e4m3", 1)
    good = na.PagedKVCache(host.k, host.v, host.table, host.k_scale, host.v_scale)

    def decode_with(cache):
        na.na_attn_decode_paged(conf, z(2, 4, 64), cache, i32(2), 9, z(2, 4, 64))

    def replaced(**kw):
        d = dict(k=good.k, v=good.v, page_table=good.page_table, k_scale=good.k_scale,
                 v_scale=good.v_scale)
        d.update(kw)
        return na.PagedKVCache(**d)

    for kw, word in ((dict(k_scale=None), "k_scale"), (dict(v_scale=None), "v_scale"),
                     (dict(k=good.k.view(torch.uint8)), "cache.k"),
                     (dict(k=z(4, 3, 16, 64, t=torch.float8_e4m3fn)), "cache.k"),
                     (dict(v=good.v[1:]), "cache.v"),
                     (dict(page_table=good.page_table[:1]), "page_table"),
                     (dict(page_table=good.page_table.long()), "page_table"),
                     (dict(k_scale=good.k_scale[1:]), "k_scale"),
                     (dict(v_scale=good.v_scale.int()), "v_scale"),
                     (dict(k_scale=None, v_scale=None), "cache.k")):
        with pytest.raises(ValueError, match=word):
            decode_with(replaced(**kw))
    with pytest.raises(ValueError, match="CUDA"):  # right shapes, but on the host
        decode_with(good)


def test_compiled_calls_answer_none_for_what_is_not_plain(lib):
    """Nothing but the plain call is made: no tensors, host tensors, another number of arguments."""
    calls = na._calls()
    host = make_paged([5, 9], 2, 64, 16, "e4m3", 1)
    cache = na.PagedKVCache(host.k, host.v, host.table, host.k_scale, host.v_scale)
    conf, t = na.AttnConfig(4, 2, 64), torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    for f, n, at, plain in ((calls.append, 14, 4, (conf, na.RopeConfig())), (calls.prefill, 13, 5, (conf,)),
                            (calls.decode, 12, 1, (conf,))):
        for filler in (None, 0, "x", t, cache, object()):
            args = list(plain) + [filler] * (n - len(plain))
            assert f(*args) is None
            args[at] = t
            assert f(*args) is None
            assert f(*args[:-1]) is None


@pytest.mark.parametrize("batch", [1, 2])
@pytest.mark.parametrize("group", [1, 32, 33, 40, 128, 130])
def test_prefill_workspace_of_a_step_without_new_tokens(lib, group, batch):
    """max_new_len 0, whatever the group: nothing is needed, as in the contiguous query."""
    c = na.AttnConfig(group, 1, 64)
    for total in (0, 1, 5):
        for top in (0, 100, 100000):
            assert na.na_prefill_paged_workspace_size(c, batch, total, 0, top) == 0
            assert na.na_prefill_workspace_size(c, batch, total, 0, top) == 0


@pytest.mark.parametrize("batch,most", [(1 << 16, 1 << 20), (64, 2 ** 31 - 1), (2 ** 31 - 1, 4)])
def test_prefill_bounds_with_too_many_units(lib, batch, most):
    """Bounds so loose that the units (query tile, kv head, sequence) exceed a grid are refused by
    the queries and the calls, over pages and not."""
    c, out = cfg(), ctypes.c_size_t(0)
    for query in (lib.na_prefill_paged_workspace_size, lib.na_prefill_workspace_size):
        assert query(ctypes.byref(c), batch, 8, most, 512, ctypes.byref(out)) == na.NA_ERR_UNSUPPORTED
    assert prefill(lib, c, paged(batch=batch), batch=batch, most=most) == na.NA_ERR_UNSUPPORTED
    flat = na.na_kv_cache(16, 16, 64, 512)
    if batch <= 64:  # (a contiguous cache has the rows of its batch)
        assert lib.na_attn_prefill_chunk(ctypes.byref(c), batch, 16, 16, 8, most, 512, 16,
                                         ctypes.byref(flat), None, 16, 16, 1 << 30, None,
                                         None) == na.NA_ERR_UNSUPPORTED
    # loose, but countable
    for query in (lib.na_prefill_paged_workspace_size, lib.na_prefill_workspace_size):
        assert query(ctypes.byref(c), 1, 8, 2 ** 31 - 1, 512, ctypes.byref(out)) == na.NA_OK


@pytest.mark.parametrize("batch", [1 << 28, 1 << 29, 2 ** 31 - 1])
def test_decode_batches_with_too_many_streams(lib, batch):
    """The workspace holds partial results of every stream (sequence, kv head): a batch whose streams
    pass 32 bits is refused, not sized by what is left of their number."""
    c, out = cfg(), ctypes.c_size_t(0)
    for query in (lib.na_decode_paged_workspace_size, lib.na_decode_workspace_size):
        assert query(ctypes.byref(c), batch, 512, 0, ctypes.byref(out)) == na.NA_ERR_UNSUPPORTED
        assert query(ctypes.byref(c), 1 << 27, 512, 0, ctypes.byref(out)) == na.NA_OK
        assert out.value > (1 << 27) * 32 * 128 * 4
        small = out.value
        assert query(ctypes.byref(c), 1 << 27, 512, 2 ** 31 - 1, ctypes.byref(out)) == na.NA_OK
        assert out.value == small
    assert decode(lib, c, paged(batch=batch), batch=batch) == na.NA_ERR_UNSUPPORTED
