"""Host-side validation of the page operations (no kernel is launched)."""
import ctypes

import pytest
import torch

import causal_gqa_attention_rope_gb300 as na
from causal_gqa_attention_rope_gb300 import _build
from paged_ref import make_paged
from pages_ref import fork


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return na.load_library()


def pool(**kw):
    base = dict(k=16, v=16, k_scale=16, v_scale=16, page_table=16, num_pages=16, page_size=64,
                batch=4, pages_per_seq=8, dtype=na.NA_KV_E4M3)
    base.update(kw)
    return na.na_paged_kv_cache(**base)


def copy(lib, c, KV=8, d=128, n=4, src=16, dst=16):
    return lib.na_pages_copy(KV, d, None if c is None else ctypes.byref(c), n, src, dst, None, None)


def compact(lib, a, z=None, KV=8, d=128, batch=4, top=0, rope=None, start=0, rd=0, flags=0, lens=16):
    r = None if rope is None else ctypes.byref(rope.c())
    return lib.na_pages_compact(KV, d, batch, ctypes.byref(a), ctypes.byref(z or pool()), None, lens,
                                top, r, start, rd, flags, None, None)


BAD = [
    (dict(k=None), na.NA_ERR_INVALID_ARG), (dict(k=24), na.NA_ERR_INVALID_ARG),
    (dict(v=24), na.NA_ERR_INVALID_ARG), (dict(v=None), na.NA_ERR_INVALID_ARG),
    (dict(k_scale=None), na.NA_ERR_INVALID_ARG), (dict(v_scale=None), na.NA_ERR_INVALID_ARG),
    (dict(dtype=3), na.NA_ERR_INVALID_ARG), (dict(num_pages=0), na.NA_ERR_INVALID_ARG),
    (dict(page_size=48), na.NA_ERR_UNSUPPORTED), (dict(page_size=256), na.NA_ERR_UNSUPPORTED),
    (dict(num_pages=1 << 22), na.NA_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", BAD, ids=lambda x: str(x))
def test_bad_pools(lib, kw, code):
    assert copy(lib, pool(**kw)) == code
    assert compact(lib, pool(**kw)) == code
    assert compact(lib, pool(), pool(**kw)) == code


def test_bad_arguments(lib):
    assert copy(lib, None) == na.NA_ERR_INVALID_ARG
    assert copy(lib, pool(), n=-1) == na.NA_ERR_INVALID_ARG
    assert copy(lib, pool(), src=None) == na.NA_ERR_INVALID_ARG
    assert copy(lib, pool(), dst=None) == na.NA_ERR_INVALID_ARG
    assert copy(lib, pool(), KV=0) == na.NA_ERR_INVALID_ARG
    assert copy(lib, pool(), d=0) == na.NA_ERR_INVALID_ARG
    assert copy(lib, pool(), d=72) == na.NA_ERR_UNSUPPORTED   # E4M3: multiples of 16
    assert copy(lib, pool(dtype=na.NA_KV_BF16), d=1032) == na.NA_ERR_UNSUPPORTED
    # a copy looks at no table, a latent cache has no v; nothing to do is fine
    assert copy(lib, pool(page_table=None, batch=0, pages_per_seq=0), n=0) == na.NA_OK
    assert copy(lib, pool(v=None, dtype=na.NA_KV_BF16), d=576, KV=1, n=0, src=None) == na.NA_OK
    assert compact(lib, pool()) == na.NA_OK
    assert compact(lib, pool(), batch=0) == na.NA_ERR_INVALID_ARG
    assert compact(lib, pool(), batch=5) == na.NA_ERR_INVALID_ARG
    assert compact(lib, pool(), top=-1) == na.NA_ERR_INVALID_ARG
    assert compact(lib, pool(), top=4, lens=None) == na.NA_ERR_INVALID_ARG
    assert compact(lib, pool(page_table=None)) == na.NA_ERR_INVALID_ARG
    assert compact(lib, pool(pages_per_seq=1 << 25)) == na.NA_ERR_UNSUPPORTED
    assert compact(lib, pool(), pool(dtype=na.NA_KV_BF16)) == na.NA_ERR_INVALID_ARG
    both = dict(dtype=na.NA_KV_BF16)
    assert compact(lib, pool(**both), pool(v=None, **both)) == na.NA_ERR_INVALID_ARG
    assert compact(lib, pool(), d=256) == na.NA_ERR_UNSUPPORTED
    assert compact(lib, pool(), flags=1) == na.NA_ERR_INVALID_ARG
    rope = na.RopeConfig()
    for start, rd, code in ((0, 63, na.NA_ERR_INVALID_ARG), (-2, 64, na.NA_ERR_INVALID_ARG),
                            (66, 64, na.NA_ERR_INVALID_ARG), (0, -2, na.NA_ERR_INVALID_ARG),
                            (64, 64, na.NA_OK), (0, 0, na.NA_OK)):
        assert compact(lib, pool(), rope=rope, start=start, rd=rd) == code
    assert compact(lib, pool(**both), pool(**both), d=576, rope=rope, rd=256) == na.NA_ERR_UNSUPPORTED
    assert compact(lib, pool(), rope=na.RopeConfig(base=1.0), rd=64) == na.NA_ERR_INVALID_ARG


def test_fork_arguments(lib):
    good = [4, 4, 16, None, 16, 16, 8, 64, 16, 100, 16, 16, 16, 16, 16, None, None]

    def call(**at):
        args = list(good)
        for i, v in at.items():
            args[int(i[1:])] = v
        return lib.na_pages_fork(*args)

    for i in (2, 4, 5, 8, 10, 11, 12, 13, 14):
        assert call(**{f"a{i}": None}) == na.NA_ERR_INVALID_ARG
    for i in (0, 1, 6, 9):
        assert call(**{f"a{i}": 0}) == na.NA_ERR_INVALID_ARG
    for kw in (dict(a0=4097), dict(a1=4097), dict(a7=48), dict(a7=8), dict(a6=1 << 25), dict(a9=1 << 25)):
        assert call(**kw) == na.NA_ERR_UNSUPPORTED


def test_binding_checks_shapes_and_types(lib):
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    names = ("parents", "lens", "table", "ref", "new_table", "new_ref", "new_lens", "copy_src", "copy_dst")
    shapes = ((4,), (5,), (5, 8), (30,), (4, 8), (30,), (4,), (4,), (4,))
    for i, name in enumerate(names):
        for bad in (i32(*shapes[i]).long(), i32(*shapes[i], 2)):
            args = [i32(*s) for s in shapes]
            args[i] = bad
            with pytest.raises(ValueError, match=name):
                na.na_pages_fork(*args[:4], 64, *args[4:])
    args = [i32(*s) for s in shapes]
    with pytest.raises(ValueError, match="grow"):
        na.na_pages_fork(*args[:4], 64, *args[4:], grow=i32(5))
    with pytest.raises(ValueError, match="CUDA"):
        na.na_pages_fork(*args[:4], 64, *args[4:])
    host = make_paged([5, 9], 2, 64, 16, "e4m3", 1)
    good = na.PagedKVCache(host.k, host.v, host.table, host.k_scale, host.v_scale)
    for kw, word in ((dict(k_scale=None), "k_scale"), (dict(v=good.v[1:]), "v"),
                     (dict(k=good.k.view(torch.uint8)), "k"), (dict(v_scale=good.v_scale[1:]), "v_scale"),
                     (dict(page_table=good.page_table.long()), "page_table")):
        d = dict(k=good.k, v=good.v, page_table=good.page_table, k_scale=good.k_scale, v_scale=good.v_scale)
        d.update(kw)
        with pytest.raises(ValueError, match=word):
            na.na_pages_copy(na.PagedKVCache(**d), i32(2), i32(2))
        with pytest.raises(ValueError, match=word):
            na.na_pages_compact(na.PagedKVCache(**d), good, i32(2), 4)
    with pytest.raises(ValueError, match="CUDA"):
        na.na_pages_copy(good, i32(2), i32(2))


def test_the_host_statement_of_a_fork():
    """Two children of one sequence, one of another, one that ends, one that begins."""
    table = [[4, 1, -1], [0, 6, -1], [5, -1, -1]]
    ref = [1, 1, 0, 0, 1, 1, 1, 0]
    new, refs, lens, src, dst, wrong = fork([1, 1, -1, 2], [0, 1, 17, 16], [20, 20, 16], table, 16, ref)
    assert not wrong
    # page 0 is shared, 6 stays with the first child, 1 and 4 (ended) are free again
    assert new == [[0, 6, -1], [0, 1, -1], [2, 3, -1], [5, 4, -1]]
    assert refs == [2, 1, 1, 1, 1, 1, 1, 0]
    assert (lens, src, dst) == ([20, 20, 0, 16], [-1, 6, -1, -1], [-1, 1, -1, -1])
