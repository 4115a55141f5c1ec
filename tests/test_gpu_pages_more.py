"""Compaction at the ends of its ranges: bounds, skipped rows, the largest scales."""
import pytest
import torch

from paged_ref import bits, make_paged
from pages_ref import turned

pytestmark = pytest.mark.gpu
DEV = "cuda"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def compact(a, z, lens, top, **kw):
    """Status of a call."""
    import causal_gqa_attention_rope_gb300 as na
    status = ints([0])
    na.na_pages_compact(a, z, ints(lens), top, status=status, **kw)
    torch.cuda.synchronize()
    return int(status.item())


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("top", [41, 100000, 2 ** 31 - 1])
def test_a_loose_bound(fmt, top):
    """No more is enqueued than the new pages have room for, and lengths that have none are reported."""
    import causal_gqa_attention_rope_gb300 as na
    old, new = make_paged([40, 41], 2, 64, 16, fmt, 1), make_paged([0, 0], 2, 64, 32, fmt, 2, room=41)
    z = new.to(DEV)
    assert compact(old.to(DEV), z, [40, 41], top) == 0
    for b, n in enumerate((40, 41)):
        for was, scale, got, got_scale in ((old.k, old.k_scale, z.k, z.k_scale), (old.v, old.v_scale, z.v, z.v_scale)):
            for j in range(n):
                x, y = was[old.table[b, j // 16], :, j % 16], got[new.table[b, j // 32], :, j % 32].cpu()
                if fmt == "bf16":
                    assert torch.equal(bits(x), bits(y))
                else:  # within the rounding to the new page's scale, at most half its smallest step or 2^-4
                    s, t = (v[i].double().cpu() - 127 for v, i in ((scale, old.table[b, j // 16]),
                                                                   (got_scale, new.table[b, j // 32])))
                    x, y = x.double() * torch.exp2(s)[:, None], y.double() * torch.exp2(t)[:, None]
                    assert ((x - y).abs() <= 2.0 ** -4 * x.abs() + torch.exp2(t - 10)[:, None]).all()
    if top > 64:
        assert compact(old.to(DEV), new.to(DEV), [40, 65], top) == na.NA_ERR_CAPACITY


def test_a_page_of_skipped_rows_keeps_its_scale():
    """None of its rows is moved: its bytes stand for what they stood for."""
    import causal_gqa_attention_rope_gb300 as na
    old, new = make_paged([40, 20], 2, 64, 16, "e4m3", 3), make_paged([40, 40], 2, 64, 16, "e4m3", 4)
    a, z = old.to(DEV), new.to(DEV)
    a.page_table = a.page_table.clone()
    a.page_table[0, 1] = old.k.shape[0]
    assert compact(a, z, [40, 20], 40) == na.NA_ERR_PAGE
    skipped, moved = int(new.table[0, 1]), [int(new.table[0, 0]), int(new.table[1, 0])]
    for was, scale, got, got_scale in ((new.k, new.k_scale, z.k, z.k_scale), (new.v, new.v_scale, z.v, z.v_scale)):
        got, got_scale = got.cpu(), got_scale.cpu()
        assert torch.equal(bits(got[skipped]), bits(was[skipped]))
        assert torch.equal(got_scale[skipped], scale[skipped])
        for pid in moved:
            assert not torch.equal(bits(got[pid]), bits(was[pid]))
