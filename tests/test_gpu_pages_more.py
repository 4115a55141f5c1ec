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


@pytest.mark.parametrize("rd", [0, 64, 34])
@pytest.mark.parametrize("scales", [(254, 254, 254), (254, 0, 250), (247, 246, 130), (0, 0, 0), (1, 254, 0)], ids=str)
def test_compact_of_scales_beyond_fp32(scales, rd):
    """Stored values of 448 * 2^127 exceed fp32; what they stand for is moved all the same."""
    import causal_gqa_attention_rope_gb300 as na
    KV, d, page, new_page = 2, 64, 16, 32
    old, new = make_paged([48], KV, d, page, "e4m3", 5), make_paged([0], KV, d, new_page, "e4m3", 6, room=48)
    for pool, scale in ((old.k, old.k_scale), (old.v, old.v_scale)):
        if rd:  # a turn makes 2^0.5 of a value at most: 362 of 256
            pool.view(torch.uint8).copy_((pool.float() / 2).to(pool.dtype).view(torch.uint8))
        for i, s in enumerate(scales):
            scale[old.table[0, i]] = s
    keep = list(range(3, 9)) + list(range(20, 30)) + [46, 33, 40, 47, 10] + list(range(11, 16)) + list(range(40, 48))
    rope = na.RopeConfig(base=1e4)
    z = new.to(DEV)
    assert compact(old.to(DEV), z, [len(keep)], len(keep), keep=ints([keep]), rope=rope if rd else None,
                   rotary_dim=rd) == 0
    at = torch.tensor(keep)
    for pool, scale, got, got_scale, is_k in ((old.k, old.k_scale, z.k.cpu(), z.k_scale.cpu(), True),
                                              (old.v, old.v_scale, z.v.cpu(), z.v_scale.cpu(), False)):
        for lo in range(0, len(keep), new_page):
            rows = at[lo:lo + new_page]
            sid, pid = old.table[0, rows // page].long(), int(new.table[0, lo // new_page])
            x = pool.view(torch.uint8)[sid, :, rows % page].view(pool.dtype).double()
            x = x * torch.exp2(scale[sid].double() - 127)[..., None]
            if rd and is_k:
                x = turned(x, (torch.arange(lo, lo + len(rows)) - rows)[:, None], rope, 0, rd)
            amax, e = x.abs().amax(dim=(0, 2)), got_scale[pid].double() - 127
            near = 2.0 ** -20  # of the page's largest, as fp32 turns it
            assert (amax * (1 - near) <= 448 * torch.exp2(e)).all()
            assert ((amax * (1 + near) > 448 * torch.exp2(e - 1)) | (e == -127)).all()
            y = got[pid, :, :len(rows)].permute(1, 0, 2).contiguous().double() * torch.exp2(e)[:, None]
            # half a step of E4M3: 2^-4 of the value, 2^-10 of the scale below its normal range
            tol = 2.0 ** -4 * x.abs() + torch.exp2(e - 10)[:, None] + near * amax[:, None]
            assert ((y - x).abs() <= tol).all()
