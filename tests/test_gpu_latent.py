"""Latent attention: the append, the absorbed form over pages and the expanded form, against the
64-bit statement."""
import math

import pytest
import torch

from harness import Guarded
from latent_ref import attend, make_latent, nan_bf16, rows_of, turn
from paged_ref import bits

pytestmark = pytest.mark.gpu
DEV = "cuda"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def packed(new):
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return cu


def randn(seed, *shape, mag=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * mag).to(torch.bfloat16)


# ----------------------------------------------------------------- append --

APPEND = [  # H, R, rd, page, prior, new, interleaved, yarn, norm, in place
    (32, 512, 64, 64, [0, 70, 1000], [1, 1, 1], True, False, True, False),
    (40, 512, 64, 16, [5, 0, 3, 31], [33, 0, 100, 1], False, True, True, True),
    (1, 128, 16, 32, [63], [70], True, False, False, True),
    (7, 256, 32, 128, [130000, 9], [3, 200], False, False, True, False),
    (130, 256, 48, 16, [0], [17], True, True, True, False),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"H{c[0]}-R{c[1]}-rd{c[2]}-p{c[3]}")
def test_append(case):
    import causal_gqa_attention_rope_gb300 as na
    H, R, rd, page, prior, new, inter, yarn, norm, place = case
    rope = na.RopeConfig(base=1e4, yarn=yarn, factor=4.0, orig_max_pos=2048)
    cfg = na.LatentConfig(H, R, rd, kv_norm=norm, rope_interleaved=inter)
    pool, table = make_latent(prior, R + rd, page, 1, room=max(new))
    T, cu = sum(new), packed(new)
    # the token rows are part of wider ones, and three more rows than there are tokens
    wide_kv, wide_q = randn(2, T + 3, R + rd + 40), randn(3, T + 3, H, 128 + rd)
    w = randn(4, R)
    dkv, dq = wide_kv.to(DEV), wide_q.to(DEV)
    dout = dq if place else torch.full((T + 3, H, R + rd), 7.0, dtype=torch.bfloat16, device=DEV)
    at = 128 if place else R
    cache, status = na.PagedLatentCache(pool.to(DEV), table.to(DEV)), ints([0])
    na.na_latent_append_paged(cfg, rope, ints(cu), ints(prior), dkv[:, 40:], dq[..., 128:],
                              dout[..., at:], cache, kv_norm_w=w.to(DEV) if norm else None, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    pos = torch.cat([torch.arange(p, p + n) for p, n in zip(prior, new)])
    x = wide_kv[:T, 40:].double()
    c = x[:, :R]
    if norm:
        c = c / torch.sqrt(c.square().mean(-1, keepdim=True) + cfg.rms_eps) * w.double()
    row = torch.cat([c, turn(x[:, R:], pos, rope, inter)], dim=-1)
    got, owned, t = cache.kv.cpu(), torch.zeros(pool.shape[:2], dtype=torch.bool), 0
    for b, (p, n) in enumerate(zip(prior, new)):
        for i in range(n):
            pid, slot = int(table[b, (p + i) // page]), (p + i) % page
            owned[pid, slot] = True
            # half a step of bf16, and fp32's few roundings before it (2^-20 of the pair)
            tol = 2.0 ** -8 * row[t].abs() + 2.0 ** -20 * (x[t].abs() + row[t].abs().amax())
            assert ((got[pid, slot].double() - row[t]).abs() <= tol).all()
            if not norm:
                assert torch.equal(bits(got[pid, slot, :R]), bits(wide_kv[t, 40:40 + R]))
            t += 1
    assert torch.equal(bits(got)[~owned], bits(pool)[~owned])
    q = turn(wide_q[:T, :, 128:], pos, rope, inter)
    out = dout.cpu()
    assert ((out[:T, :, at:].double() - q).abs() <= 2.0 ** -8 * q.abs() + 2.0 ** -20 * q.abs().amax()).all()
    rest = wide_q if place else torch.full_like(out, 7.0)
    assert torch.equal(bits(out[T:]), bits(rest[T:])) and torch.equal(bits(out[..., :at]), bits(rest[..., :at]))


def test_append_reports_and_queries_left_out():
    import causal_gqa_attention_rope_gb300 as na
    cfg = na.LatentConfig(4, 128, 32, kv_norm=False)
    pool, table = make_latent([10, 30], 160, 16, 1, room=2)
    cache, status = na.PagedLatentCache(pool.to(DEV), table.to(DEV)), ints([0])
    kv = randn(2, 4, 160).to(DEV)
    na.na_latent_append_paged(cfg, na.RopeConfig(), ints([0, 2, 4]), ints([10, 30]), kv, None, None, cache,
                              status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(bits(rows_of(cache.kv.cpu(), table, 0, 12)[10:, :128]), bits(kv.cpu()[:2, :128]))
    before = cache.kv.clone()
    na.na_latent_append_paged(cfg, na.RopeConfig(), ints([0, 2, 4]), ints([32, 48]), kv, None, None, cache,
                              status=status)  # past the tables
    torch.cuda.synchronize()
    assert int(status.item()) == na.NA_ERR_CAPACITY and torch.equal(bits(cache.kv), bits(before))
    status.zero_()
    cache.page_table[0, 0] = pool.shape[0]
    na.na_latent_append_paged(cfg, na.RopeConfig(), ints([0, 2, 2]), ints([0, 0]), kv[:2], None, None, cache,
                              status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == na.NA_ERR_PAGE and torch.equal(bits(cache.kv), bits(before))


# --------------------------------------------------------------- absorbed --

def absorbed(cfg, pool, table, prior, new, q, extra=0, bounds=None, stream=None, workspace=None):
    import causal_gqa_attention_rope_gb300 as na
    T = sum(new)
    cache = na.PagedLatentCache(pool.to(DEV), table.to(DEV))
    most, top = bounds or (max(new), max(p + n for p, n in zip(prior, new)))
    status = ints([0])
    out = Guarded((T + extra, cfg.num_heads, cfg.kv_rank), torch.bfloat16, fill=3.0)
    ws = workspace
    if ws is None:
        ws = na.workspace(na.na_latent_paged_workspace_size(cfg, len(new), T + extra, most, top), DEV)
        ws.fill_(0xFF)  # NaN bits: nothing of it is read before it is written
    na.na_attn_latent_paged(cfg, ints(packed(new)), ints(prior), most, top, q.to(DEV), cache, out.t,
                            workspace=ws, status=status, stream=stream)
    torch.cuda.synchronize()
    out.check("out")
    return out.t.cpu(), int(status.item())


def check_absorbed(H, R, rd, page, prior, new, seed=0, extra=0, bounds=None, mag=1.0, pool=None, q=None):
    import causal_gqa_attention_rope_gb300 as na
    cfg = na.LatentConfig(H, R, rd)
    lens = [p + n for p, n in zip(prior, new)]
    if pool is None:
        pool = make_latent(lens, R + rd, page, seed + 1, mag=mag)
    T = sum(new)
    if q is None:
        q = randn(seed + 2, T + extra, H, R + rd, mag=mag)
    out, status = absorbed(cfg, *pool, prior, new, q, extra, bounds)
    assert status == 0
    t = 0
    for b, (p, n) in enumerate(zip(prior, new)):
        if n == 0:
            continue
        rows = rows_of(*pool, b, p + n)[None]
        ref, tol = attend(q[t:t + n], rows, rows[..., :R], torch.arange(p + 1, p + n + 1),
                          1 / math.sqrt(cfg.nope_dim + rd))
        assert ((out[t:t + n].double() - ref).abs() <= tol).all(), (b, p, n)
        t += n
    assert (out[T:] == 3.0).all()


@pytest.mark.parametrize("R,rd", [(512, 64), (256, 64), (128, 32), (512, 16), (128, 48)])
@pytest.mark.parametrize("H,page", [(16, 64), (7, 16)])
def test_absorbed_single_tokens(R, rd, H, page):
    check_absorbed(H, R, rd, page, [0, 1, 62, 63, 64, 200, 511], [1] * 7)


@pytest.mark.parametrize("H", [1, 4, 32, 40, 64, 65, 128, 200])
def test_absorbed_heads(H):
    check_absorbed(H, 256, 64, 32, [100, 300], [1, 1], seed=H)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_absorbed_chunks(page):
    check_absorbed(5, 512, 64, page, [0, 70, 0, 127, 4], [30, 1, 0, 90, 13], seed=page)


def test_absorbed_long_and_short_together():
    check_absorbed(4, 128, 32, 64, [9000, 0, 33, 5000, 2], [1, 3, 1, 2, 1])


def test_absorbed_one_long_sequence_over_all_ctas():
    check_absorbed(16, 512, 64, 32, [20000], [1])


def test_absorbed_fresh_prompt():
    """Units that see more and more keys, over 64 per sequence (counted by whole warps)."""
    check_absorbed(24, 128, 64, 64, [0, 50], [400, 90])


def test_absorbed_many_sequences():
    check_absorbed(8, 128, 32, 16, [(37 * b) % 150 for b in range(700)], [b % 3 for b in range(700)])


def test_absorbed_padded_batch_and_loose_bounds():
    check_absorbed(12, 256, 64, 32, [60, 5], [2, 7], extra=6, bounds=(9, 64))
    check_absorbed(12, 256, 64, 128, [60, 5], [2, 7], extra=9, bounds=(8, 128))


def test_absorbed_growing_scores():
    """Later keys score higher and higher: the reference maximum is raised, rows rescaled."""
    import causal_gqa_attention_rope_gb300 as na  # noqa: F401
    pool, table = make_latent([1500], 320, 64, 5)
    flat = pool[table[0, :24].long()].flatten(0, 1)
    q = randn(6, 1, 20, 320)
    up = torch.linspace(0, 6, flat.shape[0])[:, None] * q[0, 3].float() / q[0, 3].float().norm()
    flat = (flat.float() + up).to(torch.bfloat16)
    flat[1500:] = nan_bf16(1, 1)
    pool[table[0, :24].long()] = flat.view(24, 64, 320)
    check_absorbed(20, 256, 64, 64, [1499], [1], pool=(pool, table), q=q)


@pytest.mark.parametrize("k", range(1, 9))
@pytest.mark.parametrize("H,R,rd", [(5, 512, 64), (40, 128, 32), (64, 256, 48)])
def test_absorbed_short_contexts(H, R, rd, k):
    """k tiles in as many pieces, joined in a cluster; beside them sequences with fewer tiles."""
    check_absorbed(H, R, rd, 64, [64 * k - 30], [1], seed=k)
    check_absorbed(H, R, rd, 16, [64 * k - 1, 2, 64], [1, 1, 1], seed=k)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("R,rd", [(512, 64), (256, 48), (128, 16)])
def test_absorbed_many_rows_of_long_contexts(R, rd, page):
    """Units of 128 rows in pairs of CTAs, whole and in pieces; the second CTA's half without rows."""
    check_absorbed(24, R, rd, page, [5000, 3, 2000, 10, 777], [9, 1, 4, 0, 6], seed=page)
    check_absorbed(131, R, rd, page, [4095], [1], seed=page + 1)


@pytest.mark.parametrize("R", [512, 256])
def test_absorbed_growing_scores_in_pairs(R):
    """Rows of either CTA raise their reference maxima, in tiles of either group."""
    n = 6100
    pool, table = make_latent([n], R + 64, 64, 15)
    pages = table[0, :-(-n // 64)].long()
    flat = pool[pages].flatten(0, 1)
    q = randn(16, 1, 100, R + 64)
    up = torch.linspace(0, 6, len(flat))[:, None]
    for h in (3, 77, 99):
        flat = (flat.float() + up * q[0, h].float() / q[0, h].float().norm()).to(torch.bfloat16)
        up = (up * 1.3).roll(64 * h, 0)
    flat[n:] = nan_bf16(1, 1)
    pool[pages] = flat.view(len(pages), 64, R + 64)
    check_absorbed(100, R, 64, 64, [n - 1], [1], pool=(pool, table), q=q)


def test_absorbed_reports_in_pairs():
    import causal_gqa_attention_rope_gb300 as na
    cfg = na.LatentConfig(100, 256, 64)
    pool, table = make_latent([4000, 50], 320, 32, 3)
    q = randn(4, 2, 100, 320)
    bad = table.clone()
    bad[0, 77] = pool.shape[0]
    out, status = absorbed(cfg, pool, bad, [3999, 49], [1, 1], q)
    assert status == na.NA_ERR_PAGE
    rows = rows_of(pool, table, 1, 50)[None]
    ref, tol = attend(q[1:], rows, rows[..., :256], torch.tensor([50]), 1 / math.sqrt(192))
    assert ((out[1:].double() - ref).abs() <= tol).all()
    out, status = absorbed(cfg, pool, table, [3999, 49], [1, 1], q, bounds=(1, 3999))
    assert status == na.NA_ERR_CAPACITY and (out[:1] == 3.0).all()
    assert ((out[1:].double() - ref).abs() <= tol).all()


def test_absorbed_large_values():
    check_absorbed(9, 512, 64, 64, [300, 20], [1, 4], mag=3.0)


def test_absorbed_reports():
    import causal_gqa_attention_rope_gb300 as na
    cfg = na.LatentConfig(4, 128, 32)
    pool, table = make_latent([40, 50], 160, 16, 1)
    q = randn(2, 3, 4, 160)
    out, status = absorbed(cfg, pool, table, [38, 49], [2, 1], q, bounds=(1, 50))
    assert status == na.NA_ERR_INVALID_ARG and (out[:2] == 3.0).all() and not (out[2] == 3.0).any()
    out, status = absorbed(cfg, pool, table, [38, 49], [2, 1], q, bounds=(2, 45))
    assert status == na.NA_ERR_CAPACITY and (out[2] == 3.0).all() and not (out[:2] == 3.0).any()
    bad = table.clone()
    bad[0, 1] = pool.shape[0]
    out, status = absorbed(cfg, pool, bad, [38, 49], [2, 1], q)
    assert status == na.NA_ERR_PAGE
    ref, tol = attend(q[2:], rows_of(pool, table, 1, 50)[None], rows_of(pool, table, 1, 50)[None, :, :128],
                      torch.tensor([50]), 1 / math.sqrt(160))
    assert ((out[2:].double() - ref).abs() <= tol).all()


# --------------------------------------------------------------- expanded --

def check_expanded(H, dn, rd, dv, new, lens, seed=0, extra=0, shared=False):
    import causal_gqa_attention_rope_gb300 as na
    cfg = na.LatentConfig(H, rope_dim=rd, nope_dim=dn, v_dim=dv)
    T, cu = sum(new), packed(new)
    starts, at = [], 3
    for n in lens:
        starts.append(3 if shared else at)
        at += n + 2  # rows between that nobody reads
    at = 3 + max(lens) if shared else at
    kv, wide = nan_bf16(at, H, dn + dv), nan_bf16(at, 64 + rd)
    for s, n in zip(starts, lens):
        if n:
            kv[s:s + n], wide[s:s + n, 64:] = randn(seed + s, n, H, dn + dv), randn(seed + s + 1, n, rd)
    q = randn(seed + 9, T + extra, H, dn + rd)
    status = ints([0])
    out = Guarded((T + extra, H, dv), torch.bfloat16, fill=3.0)
    na.na_attn_latent_expanded(cfg, ints(cu), ints(starts), ints(lens), max(new), max(lens), q.to(DEV),
                               kv.to(DEV), wide.to(DEV)[:, 64:], out.t, status=status)
    torch.cuda.synchronize()
    out.check("out")
    assert int(status.item()) == 0
    got = out.t.cpu()
    for b, n in enumerate(new):
        if n == 0:
            continue
        s, m = starts[b], lens[b]
        k = torch.cat([kv[s:s + m, :, :dn], wide[s:s + m, None, 64:].expand(-1, H, -1)], dim=-1)
        ref, tol = attend(q[cu[b]:cu[b] + n], k.transpose(0, 1), kv[s:s + m, :, dn:].transpose(0, 1),
                          torch.arange(m - n + 1, m + 1), 1 / math.sqrt(dn + rd))
        assert ((got[cu[b]:cu[b] + n].double() - ref).abs() <= tol).all(), b
    assert (got[T:] == 3.0).all()


@pytest.mark.parametrize("dn,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("rd", [64, 32, 16])
def test_expanded_shapes(dn, dv, rd):
    check_expanded(3, dn, rd, dv, [130, 1, 0, 77], [300, 1, 40, 77], seed=rd)


def test_expanded_rows_that_see_nothing():
    """More tokens than keys: the first rows are zeros, whole tiles of them too."""
    check_expanded(2, 128, 64, 128, [140, 300, 5, 4], [130, 20, 0, 3])


def test_expanded_padded_batch_and_many_sequences():
    check_expanded(2, 64, 64, 64, [5, 9], [50, 9], extra=7)
    check_expanded(1, 64, 32, 64, [1 + b % 5 for b in range(50)], [1 + 7 * b for b in range(50)])


def test_expanded_shared_keys_and_long_context():
    check_expanded(5, 128, 64, 128, [3, 200], [900, 900], shared=True)
    check_expanded(2, 128, 64, 128, [257], [4000])


@pytest.mark.parametrize("dn,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("rd,new,lens", [
    (64, [300], [1437]),                # two units of 256 rows, the last of less than a tile
    (32, [2900], [2600]),               # whole tiles see nothing
    (64, [512, 640, 1, 0, 900], [512, 2000, 1, 40, 1300]),
])
def test_expanded_cut_into_pieces(dn, dv, rd, new, lens):
    """Few units with many keys: clusters, some of whose CTAs have no keys."""
    check_expanded(2, dn, rd, dv, new, lens, seed=dn + dv)


def test_expanded_tall_units():
    """More units of 256 rows than SMs."""
    check_expanded(80, 64, 64, 64, [200, 270], [1100, 1300])


def test_expanded_prompts_of_many_lengths():
    """Enough units for two CTAs on every SM, most of them ending inside a tile; NaN between sequences."""
    import random

    import causal_gqa_attention_rope_gb300 as na
    r, H = random.Random(11), 32
    new = [r.randint(1, 512) for _ in range(16)]
    lens = [n + r.randint(0, 1000) for n in new]
    starts, at = [], 0
    for n in lens:
        starts.append(at)
        at += n + 70
    cfg, T, cu = na.LatentConfig(H, rope_dim=64, nope_dim=128, v_dim=128), sum(new), packed(new)
    g = torch.Generator(device=DEV).manual_seed(5)
    q, kv, pe = (torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)
                 for s in ((T, H, 192), (at, H, 256), (at, 64)))
    for s, n in zip(starts, lens):
        kv[s + n:s + n + 70], pe[s + n:s + n + 70] = math.nan, math.nan
    out, status = torch.full((T, H, 128), 3.0, dtype=torch.bfloat16, device=DEV), ints([0])
    heads = [0, 13, 31]
    want = []
    for b, n in enumerate(new):
        k0, m = starts[b], lens[b]
        kv_b, pe_b = kv[k0:k0 + m][:, heads].cpu(), pe[k0:k0 + m].cpu()
        k = torch.cat([kv_b[..., :128], pe_b[:, None].expand(-1, len(heads), -1)], dim=-1)
        want.append(attend(q[cu[b]:cu[b + 1]][:, heads].cpu(), k.transpose(0, 1),
                           kv_b[..., 128:].transpose(0, 1), torch.arange(m - n + 1, m + 1), 1 / math.sqrt(192)))
    for _ in range(5):
        out.fill_(3.0)
        na.na_attn_latent_expanded(cfg, ints(cu), ints(starts), ints(lens), max(new), max(lens), q, kv, pe, out,
                                   status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        for b, (ref, tol) in enumerate(want):
            got = out[cu[b]:cu[b + 1]][:, heads].cpu().double()
            assert ((got - ref).abs() <= tol).all(), b
        assert not torch.isnan(out).any()


def test_expanded_last_wave_cut():
    """160 equal units of 4100 keys and more: those after the last whole wave are cut."""
    import causal_gqa_attention_rope_gb300 as na
    H, n, m = 160, 150, 4170
    cfg = na.LatentConfig(H, rope_dim=64, nope_dim=64, v_dim=128)
    g = torch.Generator(device=DEV).manual_seed(4)
    q, kv, pe = (torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)
                 for s in ((n, H, 128), (m, H, 192), (m, 64)))
    out, status = torch.full((n, H, 128), 3.0, dtype=torch.bfloat16, device=DEV), ints([0])
    na.na_attn_latent_expanded(cfg, ints([0, n]), ints([0]), ints([m]), n, m, q, kv, pe, out, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    heads = [0, 1, 80] + list(range(148, 160))
    q, kv, pe, got = (x.cpu() for x in (q[:, heads], kv[:, heads], pe, out[:, heads]))
    k = torch.cat([kv[..., :64], pe[:, None].expand(-1, len(heads), -1)], dim=-1)
    ref, tol = attend(q, k.transpose(0, 1), kv[..., 64:].transpose(0, 1),
                      torch.arange(m - n + 1, m + 1), 1 / math.sqrt(128))
    assert ((got.double() - ref).abs() <= tol).all()
    assert not (out == 3.0).all(dim=-1).any()


def test_expanded_reports():
    import causal_gqa_attention_rope_gb300 as na
    cfg = na.LatentConfig(2, rope_dim=32, nope_dim=64, v_dim=64)
    q, kv, pe = randn(1, 5, 2, 96).to(DEV), randn(2, 40, 2, 128).to(DEV), randn(3, 40, 32).to(DEV)

    def status_of(starts, lens, most=3, top=40):
        status, out = ints([0]), torch.full((5, 2, 64), 3.0, dtype=torch.bfloat16, device=DEV)
        na.na_attn_latent_expanded(cfg, ints([0, 3, 5]), ints(starts), ints(lens), most, top, q, kv, pe, out,
                                   status=status)
        torch.cuda.synchronize()
        return int(status.item()), (out == 3.0).flatten(1).all(dim=1).tolist()

    assert status_of([0, 10], [10, 30]) == (0, [False] * 5)
    skip0, skip1 = [True] * 3 + [False] * 2, [False] * 3 + [True] * 2
    assert status_of([0, 10], [10, 30], most=2) == (na.NA_ERR_INVALID_ARG, skip0)
    assert status_of([0, 10], [10, 31]) == (na.NA_ERR_CAPACITY, skip1)
    assert status_of([0, 10], [10, 30], top=29) == (na.NA_ERR_CAPACITY, skip1)
    assert status_of([-1, 10], [10, 30]) == (na.NA_ERR_CAPACITY, skip0)
    assert status_of([0, 10], [-1, 30]) == (na.NA_ERR_CAPACITY, skip0)


# --------------------------------------------------------------- together --

def test_a_prompt_then_tokens_in_both_forms():
    """Rows appended in two chunks; the same queries through both forms, the maps in 64 bits; then the
    sequence forked, its copy evicted to half and attended again."""
    import causal_gqa_attention_rope_gb300 as na
    H, R, rd, dn, dv, page, T = 6, 128, 32, 64, 64, 16, 75
    cfg = na.LatentConfig(H, R, rd, dn, dv, rope_interleaved=True)
    rope = na.RopeConfig(base=1e4)
    pool, table = make_latent([0, 0], R + rd, page, 1, room=T + 5)
    cache, status = na.PagedLatentCache(pool.to(DEV), table.to(DEV)), ints([0])
    kv, w = randn(2, T, R + rd).to(DEV), randn(3, R).to(DEV)
    up_k, up_v = randn(4, H, dn, R, mag=R ** -0.5), randn(5, H, dv, R, mag=R ** -0.5)
    q = randn(6, T, H, dn + rd).to(DEV)
    q_rot, q_lat = q.clone(), torch.zeros(T, H, R + rd, dtype=torch.bfloat16, device=DEV)
    for a, z in ((0, 50), (50, T)):
        for dst in (q_rot[a:z, :, dn:], q_lat[a:z, :, R:]):
            na.na_latent_append_paged(cfg, rope, ints([0, z - a, z - a]), ints([a, 0]), kv[a:z], q[a:z, :, dn:],
                                      dst, cache, kv_norm_w=w, status=status)
    assert torch.equal(bits(q_rot[..., dn:]), bits(q_lat[..., R:]))
    q_lat[..., :R] = torch.einsum("thd,hdr->thr", q[..., :dn].double().cpu(), up_k.double()).to(torch.bfloat16)
    out = torch.zeros(T, H, R, dtype=torch.bfloat16, device=DEV)
    ws = na.workspace(na.na_latent_paged_workspace_size(cfg, 2, T, T, T), DEV)
    na.na_attn_latent_paged(cfg, ints([0, T, T]), ints([0, 0]), T, T, q_lat, cache, out, workspace=ws,
                            status=status)
    # the rows out of their pages, expanded
    flat = torch.zeros(5, page, R + rd, dtype=torch.bfloat16, device=DEV)
    na.na_pages_compact(cache, na.PagedLatentCache(flat, ints([list(range(5)), [-1] * 5])), ints([T, 0]), T,
                        status=status)
    rows = flat.flatten(0, 1)[:T]
    assert torch.equal(bits(rows.cpu()), bits(rows_of(cache.kv.cpu(), table, 0, T)))
    c = rows[:, :R].double().cpu()
    kv_big = torch.cat([torch.einsum("tr,hdr->thd", c, up_k.double()),
                        torch.einsum("tr,hdr->thd", c, up_v.double())], dim=-1).to(DEV, torch.bfloat16)
    direct = torch.zeros(T, H, dv, dtype=torch.bfloat16, device=DEV)
    na.na_attn_latent_expanded(cfg, ints([0, T]), ints([0]), ints([T]), T, T, q_rot, kv_big, rows[:, R:], direct,
                               status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    through = torch.einsum("thr,hdr->thd", out.double().cpu(), up_v.double())
    # Both within their roundings of the same numbers: the queries', keys' and values' to bf16 (2^-8
    # each: of scores of size ~4 and of values) and the results'; together below 2^-8 (4 + 4 + 1 + 1).
    assert (through - direct.double().cpu()).abs().max() <= 10 * 2.0 ** -8 * through.abs().max()
    # two children of the sequence; the second one's last page is its own
    ref = torch.zeros(pool.shape[0], dtype=torch.int32, device=DEV)
    ref[cache.page_table[0, :5].long()] = 1
    table1 = torch.full_like(cache.page_table, -1)
    table1[0, :5] = cache.page_table[0, :5]
    outs = [torch.zeros(s, dtype=torch.int32, device=DEV) for s in (table1.shape, ref.shape, (2,), (2,), (2,))]
    na.na_pages_fork(ints([0, 0]), ints([T, 0]), table1, ref, page, *outs, status=status)
    forked = na.PagedLatentCache(cache.kv, outs[0])
    na.na_pages_copy(forked, outs[3], outs[4], status=status)
    keep = list(range(0, T, 2))
    free = [i for i, n in enumerate(outs[1].tolist()) if n == 0][:3]
    half = na.PagedLatentCache(cache.kv, ints([free]))
    na.na_pages_compact(na.PagedLatentCache(cache.kv, outs[0][1:]), half, ints([len(keep)]), len(keep),
                        keep=ints([keep]), rope=rope, rotary_start=R, interleaved=True, status=status)
    got = torch.zeros(1, H, R, dtype=torch.bfloat16, device=DEV)
    na.na_attn_latent_paged(cfg, ints([0, 1]), ints([len(keep) - 1]), 1, 48, q_lat[:1], half, got,
                            workspace=ws, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    kept = rows.cpu().double()[keep]
    kept[:, R:] = turn(kept[:, R:], torch.arange(len(keep)) - torch.tensor(keep), rope, True)
    kept = kept.to(torch.bfloat16)[None]
    want, tol = attend(q_lat[:1].cpu(), kept, kept[..., :R], torch.tensor([len(keep)]), 1 / math.sqrt(dn + rd))
    # the kept rows' second rounding may fall to the other side of a border: one more step of a score
    tol = tol + 2.0 ** -8 * want.abs().amax()
    assert ((got.cpu().double() - want).abs() <= tol).all()


def test_streams_and_graphs():
    """The append and both forms on a side stream, then captured and replayed twice: the same bits;
    two calls at once have their own workspaces."""
    import causal_gqa_attention_rope_gb300 as na
    H, R, rd, page = 16, 256, 64, 32
    cfg, rope = na.LatentConfig(H, R, rd, 64, 64), na.RopeConfig()
    prior, new = [300, 40, 2000], [1, 1, 1]
    pool, table = make_latent(prior, R + rd, page, 1, room=1)
    cache, status = na.PagedLatentCache(pool.to(DEV), table.to(DEV)), ints([0])
    kv, q, w = randn(2, 3, R + rd).to(DEV), randn(3, 3, H, R + rd).to(DEV), randn(4, R).to(DEV)
    cu, lens = ints([0, 1, 2, 3]), ints(prior)
    size = na.na_latent_paged_workspace_size(cfg, 3, 3, 1, 2001)
    big_kv, big_q = randn(5, 200, H, 128).to(DEV), randn(6, 3, H, 128).to(DEV)
    streams = [torch.cuda.Stream() for _ in range(2)]
    qs = [q.clone() for _ in streams]
    outs = [torch.zeros(3, H, R, dtype=torch.bfloat16, device=DEV) for _ in streams]
    wide = [torch.zeros(3, H, 64, dtype=torch.bfloat16, device=DEV) for _ in streams]
    spaces = [na.workspace(size, DEV) for _ in streams]

    def step(i):
        qs[i].copy_(q)
        na.na_latent_append_paged(cfg, rope, cu, lens, kv, qs[i][..., R:], qs[i][..., R:], cache, kv_norm_w=w,
                                  status=status)
        na.na_attn_latent_paged(cfg, cu, lens, 1, 2001, qs[i], cache, outs[i], workspace=spaces[i], status=status)
        na.na_attn_latent_expanded(cfg, cu, ints_0, ints_200, 1, 200, big_q, big_kv, kv200, wide[i], status=status)

    ints_0, ints_200, kv200 = ints([0, 0, 0]), ints([200, 200, 150]), randn(7, 200, rd).to(DEV)
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                step(i)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(bits(outs[0]), bits(outs[1])) and torch.equal(bits(wide[0]), bits(wide[1]))
    first = [t.clone() for t in (outs[0], wide[0], cache.kv)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(0)
    outs[0].zero_()
    wide[0].zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, (outs[0], wide[0], cache.kv)):
        assert torch.equal(bits(a), bits(b))


def test_readme_example_runs():
    """The README's latent example as written, its rows and both forms finite, the fork's copy equal."""
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    first, latent = (re.findall(rf"```{kind}\n(.*?)```", text, flags=re.S)[0] for kind in ("python", "py"))
    scope = {}
    for block in (first, latent):
        exec(compile(block, "README example", "exec"), scope)
    assert torch.isfinite(scope["out"].float()).all() and torch.isfinite(scope["out1"].float()).all()
    two, page = scope["two"], int(scope["dst"][1])
    assert scope["new_lens"].tolist() == [129, 129] and two.page_table[1, :3].tolist() == [0, 1, page]
    assert torch.equal(bits(two.kv[page]), bits(two.kv[2]))


def test_long_contexts_at_once_and_captured():
    """Absorbed pairs and expanded pieces, clusters both, on two streams at once; then captured."""
    import causal_gqa_attention_rope_gb300 as na
    H, R, n, m = 72, 256, 3, 6000
    cfg = na.LatentConfig(H, R, 64, 64, 64)
    pool, table = make_latent([m], R + 64, 64, 1)
    cache, status = na.PagedLatentCache(pool.to(DEV), table.to(DEV)), ints([0])
    g = torch.Generator(device=DEV).manual_seed(8)
    q, big_q, kv, pe = (torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)
                        for s in ((n, H, R + 64), (300, H, 128), (m, H, 128), (m, 64)))
    cu, prior, cu_big, zero, keys = ints([0, n]), ints([m - n]), ints([0, 300]), ints([0]), ints([m])
    size = na.na_latent_paged_workspace_size(cfg, 1, n, n, m)
    outs = [torch.zeros(n, H, R, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    wide = [torch.zeros(300, H, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    spaces = [na.workspace(size, DEV) for _ in range(2)]

    def step(i):
        na.na_attn_latent_paged(cfg, cu, prior, n, m, q, cache, outs[i], workspace=spaces[i], status=status)
        na.na_attn_latent_expanded(cfg, cu_big, zero, keys, 300, m, big_q, kv, pe, wide[i], status=status)

    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                step(i)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(bits(outs[0]), bits(outs[1])) and torch.equal(bits(wide[0]), bits(wide[1]))
    first = outs[0].clone(), wide[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(0)
    outs[0].zero_()
    wide[0].zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(first[0]), bits(outs[0])) and torch.equal(bits(first[1]), bits(wide[0]))
    rows = rows_of(pool, table, 0, m)[None]
    ref, tol = attend(q.cpu(), rows, rows[..., :R], torch.arange(m - n + 1, m + 1), 1 / math.sqrt(128))
    assert ((first[0].cpu().double() - ref).abs() <= tol).all()
