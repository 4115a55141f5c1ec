"""Forks of page tables, copies of pages and compaction, against the host statement."""
import random

import pytest
import torch

from pages_ref import fork, turned
from paged_ref import bits, make_paged

pytestmark = pytest.mark.gpu
DEV = "cuda"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def run_fork(parents, grow, lens, table, page, ref, stream=None):
    import causal_gqa_attention_rope_gb300 as na
    B, P = len(parents), len(table[0])
    out = [torch.full(s, -9, dtype=torch.int32, device=DEV) for s in ((B, P), (len(ref),), (B,), (B,), (B,))]
    status = ints([0])
    na.na_pages_fork(ints(parents), ints(lens), ints(table), ints(ref), page, *out,
                     grow=None if grow is None else ints(grow), status=status, stream=stream)
    torch.cuda.synchronize()
    return [t.tolist() for t in out] + [int(status.item())]


CODES = {"argument": -1, "capacity": -3, "page": -7}


def check_fork(*args):
    got, want = run_fork(*args), fork(*args)
    for g, w, what in zip(got, want, ("table", "ref", "lens", "src", "dst")):
        assert g == w, what
    assert got[5] in ({CODES[w] for w in want[5]} or {0})
    return got


def a_batch(r, B, page, most, pages_free, P=None):
    lens = [r.choice((0, 1, page - 1, page, page + 1, r.randint(0, most))) for _ in range(B)]
    per = [-(-n // page) + (r.random() < 0.3) for n in lens]
    P = P or max(per) + 2
    ids = list(range(sum(per) + pages_free))
    r.shuffle(ids)
    table, at = [], 0
    for n in per:
        table.append(ids[at:at + n] + [-1] * (P - n))
        at += n
    ref = [0] * len(ids)
    for row in table:
        for e in row:
            if e >= 0:
                ref[e] += 1
    return lens, table, ref


@pytest.mark.parametrize("B,page,most,seed", [(1, 16, 40, 0), (2, 128, 1000, 1), (7, 32, 300, 2),
                                              (64, 64, 8192, 3), (257, 16, 2000, 4), (1100, 16, 90, 5)])
def test_fork(B, page, most, seed):
    r = random.Random(seed)
    lens, table, ref = a_batch(r, B, page, most, 4 * B)
    for _ in range(3):
        parents = [r.choice((-1, b, r.randrange(B), r.randrange(max(1, B // 4)))) for b in range(B)]
        grow = [r.choice((0, 1, page, r.randint(0, 2 * page))) for _ in range(B)]
        P = len(table[0])
        grow = [min(g, P * page - (lens[p] if p >= 0 else 0)) for g, p in zip(grow, parents)]
        got = check_fork(parents, grow, lens, table, page, ref)
        # the next step, from this one's results
        table, ref = got[0], got[1]
        lens = [n + g for n, g in zip(got[2], grow)]
        if got[5]:
            break
        assert sum(ref) == sum(e >= 0 for row in table for e in row)


def test_fork_to_another_batch_size():
    r = random.Random(9)
    lens, table, ref = a_batch(r, 5, 32, 200, 20)
    check_fork([4, 4, 4, 0, -1, 4, 0, 2], None, lens, table, 32, ref)
    check_fork([3], [5], lens, table, 32, ref)


def test_fork_keeps_counts_of_other_holders():
    """Pages that something else holds too do not become free when their sequence ends."""
    got = check_fork([-1, 0], [16, 0], [32, 20], [[2, 0, -1], [1, 3, -1]], 16, [2, 1, 1, 1, 0])
    assert got[1][0] >= 1 and 0 not in got[0][0]


def test_fork_reports():
    full = [[0, 1], [2, 3]]
    ok = (full, 16, [1, 1, 1, 1])
    assert check_fork([5, 1], None, [32, 32], *ok)[5] == CODES["argument"]
    assert check_fork([0, 1], [-1, 0], [32, 32], *ok)[5] == CODES["argument"]
    assert check_fork([0, 1], [1, 0], [32, 32], *ok)[5] == CODES["capacity"]      # row full
    assert check_fork([0, 0], [0, 0], [32, 20], *ok)[5] == 0                      # whole pages shared
    assert check_fork([1, 1, 1, 0], None, [32, 20], *ok)[5] == CODES["capacity"]  # no page free
    assert check_fork([0, 1], None, [40, 32], *ok)[5] == CODES["page"]            # fewer pages than tokens
    assert check_fork([0, 1], None, [16, 32], [[0, 9], [2, 3]], 16, [1, 0, 1, 1])[5] == CODES["page"]


@pytest.mark.parametrize("fmt,KV,d,page", [("bf16", 8, 128, 64), ("e4m3", 2, 64, 16),
                                           ("latent", 1, 576, 16), ("bf16", 3, 72, 32), ("e4m3", 5, 128, 128)])
def test_copy(fmt, KV, d, page):
    import causal_gqa_attention_rope_gb300 as na
    g = torch.Generator().manual_seed(7)
    n = 40
    shape = (n, page, d) if fmt == "latent" else (n, KV, page, d)
    size = 1 if fmt == "e4m3" else 2
    raw = [torch.randint(0, 256, (*shape[:-1], d * size), generator=g, dtype=torch.uint8) for _ in range(2)]
    scales = [torch.randint(0, 256, (n, KV), generator=g, dtype=torch.uint8) for _ in range(2)]
    kind = torch.float8_e4m3fn if fmt == "e4m3" else torch.bfloat16
    dev = [t.to(DEV).view(kind) for t in raw]
    dsc = [t.to(DEV) for t in scales]
    order = torch.randperm(n, generator=g)
    src, dst = order[:15].int(), order[15:30].int()
    src[3], dst[5], src[7], dst[7] = -1, -2, -1, -1
    if fmt == "latent":
        cache = na.PagedLatentCache(dev[0], None)
    elif fmt == "e4m3":
        cache = na.PagedKVCache(*dev, None, *dsc)
    else:
        cache = na.PagedKVCache(*dev, None)
    status = ints([0])
    na.na_pages_copy(cache, src.to(DEV), dst.to(DEV), status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    real = (src >= 0) & (dst >= 0)
    for i, (t, s) in enumerate(zip(raw, scales)):
        if fmt != "latent" or i == 0:
            t[dst[real].long()] = t[src[real].long()]
        if fmt == "e4m3":
            s[dst[real].long()] = s[src[real].long()]
        assert torch.equal(dev[i].view(torch.uint8).cpu(), t)
        assert torch.equal(dsc[i].cpu(), s)
    na.na_pages_copy(cache, ints([n, 0]), ints([0, n + 5]), status=status)
    na.na_pages_copy(cache, ints([]), ints([]), status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == na.NA_ERR_PAGE
    assert torch.equal(dev[0].view(torch.uint8).cpu(), raw[0])


def keeps(r, lens, part):
    out = []
    for n in lens:
        m = 0 if n == 0 else max(1, round(n * part))
        keep = sorted(r.sample(range(n), m))
        if m > 2 and r.random() < 0.3:
            r.shuffle(keep)  # any order will do, and a position twice
            keep[0] = keep[1]
        out.append(keep)
    return out


CASES = [  # fmt, KV, d, page, new page, lens, part kept, rotary start, rotary dim, interleaved
    ("bf16", 8, 128, 64, 64, [700, 0, 65, 1], 0.4, 0, 128, False),
    ("bf16", 2, 64, 16, 32, [33, 16, 200], 1.0, 0, 32, True),
    ("bf16", 1, 64, 128, 16, [300], 0.5, 0, 18, False),
    ("bf16", 3, 128, 32, 32, [90, 31], 0.7, 24, 96, True),
    ("bf16", 5, 128, 32, 64, [90, 31], 0.7, 0, 0, False),
    ("e4m3", 2, 64, 32, 32, [300, 0, 77, 1], 0.5, 0, 64, False),
    ("e4m3", 8, 128, 64, 64, [500, 129], 0.3, 0, 128, False),
    ("e4m3", 1, 128, 128, 16, [260], 0.9, 0, 34, True),
    ("e4m3", 2, 64, 16, 128, [100, 50], 1.0, 0, 0, False),
    ("e4m3", 2, 64, 16, 128, [100, 50], 0.5, 32, 32, True),
    ("latent", 1, 576, 64, 32, [200, 63], 0.5, 512, 64, True),
    ("latent", 1, 160, 16, 16, [40], 0.6, 128, 32, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}x{c[2]}-p{c[3]}to{c[4]}-rd{c[8]}")
def test_compact(case):
    import causal_gqa_attention_rope_gb300 as na
    fmt, KV, d, page, new_page, lens, part, start, rd, inter = case
    r = random.Random(str(case))
    rope = na.RopeConfig(base=1e4, yarn=rd == 96, factor=4.0, orig_max_pos=64)
    old = make_paged(lens, KV, d, page, "e4m3" if fmt == "e4m3" else "bf16", 11)
    keep = keeps(r, lens, part)
    new_lens = [len(k) for k in keep]
    new = make_paged([0] * len(lens), KV, d, new_page, "e4m3" if fmt == "e4m3" else "bf16", 12, room=max(new_lens))
    if fmt == "latent":
        a = na.PagedLatentCache(old.k[:, 0].to(DEV), old.table.to(DEV))
        z = na.PagedLatentCache(new.k[:, 0].to(DEV), new.table.to(DEV))
    else:
        a, z = old.to(DEV), new.to(DEV)
    top = max(new_lens)
    table = torch.zeros(len(lens), top, dtype=torch.int32)
    for b, k in enumerate(keep):
        table[b, :len(k)] = torch.tensor(k, dtype=torch.int32)
    whole = part == 1.0 and keep == [list(range(n)) for n in lens]
    status = ints([0])
    na.na_pages_compact(a, z, ints(new_lens), top, keep=None if whole else table.to(DEV),
                        rope=rope if rd else None, rotary_start=start, rotary_dim=rd, interleaved=inter,
                        status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    pools = [(old.k, old.k_scale, new.k, new.k_scale, z.kv[:, None] if fmt == "latent" else z.k,
              None if fmt == "latent" else z.k_scale, True)]
    if fmt != "latent":
        pools.append((old.v, old.v_scale, new.v, new.v_scale, z.v, z.v_scale, False))
    for pool, scale, was, was_scale, got, got_scale, is_k in pools:
        got, expect = got.cpu(), bits(was).clone()
        got_scale = None if got_scale is None else got_scale.cpu()
        written = torch.zeros(was.shape[:3], dtype=torch.bool)
        for b, kept in enumerate(keep):
            for lo in range(0, len(kept), new_page):
                at = torch.tensor(kept[lo:lo + new_page])
                pid, m = int(new.table[b, lo // new_page]), len(at)
                sid = old.table[b, at // page].long()
                x = pool.view(torch.uint8 if scale is not None else torch.bfloat16)[sid, :, at % page]
                raw = x
                x = x.view(pool.dtype).double()
                if scale is not None:
                    x = x * torch.exp2(scale[sid].double() - 127)[..., None]
                shift = torch.arange(lo, lo + m) - at
                if rd and is_k:
                    x = turned(x, shift[:, None], rope, start, rd, inter)
                rows = got[pid, :, :m].permute(1, 0, 2)
                written[pid, :, :m] = True
                if scale is None:
                    if rd and is_k:
                        # half a step of bf16, and 2^-22 of the pair (fp32 within 2^-23)
                        tol = 2.0 ** -8 * x.abs() + 2.0 ** -22 * x.abs().amax()
                        assert ((rows.double() - x).abs() <= tol).all()
                        still = shift == 0
                        assert torch.equal(bits(rows[still]), bits(raw[still]))
                        other = [e for e in range(d) if not start <= e < start + rd]
                        assert torch.equal(bits(rows[..., other]), bits(raw[..., other]))
                    else:
                        assert torch.equal(bits(rows), bits(raw))
                    continue
                amax = x.abs().amax(dim=(0, 2))
                e = got_scale[pid].double() - 127
                near = 2.0 ** -20  # of fp32's largest in the page
                assert (amax * (1 - near) <= 448 * torch.exp2(e)).all()
                assert (amax * (1 + near) > 448 * torch.exp2(e - 1)).all()
                y = rows.view(torch.uint8).view(rows.dtype).double() * torch.exp2(e)[:, None]
                # half a step of E4M3: 2^-4 of the value, 2^-10 of the scale below its normal range
                tol = 2.0 ** -4 * x.abs() + torch.exp2(e - 10)[:, None] + near * amax[:, None]
                assert ((y - x).abs() <= tol).all()
        # every other slot as it was
        assert torch.equal(bits(got)[~written], expect[~written])


def test_compact_reports():
    import causal_gqa_attention_rope_gb300 as na
    old, new = make_paged([40, 40], 2, 64, 16, "bf16", 1), make_paged([0, 0], 2, 64, 16, "bf16", 2, room=20)
    keep = ints([[0, 47, 48, 5], [-1, 1, 2, 3]])  # positions are those of the table: 0 .. 47

    def status_of(**kw):
        z, status = new.to(DEV), ints([0])
        args = dict(cache=old.to(DEV), keep=keep, keep_lens=ints([2, 0]), max_keep=4)
        args.update(kw)
        na.na_pages_compact(args.pop("cache"), z, args.pop("keep_lens"), args.pop("max_keep"), status=status,
                            **args)
        torch.cuda.synchronize()
        return int(status.item()), z

    assert status_of()[0] == 0
    assert status_of(keep_lens=ints([3, 0]))[0] == na.NA_ERR_CAPACITY   # past the table
    assert status_of(keep_lens=ints([0, 1]))[0] == na.NA_ERR_CAPACITY   # negative position
    code, z = status_of(keep_lens=ints([5, 0]))                         # longer than max_keep
    assert code == na.NA_ERR_CAPACITY and torch.equal(bits(z.k.cpu()), bits(new.k))
    assert status_of(keep_lens=ints([-3, 0]))[0] == 0
    bad = old.to(DEV)
    bad.page_table = bad.page_table.clone()
    bad.page_table[0, 0] = 1000
    assert status_of(cache=bad)[0] == na.NA_ERR_PAGE


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_a_step_on_a_side_stream_and_in_a_graph(fmt):
    """Fork, copy, compaction: on a side stream, then captured and replayed."""
    import causal_gqa_attention_rope_gb300 as na
    r = random.Random(3)
    lens = [70, 40, 100]
    old = make_paged(lens, 2, 64, 32, fmt, 5, spare=30, room=16)
    pages = old.k.shape[0]
    ref = [0] * pages
    for row in old.table.tolist():
        for e in row:
            if e >= 0:
                ref[e] = 1
    parents, grow = [2, 0, 0], [5, 40, 1]
    want = fork(parents, grow, lens, old.table.tolist(), 32, ref)
    assert not want[5]
    keep = keeps(r, want[2], 0.5)  # (of the new sequences: the old rows' pages may be others' by then)
    top = max(map(len, keep))
    table = ints([k + [0] * (top - len(k)) for k in keep])
    kl, dev = ints([len(k) for k in keep]), old.to(DEV)
    free = [i for i, c in enumerate(want[1]) if c == 0]
    to = ints([free[4 * b:4 * b + 4] for b in range(3)])
    args = [ints(x) for x in (parents, lens, old.table.tolist(), ref)]
    out = [torch.zeros(s, dtype=torch.int32, device=DEV) for s in (old.table.shape, (pages,), (3,), (3,), (3,))]
    status, g = ints([0]), ints(grow)
    rope = na.RopeConfig()

    def step():
        na.na_pages_fork(*args, 32, *out, grow=g, status=status)
        na.na_pages_copy(dev, out[3], out[4], status=status)
        here = na.PagedKVCache(dev.k, dev.v, out[0], dev.k_scale, dev.v_scale)
        na.na_pages_compact(here, na.PagedKVCache(dev.k, dev.v, to, dev.k_scale, dev.v_scale), kl, top,
                            keep=table, rope=rope, status=status)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    first = [t.clone() for t in out] + [bits(dev.k).clone(), bits(dev.v).clone()]
    assert [t.tolist() for t in out] == list(want[:5])
    moved = [t.to(DEV) for t in (old.k, old.v)]
    dev.k.view(torch.uint8).copy_(moved[0].view(torch.uint8))
    dev.v.view(torch.uint8).copy_(moved[1].view(torch.uint8))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in out:
        t.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for a, b in zip(first, out + [bits(dev.k), bits(dev.v)]):
        assert torch.equal(a, b)
