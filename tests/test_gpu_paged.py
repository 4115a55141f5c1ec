"""The paged cache on the GPU: the append into bf16 and E4M3 pages and the two
attention calls over them, against 64-bit statements (paged_ref.py)."""
import itertools

import pytest
import torch

import causal_gqa_attention_rope_gb300 as na
from harness import Guarded
from paged_ref import (Paged, attend, bits, exponent, make_paged, normed_rotated, v_normed,
                       values)

pytestmark = pytest.mark.gpu
DEV = "cuda"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def rnd(g, *shape, mag=1.0):
    return (torch.randn(*shape, generator=g) * mag).to(torch.bfloat16)


def cu_of(new):
    return ints([0] + list(itertools.accumulate(new)))


def check(got, ref, tol, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), f"{what}: non-finite values"
    off = (got - ref).abs()
    bad = off > tol
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} values off by more than the "
                           f"roundings allow; worst {float((off / tol.clamp(min=1e-300)).max()):.2f}x")


# ----------------------------------------------------------------- append --

APPEND = [
    # d, rd, page, KV, H, flags, (prior, new) per sequence
    (128, 128, 64, 8, 32, {}, [(0, 1), (63, 1), (64, 1), (65, 2)]),
    (128, 64, 16, 4, 20, dict(yarn=True), [(5, 40), (0, 0), (16, 16), (31, 1), (0, 17)]),
    (64, 64, 32, 2, 4, dict(qk_norm=True), [(10, 60), (100, 1), (0, 33)]),
    (128, 34, 128, 1, 3, dict(qk_norm=True, zero=True, v_norm=True), [(120, 20), (0, 260)]),
    (64, 18, 16, 3, 3, dict(v_norm=True), [(0, 15), (15, 2), (16, 1)]),
    (64, 0, 64, 2, 2, {}, [(7, 64), (0, 1)]),
    (64, 48, 128, 2, 16, {}, [(0, 128), (127, 130)]),
    (128, 128, 32, 2, 2, {}, [(i % 70, 1 + i % 3) for i in range(75)]),
]


def append_case(case, seed, fmt, mag=1.0):
    d, rd, page, KV, H, flags, seqs = case
    prior, new = [p for p, _ in seqs], [n for _, n in seqs]
    cache = make_paged(prior, KV, d, page, fmt, seed, room=max(new), mag=mag)
    g = torch.Generator().manual_seed(seed + 1)
    T = sum(new)
    q, k, v = rnd(g, T, H, d), rnd(g, T, KV, d, mag=mag), rnd(g, T, KV, d, mag=mag)
    qw = kw = None
    if flags.get("qk_norm"):
        qw, kw = rnd(g, d) * 0.1 + 1, rnd(g, d) * 0.1 + 1
    cfg = na.AttnConfig(H, KV, d, rotary_dim=rd, qk_norm=bool(flags.get("qk_norm")),
                        qk_norm_zero_centered=bool(flags.get("zero")),
                        v_norm=bool(flags.get("v_norm")))
    rope = na.RopeConfig(base=1e6, yarn=bool(flags.get("yarn")), factor=4.0, orig_max_pos=8192)
    return cfg, rope, prior, new, cache, q, k, v, qw, kw


def run_append(cfg, rope, prior, new, cache, q, k, v, qw, kw):
    mv = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    dc = cache.to(DEV)
    gq = Guarded(q.shape, q.dtype, DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    na.na_rope_append_kv_paged(cfg, rope, cu_of(new), ints(prior), mv(q), mv(k), mv(v), gq.t, dc,
                               q_norm_w=mv(qw), k_norm_w=mv(kw), status=status)
    torch.cuda.synchronize()
    gq.check("q_out")
    return gq.t.cpu(), Paged.back(dc), int(status.item())


def places(prior, new):
    """(sequence, position, token row) of every new token."""
    t = 0
    for b, (p, n) in enumerate(zip(prior, new)):
        for i in range(n):
            yield b, p + i, t
            t += 1


@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"d{c[0]}rd{c[1]}p{c[2]}")
def test_append_bf16_pages_equal_the_contiguous_append(case):
    cfg, rope, prior, new, cache, q, k, v, qw, kw = append_case(case, 11, "bf16")
    q_out, after, status = run_append(cfg, rope, prior, new, cache, q, k, v, qw, kw)
    assert status == 0
    cap = max(p + n for p, n in zip(prior, new))
    flat = na.KVCache(torch.zeros(len(prior), cfg.num_kv_heads, cap, cfg.head_dim,
                                  dtype=torch.bfloat16, device=DEV),
                      torch.zeros(len(prior), cfg.num_kv_heads, cap, cfg.head_dim,
                                  dtype=torch.bfloat16, device=DEV))
    mv = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    q_ref = torch.empty_like(q, device=DEV)
    na.na_rope_append_kv(cfg, rope, cu_of(new), ints(prior), mv(q), mv(k), mv(v), q_ref, flat,
                         q_norm_w=mv(qw), k_norm_w=mv(kw))
    assert torch.equal(bits(q_out), bits(q_ref.cpu()))
    for pool, was, ref in ((after.k, cache.k, flat.k.cpu()), (after.v, cache.v, flat.v.cpu())):
        want = was.clone()
        for b, pos, _ in places(prior, new):
            want[int(cache.table[b, pos // cache.page]), :, pos % cache.page] = ref[b, :, pos]
        assert torch.equal(bits(pool), bits(want))  # and nothing else was written


def e4m3_step(y):
    """Spacing of E4M3 at y (values of a page divided by its scale)."""
    return torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)


@pytest.mark.parametrize("mag", [1.0, 2.0 ** 20, 2.0 ** -30])
@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"d{c[0]}rd{c[1]}p{c[2]}")
def test_append_e4m3_pages(case, mag):
    """Scales exactly by the rule; new values within half a step of E4M3 (and the
    2^-20 of the page's largest that the fp32 arithmetic may be off); earlier
    values of a page whose scale grew rounded to it; everything else untouched."""
    cfg, rope, prior, new, cache, q, k, v, qw, kw = append_case(case, 12, "e4m3", mag)
    q_out, after, status = run_append(cfg, rope, prior, new, cache, q, k, v, qw, kw)
    assert status == 0
    page = cache.page
    spots = list(places(prior, new))
    pos = torch.tensor([p for _, p, _ in spots])
    # eps of the norms is 1e-6 as in the config
    rq = normed_rotated(q, pos, rope, cfg.rotary_dim, qw, 1e-6, cfg.qk_norm_zero_centered)
    check(q_out, rq, 2.0 ** -8 * rq.abs() * (1 + 2.0 ** -10) + 2.0 ** -20, "q_out")
    rk = normed_rotated(k, pos, rope, cfg.rotary_dim, kw, 1e-6, cfg.qk_norm_zero_centered)
    rv = v_normed(v, 1e-6) if cfg.v_norm else v.double()
    for name, x, pool, was, scale, scale_was in (
            ("k", rk, after.k, cache.k, after.k_scale, cache.k_scale),
            ("v", rv, after.v, cache.v, after.v_scale, cache.v_scale)):
        want_bits, want_scale = bits(was).clone(), scale_was.clone()
        by_page = {}
        for b, p, t in spots:
            by_page.setdefault((b, p // page), []).append((p % page, t))
        for (b, i), rows in by_page.items():
            pid = int(cache.table[b, i])
            y = x[[t for _, t in rows]]  # [tokens, KV, d]
            e = exponent(y.abs().amax(dim=(0, 2)))
            held = rows[0][0]
            if held:
                e_old = scale_was[pid].double() - 127
                e = torch.maximum(e, e_old)
                old = (was[pid, :, :held].double() * torch.exp2(e_old - e)[:, None, None])
                want_bits[pid, :, :held] = old.float().to(torch.float8_e4m3fn).view(torch.uint8)
            want_scale[pid] = (e + 127).to(torch.uint8)
            unit = torch.exp2(e)[None, :, None]
            got = pool[pid].double()[:, [s for s, _ in rows]].transpose(0, 1) * unit
            tol = (0.5 * e4m3_step(y / unit) + 448 * 2.0 ** -20) * unit
            check(got, y, tol, f"{name} page {pid}")
            for s, _ in rows:
                want_bits[pid, :, s] = bits(pool)[pid, :, s]  # compared above
        assert torch.equal(scale, want_scale), name
        # minus zero and zero are the same value of a rescaled token
        same = (bits(pool) == want_bits) | ((bits(pool) & 0x7F == 0) & (want_bits & 0x7F == 0))
        assert same.all(), f"{name}: {int((~same).sum())} other bytes changed"


def test_append_e4m3_token_by_token_is_the_chunk():
    """A page filled one token at a time ends with the chunk's scale, and with its
    values but for those that an intermediate scale pushed below E4M3's normal
    range or rounded there twice: at most one step of the final scale's
    subnormals apart."""
    case = (128, 128, 32, 2, 4, {}, [(0, 50), (3, 40)])
    cfg, rope, prior, new, cache, q, k, v, qw, kw = append_case(case, 13, "e4m3")
    k[5::7] *= 8  # scales grow along the way
    _, whole, _ = run_append(cfg, rope, prior, new, cache, q, k, v, qw, kw)
    dc = cache.to(DEV)
    starts = [0, new[0]]
    for i in range(max(new)):
        live = [b for b in range(2) if i < new[b]]
        rows = torch.tensor([starts[b] + i for b in live])
        n = [1 if i < new[b] else 0 for b in range(2)]
        at = [prior[b] + min(i, new[b]) for b in range(2)]
        q_out = torch.empty(len(live), 4, 128, dtype=torch.bfloat16, device=DEV)
        na.na_rope_append_kv_paged(cfg, rope, cu_of(n), ints(at), q[rows].to(DEV), k[rows].to(DEV),
                                   v[rows].to(DEV), q_out, dc)
    steps = Paged.back(dc)
    assert torch.equal(steps.k_scale, whole.k_scale) and torch.equal(steps.v_scale, whole.v_scale)
    for a, b in ((steps.k, whole.k), (steps.v, whole.v)):
        a, b = a.double(), b.double()
        both = torch.isfinite(a)
        assert torch.equal(both, torch.isfinite(b))
        a, b = a[both], b[both]
        normal = b.abs() >= 2.0 ** -6
        assert torch.equal(a[normal], b[normal])
        assert ((a - b)[~normal].abs() <= 2.0 ** -9).all()


# ----------------------------------------------------------------- decode --

# calls with enough rows for four per thread, and next to it
MANY = [
    (128, 128, 16, 4, 32, dict(qk_norm=True), [(0, 700), (3, 517), (40, 231)]),
    (128, 64, 64, 8, 16, {}, [(100, 2500)]),
    (64, 64, 32, 2, 64, {}, [(31, 1301), (0, 64), (5, 1)]),
    (64, 32, 128, 8, 48, dict(qk_norm=True, zero=True, v_norm=True), [(7, 1500)]),
    (128, 128, 128, 1, 40, {}, [(127, 1300)]),
]


# rotary dimensions that are no multiple of 16, with and without norms, few rows and many
ODD = [
    (128, 34, 64, 8, 40, {}, [(100, 700), (0, 1), (63, 2)]),
    (128, 34, 16, 2, 8, dict(yarn=True), [(5, 40), (0, 0), (16, 16), (31, 1), (0, 17)]),
    (64, 18, 32, 2, 6, {}, [(10, 60), (100, 1), (0, 33)]),
    (64, 18, 128, 2, 16, dict(qk_norm=True), [(0, 128), (127, 900)]),
    (128, 2, 128, 1, 3, dict(qk_norm=True, zero=True), [(120, 20), (0, 260)]),
    (128, 126, 16, 1, 5, dict(v_norm=True), [(3, 50), (0, 7)]),
    (64, 62, 64, 3, 3, {}, [(i % 70, 1 + i % 3) for i in range(75)]),
]


# two tokens per sequence or fewer on the average, one sequence with many
FEW = [
    (128, 64, 64, 2, 4, dict(qk_norm=True), [(10, 70)] + [(i, 0) for i in range(40)]),
    (64, 64, 128, 3, 3, dict(v_norm=True), [(100, 60)] + [(5, 0)] * 30 + [(127, 2)]),
    (128, 128, 16, 1, 2, dict(qk_norm=True, zero=True), [(3, 30), (0, 0), (15, 2)] + [(7, 1)] * 60),
    (64, 32, 32, 8, 8, {}, [(i, 1) for i in range(64)]),
]


@pytest.mark.parametrize("mag", [1.0, 2.0 ** 20])
@pytest.mark.parametrize("case", FEW, ids=lambda c: f"d{c[0]}rd{c[1]}p{c[2]}")
def test_append_few_tokens(case, mag):
    test_append_e4m3_pages(case, mag)


@pytest.mark.parametrize("mag", [1.0, 2.0 ** -30])
@pytest.mark.parametrize("case", ODD, ids=lambda c: f"d{c[0]}rd{c[1]}p{c[2]}")
def test_append_odd_rotary_dimensions(case, mag):
    test_append_bf16_pages_equal_the_contiguous_append(case)
    test_append_e4m3_pages(case, mag)


@pytest.mark.parametrize("case", MANY, ids=lambda c: f"d{c[0]}rd{c[1]}p{c[2]}")
def test_append_many_rows(case):
    test_append_bf16_pages_equal_the_contiguous_append(case)
    test_append_e4m3_pages(case, 1.0)



DECODE = [
    # fmt, d, page, KV, G, lens, options
    ("e4m3", 128, 64, 8, 4, [1, 64, 65, 700], dict(probs=True)),
    ("e4m3", 64, 16, 2, 2, [0, 15, 16, 17, 333], dict(probs=True)),
    ("e4m3", 128, 128, 1, 8, [129, 5000], dict(gate=True, splits=3)),
    ("e4m3", 128, 16, 4, 5, [40, 1, 2049], dict(softcap=20.0, probs=True)),
    ("e4m3", 64, 32, 3, 3, [200, 31, 1000], dict(window=100, probs=True)),
    ("e4m3", 128, 32, 2, 16, [513, 3, 64], dict(window=7, gate=True)),
    ("e4m3", 64, 128, 1, 7, [127, 128, 1300], dict(probs=True)),
    ("bf16", 128, 64, 8, 4, [1, 64, 65, 700], dict(probs=True)),
    ("bf16", 64, 16, 2, 2, [0, 15, 16, 17, 333], dict(probs=True, gate=True)),
    ("bf16", 128, 16, 1, 12, [3000, 63], dict(window=1000, probs=True)),
    ("bf16", 64, 128, 4, 1, [127, 1, 900], dict(softcap=5.0)),
    ("bf16", 128, 32, 2, 6, [100, 31], dict(splits=2)),
    # short sequences: one CTA per stream
    ("e4m3", 128, 16, 2, 16, [300, 1, 0, 512], dict(window=40, probs=True)),
    ("e4m3", 128, 64, 2, 3, [500, 64, 63], dict(softcap=9.0, gate=True, probs=True)),
    ("bf16", 64, 32, 1, 5, [0, 400, 33], dict(window=64, probs=True, gate=True)),
    ("bf16", 128, 128, 2, 8, [512, 129], dict(softcap=9.0, probs=True)),
    ("bf16", 128, 128, 2, 8, [513, 129], dict(probs=True)),
    ("e4m3", 64, 16, 2, 4, [0, 0], {}),
    ("bf16", 64, 16, 1, 2, [i % 40 for i in range(700)], {}),
    ("e4m3", 64, 16, 1, 2, [(i * 37) % 600 for i in range(300)], {}),
]


def run_decode(cfg, q, cache, lens, gate=None, probs=False, splits=0):
    B, H, d = q.shape
    top = max(lens)
    go = Guarded(q.shape, q.dtype, DEV)
    gp = Guarded((B, H, max(top, 1)), torch.float32, DEV, fill=-7.0) if probs else None
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = na.workspace(na.na_decode_paged_workspace_size(cfg, B, top, splits), DEV)
    na.na_attn_decode_paged(cfg, q.to(DEV), cache, ints(lens), top, go.t,
                            probs=None if gp is None else gp.t,
                            gate=None if gate is None else gate.to(DEV), workspace=ws,
                            num_splits=splits, status=status)
    torch.cuda.synchronize()
    go.check("out")
    if gp is not None:
        gp.check("probs")
    return go.t.cpu(), None if gp is None else gp.t.cpu(), int(status.item())


@pytest.mark.parametrize("case", DECODE, ids=lambda c: f"{c[0]}d{c[1]}p{c[2]}g{c[4]}")
def test_decode(case):
    fmt, d, page, KV, G, lens, opt = case
    H = KV * G
    cache = make_paged(lens, KV, d, page, fmt, 21)
    window = opt.get("window", 0)
    if window:  # pages before every window are given away
        for b, n in enumerate(lens):
            cache.table[b, :max(0, n - window) // page] = -1
    g = torch.Generator().manual_seed(22)
    q = rnd(g, len(lens), H, d)
    gate = rnd(g, len(lens), H, d) if opt.get("gate") else None
    cfg = na.AttnConfig(H, KV, d, out_gate=gate is not None, softcap=opt.get("softcap", 0.0),
                        window=window)
    out, probs, status = run_decode(cfg, q, cache.to(DEV), lens, gate, opt.get("probs", False),
                                    opt.get("splits", 0))
    assert status == 0
    ref = attend(cache, q, [(b, n - 1, 1) if n else (b, 0, 0) for b, n in enumerate(lens)],
                 softcap=cfg.softcap, window=window, gate=gate)
    check(out, ref.out, ref.tol, "out")
    if probs is not None:
        for b, n in enumerate(lens):
            if n:
                check(probs[b, :, :n], ref.probs[b], ref.probs_tol[b], f"probs {b}")
            assert (probs[b, :, n:] == -7.0).all()


@pytest.mark.parametrize("case", [c for c in DECODE if "splits" not in c[6] and len(c[5]) < 10],
                         ids=lambda c: f"{c[0]}d{c[1]}p{c[2]}g{c[4]}")
def test_decode_cut_over_the_grid(case):
    """The calls that take one CTA or one cluster per stream, through the merge pass instead."""
    test_decode(case[:6] + (dict(case[6], splits=4),))


# streams of a few CTAs each: the first, the last or every CTA but one without keys, windows
# that start inside a CTA's share, and the lengths at which the number of CTAs changes
CLUSTERS = [
    ("bf16", 128, 64, 1, 4, [257, 0, 1, 64, 65], dict(probs=True)),
    ("e4m3", 128, 64, 1, 4, [257, 0, 1, 64, 65], dict(probs=True, gate=True)),
    ("bf16", 64, 16, 2, 8, [1024, 449, 448, 1023], dict(probs=True)),
    ("e4m3", 64, 16, 2, 8, [1025, 449, 448, 129], dict(probs=True)),
    ("bf16", 128, 128, 2, 3, [2048, 1, 0, 1500, 77], dict(window=130, probs=True, gate=True)),
    ("e4m3", 128, 128, 2, 3, [2048, 1, 0, 1500, 77], dict(window=130, probs=True)),
    ("bf16", 64, 32, 3, 1, [900, 65], dict(window=1, probs=True)),
    ("e4m3", 64, 32, 3, 1, [900, 65], dict(window=1, softcap=3.0, probs=True)),
    ("e4m3", 128, 16, 8, 2, [4096, 3999, 7], dict(softcap=30.0)),
    ("bf16", 128, 64, 4, 2, [4096, 4095], dict(probs=True)),
    ("bf16", 64, 64, 8, 1, [600] * 8, dict(probs=True)),
    ("e4m3", 64, 64, 16, 1, [600 - 31 * i for i in range(16)], {}),
    ("e4m3", 128, 64, 1, 40, [2000, 511], dict(probs=True)),
]


@pytest.mark.parametrize("case", CLUSTERS, ids=lambda c: f"{c[0]}d{c[1]}p{c[2]}g{c[4]}n{max(c[5])}")
def test_decode_clusters(case):
    test_decode(case)


@pytest.mark.parametrize("mag", [2.0 ** 30, 2.0 ** -40])
def test_decode_e4m3_scales_far_from_one(mag):
    """V of any magnitude, and page scales that differ by 2^10 within a sequence."""
    lens, KV, d, page = [300, 70], 2, 128, 32
    ks = make_paged(lens, KV, d, page, "e4m3", 23)
    vs = make_paged(lens, KV, d, page, "e4m3", 23, mag=mag, spread=5.0)  # one seed: the same table
    cache = Paged(ks.k, vs.v, ks.table, ks.k_scale, vs.v_scale)
    g = torch.Generator().manual_seed(25)
    q = rnd(g, 2, 8, d)
    out, _, status = run_decode(na.AttnConfig(8, KV, d), q, cache.to(DEV), lens)
    assert status == 0
    ref = attend(cache, q, [(b, n - 1, 1) for b, n in enumerate(lens)])
    check(out, ref.out, ref.tol, "out")


def test_decode_shared_pages():
    """Two sequences that share their first pages (a common prompt)."""
    cache = make_paged([200, 150], 2, 64, 32, "e4m3", 26)
    cache.table[1, :4] = cache.table[0, :4]
    g = torch.Generator().manual_seed(27)
    q = rnd(g, 2, 4, 64)
    out, _, status = run_decode(na.AttnConfig(4, 2, 64), q, cache.to(DEV), [200, 150])
    assert status == 0
    ref = attend(cache, q, [(0, 199, 1), (1, 149, 1)])
    check(out, ref.out, ref.tol, "out")


# ---------------------------------------------------------------- prefill --

PREFILL = [
    # fmt, d, page, KV, G, (prior, new), options
    ("bf16", 128, 64, 2, 4, [(0, 128)], {}),
    ("bf16", 128, 16, 2, 4, [(100, 37), (0, 1), (500, 3), (0, 0), (17, 129)], dict(gate=True)),
    ("bf16", 64, 128, 1, 8, [(1000, 5), (3, 130)], dict(softcap=10.0)),
    ("bf16", 64, 32, 2, 3, [(700, 40), (0, 33)], dict(window=50)),
    ("bf16", 128, 32, 1, 1, [(4000, 64)], {}),
    ("e4m3", 128, 64, 2, 4, [(0, 128)], {}),
    ("e4m3", 128, 16, 2, 4, [(100, 37), (0, 1), (500, 3), (0, 0), (17, 129)], dict(gate=True)),
    ("e4m3", 64, 128, 1, 8, [(1000, 5), (3, 130)], dict(softcap=10.0)),
    ("e4m3", 64, 32, 2, 3, [(700, 40), (0, 33)], dict(window=50)),
    ("e4m3", 128, 32, 1, 1, [(4000, 64)], {}),
    ("e4m3", 128, 128, 1, 2, [(250, 300)], dict(window=260)),
    ("e4m3", 64, 16, 1, 1, [(5000, 2)], {}),
    # several waves of units, more tiles each than any ring holds
    ("e4m3", 128, 16, 4, 4, [(1400 + 17 * i, 1 + i % 5) for i in range(60)], {}),
    ("bf16", 128, 32, 4, 4, [(1400 + 17 * i, 1 + i % 5) for i in range(60)], {}),
    ("e4m3", 64, 64, 4, 2, [(2000 - 11 * i, 1 + i % 3) for i in range(45)], dict(gate=True)),
    # groups that are no power of two; few rows (laid over the tile four times) and many
    ("e4m3", 128, 32, 2, 5, [(900, 6), (40, 1), (0, 3), (0, 0), (127, 2)], dict(gate=True)),
    ("e4m3", 128, 32, 2, 5, [(900, 60), (40, 7), (0, 26), (3, 25)], {}),
    ("bf16", 64, 16, 2, 3, [(300, 10), (5000, 1), (0, 9)], dict(window=70)),
    ("bf16", 128, 64, 1, 6, [(300, 50), (0, 129)], dict(softcap=8.0)),
    ("e4m3", 64, 16, 1, 12, [(700, 2), (31, 1)], dict(softcap=8.0, window=500)),
    ("e4m3", 64, 64, 3, 1, [(60, 32), (1000, 31)], dict(window=33)),
    ("bf16", 128, 16, 1, 32, [(100, 1), (2000, 1)], {}),
    ("e4m3", 64, 16, 1, 40, [(100, 3), (600, 4)], {}),
    ("e4m3", 64, 16, 1, 130, [(100, 3)], {}),
    # more sequences than are ranked
    ("e4m3", 64, 16, 1, 2, [(i % 50, i % 4) for i in range(270)], {}),
    ("bf16", 64, 16, 1, 2, [(200 - i % 50, i % 30) for i in range(100)], {}),
]


def run_prefill(cfg, q, cache, prior, new, gate=None):
    T = sum(new)
    top, most = max(p + n for p, n in zip(prior, new)), max(new)
    go = Guarded(q.shape, q.dtype, DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = na.workspace(na.na_prefill_paged_workspace_size(cfg, len(new), T, most, top), DEV)
    na.na_attn_prefill_chunk_paged(cfg, cu_of(new), ints(prior), most, top, q.to(DEV), cache, go.t,
                                   gate=None if gate is None else gate.to(DEV), workspace=ws,
                                   status=status)
    torch.cuda.synchronize()
    go.check("out")
    return go.t.cpu(), int(status.item())


def prefill_case(case, seed):
    fmt, d, page, KV, G, seqs, opt = case
    prior, new = [p for p, _ in seqs], [n for _, n in seqs]
    cache = make_paged([p + n for p, n in seqs], KV, d, page, fmt, seed)
    window = opt.get("window", 0)
    if window:
        for b, p in enumerate(prior):
            cache.table[b, :max(0, p - window + 1) // page] = -1
    g = torch.Generator().manual_seed(seed + 1)
    q = rnd(g, sum(new), KV * G, d)
    gate = rnd(g, sum(new), KV * G, d) if opt.get("gate") else None
    cfg = na.AttnConfig(KV * G, KV, d, out_gate=gate is not None, softcap=opt.get("softcap", 0.0),
                        window=window)
    starts = [0] + list(itertools.accumulate(new))
    return cfg, cache, q, gate, prior, new, [(starts[b], p, n) for b, (p, n) in enumerate(seqs)]


@pytest.mark.parametrize("case", PREFILL, ids=lambda c: f"{c[0]}d{c[1]}p{c[2]}g{c[4]}b{len(c[5])}")
def test_prefill(case):
    cfg, cache, q, gate, prior, new, spans = prefill_case(case, 31)
    out, status = run_prefill(cfg, q, cache.to(DEV), prior, new, gate)
    assert status == 0
    ref = attend(cache, q, spans, softcap=cfg.softcap, window=cfg.window, gate=gate)
    check(out, ref.out, ref.tol, "out")


@pytest.mark.parametrize("e", [-100, -45, -20, 8, 30, 50])
def test_prefill_e4m3_scales_far_from_one(e):
    """V's scale far from one on every page (K's stays at unit scale)."""
    case = ("e4m3", 128, 64, 1, 2, [(300, 40)], {})
    cfg, cache, q, gate, prior, new, spans = prefill_case(case, 35)
    live = cache.v_scale != 255
    cache.v_scale[live] = (cache.v_scale[live].int() + e).to(torch.uint8)
    out, status = run_prefill(cfg, q, cache.to(DEV), prior, new)
    assert status == 0
    ref = attend(cache, q, spans)
    check(out, ref.out, ref.tol, "out")


def test_v_scale_above_the_largest_is_reported():
    cache = make_paged([40], 1, 64, 16, "e4m3", 36)
    cache.v_scale[cache.v_scale != 255] = 127 + 48
    g = torch.Generator().manual_seed(37)
    cfg, q = na.AttnConfig(2, 1, 64), rnd(g, 1, 2, 64)
    assert run_decode(cfg, q, cache.to(DEV), [40])[2] == na.NA_ERR_UNSUPPORTED
    assert run_prefill(cfg, q, cache.to(DEV), [39], [1])[1] == na.NA_ERR_UNSUPPORTED


@pytest.mark.parametrize("d,page", [(128, 64), (64, 16)])
@pytest.mark.parametrize("e", [-73, -66, -65, -64, -63, -56, -55, -54, -49])
@pytest.mark.parametrize("call", ["decode", "prefill"])
def test_v_scales_around_the_last_multiple(call, e, d, page):
    """Scales 2^e of V where E4M3 values reach the multiples of 2^-64 that they are rounded
    to (the largest value is 2^(e + 8.8)): page scales of one sequence lie around e."""
    lens, KV = [300, 45], 2
    cache = make_paged(lens, KV, d, page, "e4m3", 33)
    live = cache.v_scale != 255
    mid = int(cache.v_scale[live].int().median())
    cache.v_scale[live] = (cache.v_scale[live].int() - mid + e + 127).to(torch.uint8)
    g = torch.Generator().manual_seed(34)
    cfg = na.AttnConfig(2 * KV, KV, d)
    q = rnd(g, 2, 2 * KV, d)
    if call == "decode":
        out, _, status = run_decode(cfg, q, cache.to(DEV), lens)
    else:
        out, status = run_prefill(cfg, q, cache.to(DEV), [n - 1 for n in lens], [1, 1])
    assert status == 0
    ref = attend(cache, q, [(0, 299, 1), (1, 44, 1)])
    check(out, ref.out, ref.tol, "out")


@pytest.mark.parametrize("call", ["decode", "prefill"])
def test_pages_of_zeros(call):
    """Pages whose K or V is all zero have scale byte 0 (2^-127): they still weigh in
    the softmax, alone or beside other pages."""
    lens, KV, d, page = [100, 32, 200], 2, 64, 16
    cache = make_paged(lens, KV, d, page, "e4m3", 38)
    for b, pages in ((0, [1, 3]), (1, [0, 1]), (2, [12])):
        for i in pages:
            pid = int(cache.table[b, i])
            for pool, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
                pool.view(torch.uint8)[pid], scale[pid] = 0, 0
    g = torch.Generator().manual_seed(39)
    cfg, q = na.AttnConfig(4, KV, d), rnd(g, 3, 4, d)
    if call == "decode":
        out, _, status = run_decode(cfg, q, cache.to(DEV), lens)
    else:
        out, status = run_prefill(cfg, q, cache.to(DEV), [n - 1 for n in lens], [1] * 3)
    assert status == 0
    ref = attend(cache, q, [(b, n - 1, 1) for b, n in enumerate(lens)])
    check(out, ref.out, ref.tol, "out")


# --------------------------------------------------- together, graphs, ... --

@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_prompt_then_decode_with_importance(fmt):
    """Two prompts in chunks, then decode steps with probabilities and importance,
    each step's attention checked against the pages as they stand."""
    KV, G, d, page = 2, 4, 128, 16
    H, B = KV * G, 2
    cfg = na.AttnConfig(H, KV, d, qk_norm=True, window=0)
    rope = na.RopeConfig(base=1e6)
    g = torch.Generator().manual_seed(41)
    qw, kw = (rnd(g, d) * 0.1 + 1).to(DEV), (rnd(g, d) * 0.1 + 1).to(DEV)
    host = make_paged([0, 0], KV, d, page, fmt, 42, room=150)
    cache = host.to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    at = [0, 0]
    top = 150
    imp = torch.zeros(B, top, device=DEV)
    imp_ref = torch.zeros(B, top, dtype=torch.float64)
    dws = na.workspace(na.na_decode_paged_workspace_size(cfg, B, top), DEV)
    for new in ([40, 13], [70, 90], [1, 1], [1, 1], [1, 1]):
        T = sum(new)
        q, k, v = (rnd(g, T, n, d).to(DEV) for n in (H, KV, KV))
        q_rot, out = torch.empty_like(q), torch.empty_like(q)
        na.na_rope_append_kv_paged(cfg, rope, cu_of(new), ints(at), q, k, v, q_rot, cache,
                                   q_norm_w=qw, k_norm_w=kw, status=status)
        probs = None
        if max(new) > 1:
            ws = na.workspace(na.na_prefill_paged_workspace_size(cfg, B, T, max(new), top), DEV)
            na.na_attn_prefill_chunk_paged(cfg, cu_of(new), ints(at), max(new), top, q_rot, cache,
                                           out, workspace=ws, status=status)
        else:
            lens = ints([n + 1 for n in at])
            probs = torch.empty(B, H, top, device=DEV)
            na.na_attn_decode_paged(cfg, q_rot, cache, lens, top, out, probs=probs, workspace=dws,
                                    status=status)
            na.na_decode_importance(cfg, probs, lens, top, imp, accumulate=True, status=status)
        assert int(status.item()) == 0
        spans = [(0, at[0], new[0]), (new[0], at[1], new[1])]
        ref = attend(Paged.back(cache), q_rot.cpu(), spans)
        check(out, ref.out, ref.tol, f"step {new}")
        if probs is not None:
            for b in range(B):
                n = at[b] + 1
                check(probs[b, :, :n], ref.probs[b], ref.probs_tol[b], "probs")
                imp_ref[b, :n] += ref.probs[b].sum(0)
        at = [a + n for a, n in zip(at, new)]
    # three steps' sums over H heads, fp32
    check(imp, imp_ref, (imp_ref + 1) * 2.0 ** -14, "importance")


def test_graph_replay_with_new_lengths():
    """A decode step (append, attend) captured once and replayed while the
    sequences grow, on a side stream; then the same steps without the graph."""
    KV, G, d, page = 2, 4, 64, 16
    H, B, top = KV * G, 3, 100
    cfg, rope = na.AttnConfig(H, KV, d), na.RopeConfig()
    start = [0, 14, 63]
    host = make_paged(start, KV, d, page, "e4m3", 51, room=40)
    g = torch.Generator().manual_seed(52)
    steps = [[rnd(g, B, n, d) for n in (H, KV, KV)] for _ in range(6)]

    def run(graph):
        cache = host.to(DEV)
        q, k, v = (torch.zeros_like(t, device=DEV) for t in steps[0])
        q_rot, out = torch.empty_like(q), torch.empty_like(q)
        cu, prior, lens = cu_of([1] * B), ints(start), ints([n + 1 for n in start])
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        ws = na.workspace(na.na_decode_paged_workspace_size(cfg, B, top), DEV)

        def step():
            na.na_rope_append_kv_paged(cfg, rope, cu, prior, q, k, v, q_rot, cache, status=status)
            na.na_attn_decode_paged(cfg, q_rot, cache, lens, top, out, workspace=ws, status=status)

        s = torch.cuda.Stream()
        outs = []
        with torch.cuda.stream(s):
            gr = None
            for i, (a, b, c) in enumerate(steps):
                q.copy_(a), k.copy_(b), v.copy_(c)
                prior.copy_(ints([n + i for n in start]))
                lens.copy_(ints([n + i + 1 for n in start]))
                if not graph:
                    step()
                else:
                    if gr is None:
                        s.synchronize()
                        gr = torch.cuda.CUDAGraph()
                        with torch.cuda.graph(gr, stream=s):
                            step()
                    gr.replay()
                outs.append(out.clone())
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        return torch.stack(outs).cpu(), Paged.back(cache)

    (a, ca), (b, cb) = run(True), run(False)
    assert torch.equal(bits(a), bits(b))
    for x, y in ((ca.k, cb.k), (ca.v, cb.v), (ca.k_scale, cb.k_scale), (ca.v_scale, cb.v_scale)):
        assert torch.equal(bits(x), bits(y))


@pytest.mark.parametrize("fmt,rd", [("bf16", 64), ("e4m3", 64), ("bf16", 18), ("e4m3", 18)])
def test_padded_batch_leaves_the_rest_alone(fmt, rd):
    """total_tokens above cu_seqlens[batch]: rows of q_out and out behind the last
    sequence, and the pages, as without them."""
    case = (64, rd, 16, 2, 4, {}, [(20, 9), (3, 40)])
    cfg, rope, prior, new, cache, q, k, v, _, _ = append_case(case, 63, fmt)
    q_ref, after, _ = run_append(cfg, rope, prior, new, cache, q, k, v, None, None)
    pad = lambda t: torch.cat([t, torch.ones(15, *t.shape[1:], dtype=t.dtype)]).to(DEV)  # noqa: E731
    dc = cache.to(DEV)
    T = sum(new)
    q_out = torch.full((T + 15, 4, 64), -3.0, dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    na.na_rope_append_kv_paged(cfg, rope, cu_of(new), ints(prior), pad(q), pad(k), pad(v), q_out, dc,
                               status=status)
    out = torch.full_like(q_out, -5.0)
    ws = na.workspace(na.na_prefill_paged_workspace_size(cfg, 2, T + 15, 40, 43), DEV)
    na.na_attn_prefill_chunk_paged(cfg, cu_of(new), ints(prior), 40, 43, q_out, dc, out,
                                   workspace=ws, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(bits(q_out[:T].cpu()), bits(q_ref)) and (q_out[T:] == -3.0).all()
    assert (out[T:] == -5.0).all()
    got = Paged.back(dc)
    for a, b in ((got.k, after.k), (got.v, after.v)):
        assert torch.equal(bits(a), bits(b))
    ref = attend(after, q_ref, [(0, 20, 9), (9, 3, 40)])
    check(out[:T], ref.out, ref.tol, "out")


def test_append_many_sequences():
    """A 32-way search of three rounds: 1100 sequences of zero to two tokens."""
    seqs = [(i % 23, i % 3) for i in range(1100)]
    test_append_e4m3_pages((64, 64, 16, 1, 1, {}, seqs), 1.0)
    test_append_bf16_pages_equal_the_contiguous_append((64, 64, 16, 1, 1, {}, seqs))


def test_append_e4m3_zeros_first():
    """A page of zeros has scale byte 0, and takes the scale of what follows."""
    case = (64, 64, 16, 1, 1, {}, [(0, 4)])
    cfg, rope, prior, new, cache, q, k, v, _, _ = append_case(case, 64, "e4m3")
    cache.table = torch.zeros(1, 2, dtype=torch.int32)
    z = torch.zeros_like(k)
    _, after, _ = run_append(cfg, rope, [0], [4], cache, q, z, z, None, None)
    assert int(after.k_scale[0, 0]) == 0 and int(after.v_scale[0, 0]) == 0
    _, after, _ = run_append(cfg, rope, [4], [4], after, q, k, v, None, None)
    e = exponent(v.double().abs().amax())
    assert int(after.v_scale[0, 0]) == int(e) + 127
    assert (values(after.v, after.v_scale, torch.zeros(1))[0, :4] == 0).all()
    got = values(after.v, after.v_scale, torch.zeros(1))[0, 4:8]
    want = v[:, 0].double()
    check(got, want, 0.5 * e4m3_step(want / 2.0 ** e) * 2.0 ** e, "values")


def test_two_streams_at_once():
    """Two decodes on two streams, each with its own workspace, at the same time."""
    cases = []
    for seed, lens in ((81, [3000, 900, 40]), (82, [5000, 16])):
        cache = make_paged(lens, 2, 128, 64, "e4m3", seed)
        q = rnd(torch.Generator().manual_seed(seed), len(lens), 8, 128)
        cfg = na.AttnConfig(8, 2, 128)
        ref = attend(cache, q, [(b, n - 1, 1) for b, n in enumerate(lens)])
        cases.append((cfg, q.to(DEV), cache.to(DEV), ints(lens), max(lens),
                      torch.empty(len(lens), 8, 128, dtype=torch.bfloat16, device=DEV),
                      na.workspace(na.na_decode_paged_workspace_size(cfg, len(lens), max(lens)), DEV),
                      torch.cuda.Stream(), ref))
    torch.cuda.synchronize()
    for _ in range(20):
        for cfg, q, cache, lens, top, out, ws, st, _ in cases:
            na.na_attn_decode_paged(cfg, q, cache, lens, top, out, workspace=ws, stream=st)
    torch.cuda.synchronize()
    for *_, out, _, _, ref in cases:
        check(out, ref.out, ref.tol, "out")


def test_first_calls_inside_a_capture():
    """A layer's three calls captured without having run before (in a thread of
    their own), replayed: the chunk, then the decode, match the pages."""
    import threading
    KV, G, d, page = 1, 3, 64, 128
    cfg, rope = na.AttnConfig(KV * G, KV, d), na.RopeConfig()
    host = make_paged([0, 0], KV, d, page, "e4m3", 91, room=300)
    g = torch.Generator().manual_seed(92)
    q, k, v = (rnd(g, 300, n, d).to(DEV) for n in (KV * G, KV, KV))
    failed = []

    def work():
        try:
            cache = host.to(DEV)
            q_rot, out = torch.empty_like(q), torch.empty_like(q)
            cu, prior, lens = cu_of([200, 100]), ints([0, 0]), ints([200, 100])
            dec = torch.empty(2, KV * G, d, dtype=torch.bfloat16, device=DEV)
            status = torch.zeros(1, dtype=torch.int32, device=DEV)
            ws = na.workspace(na.na_prefill_paged_workspace_size(cfg, 2, 300, 200, 200), DEV)
            dws = na.workspace(na.na_decode_paged_workspace_size(cfg, 2, 1000), DEV)
            ends = torch.tensor([199, 299], device=DEV)
            torch.cuda.synchronize()
            s = torch.cuda.Stream()
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=s):
                na.na_rope_append_kv_paged(cfg, rope, cu, prior, q, k, v, q_rot, cache, status=status)
                na.na_attn_prefill_chunk_paged(cfg, cu, prior, 200, 200, q_rot, cache, out,
                                               workspace=ws, status=status)
                na.na_attn_decode_paged(cfg, q_rot.index_select(0, ends), cache, lens, 300, dec,
                                        workspace=dws, status=status)
            gr.replay()
            torch.cuda.synchronize()
            assert int(status.item()) == 0
            c = Paged.back(cache)
            ref = attend(c, q_rot.cpu(), [(0, 0, 200), (200, 0, 100)])
            check(out, ref.out, ref.tol, "chunk")
            check(dec, ref.out[[199, 299]], ref.tol[[199, 299]], "decode")
        except BaseException as e:  # noqa: BLE001 - reported by the test's thread
            failed.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    if failed:
        raise failed[0]


# ------------------------------------------------- reported by the device --

@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_capacity_reported_and_other_sequences_served(fmt):
    """An append past the table's pages, and lengths past the bound: reported, the
    tokens that fit and the other sequence as usual."""
    case = (64, 64, 16, 2, 4, {}, [(28, 4), (3, 2)])
    cfg, rope, prior, new, cache, q, k, v, qw, kw = append_case(case, 61, fmt)
    cache.table = cache.table[:, :2].contiguous()  # 32 positions a sequence
    _, good, status = run_append(cfg, rope, prior, new, cache, q, k, v, qw, kw)
    assert status == 0
    prior[0] = 30  # two of the four tokens are past the capacity
    _, after, status = run_append(cfg, rope, prior, new, cache, q, k, v, qw, kw)
    assert status == na.NA_ERR_CAPACITY
    pid = int(cache.table[1, 0])
    assert torch.equal(bits(after.k)[pid, :, 3:5], bits(good.k)[pid, :, 3:5])
    out, _, status = run_decode_bound(cfg, q[:2], good, [40, 5], 32)
    assert status == na.NA_ERR_CAPACITY
    assert (out[0] == 0).all()
    ref = attend(good, q[:2], [(0, 0, 0), (1, 4, 1)])
    check(out[1], ref.out[1], ref.tol[1], "the other sequence")


def run_decode_bound(cfg, q, cache, lens, bound):
    out = torch.zeros(q.shape, dtype=q.dtype, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = na.workspace(na.na_decode_paged_workspace_size(cfg, len(lens), bound), DEV)
    na.na_attn_decode_paged(cfg, q.to(DEV), cache.to(DEV), ints(lens), bound, out, workspace=ws,
                            status=status)
    torch.cuda.synchronize()
    return out.cpu(), None, int(status.item())


@pytest.mark.parametrize("bad", [-1, 1000, 2 ** 31 - 1])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_page_index_outside_the_cache(fmt, bad):
    """Reported as NA_ERR_PAGE by every call; the other sequence is served."""
    case = (64, 64, 16, 2, 4, {}, [(20, 30), (40, 3)])
    cfg, rope, prior, new, cache, q, k, v, qw, kw = append_case(case, 71, fmt)
    _, good, _ = run_append(cfg, rope, prior, new, cache, q, k, v, qw, kw)
    was = int(cache.table[0, 2])
    cache.table[0, 2] = bad  # positions 32 .. 47 of sequence 0
    _, after, status = run_append(cfg, rope, prior, new, cache, q, k, v, qw, kw)
    assert status == na.NA_ERR_PAGE
    assert torch.equal(bits(after.k)[was], bits(cache.k)[was])  # its page is as it was
    pid = int(cache.table[1, 2])
    assert torch.equal(bits(after.k)[pid], bits(good.k)[pid])
    good.table[0, 2] = bad
    out, _, status = run_decode(cfg, q[:2], good.to(DEV), [50, 43])
    assert status == na.NA_ERR_PAGE
    ref = attend(good, q[:2], [(0, 0, 0), (1, 42, 1)])
    check(out[1], ref.out[1], ref.tol[1], "decode of the other sequence")
    out, status = run_prefill(cfg, q, good.to(DEV), prior, new)
    assert status == na.NA_ERR_PAGE
    ref = attend(good, q, [(0, 0, 0), (30, 40, 3)])
    check(out[30:], ref.out[30:], ref.tol[30:], "prefill of the other sequence")
