"""Performance cases of a latent cache with the attention that reads it, and of a paged cache's pages.

Latent attention keeps one row for each token and layer, shared by all heads:
a latent vector c of R numbers, from which every head's keys and values come by
linear maps, and rd rotated dimensions that all heads' keys share.  A page is
[page, R + rd] in bf16; the page table is [batch, pages a sequence].

  latent_append  c = norm(kv[:R]) and RoPE(kv[R:]) go into their pages, and the
                 queries' rotated parts to where the attention reads them.
  absorbed       q [T, H, R + rd] (the map to the keys already in the queries)
                 against the pages: softmax(scale q . row) times the rows' first R
                 numbers.  Single tokens and chunks.
  expanded       q [T, H, dn + rd] against kv [keys, H, dn + dv], which the maps
                 made of the latents, and the shared rotated part k_pe [keys, rd].
  fork           one step of a batch's page tables: sequences go on as their
                 parents do, are dropped or begin; full pages are shared, a part-filled
                 one is copied for all children but the first, and pages that
                 nobody holds any more are free again.  Then the copies.
  compact        the kept tokens of each sequence move to the front of new pages;
                 keys are turned from their old positions to the new ones.

`run` computes them in plain torch, or, with `own`, through the library.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0


# ---------------------------------------------------------------- cases ----

def listed():
    return [
        # a decode step's new tokens: 64 sequences, one token each
        _latent("latent_append_step", op="latent_append", B=64, new=(1, 1), prior=(0, 1024), H=32,
                R=512, rd=64, page=64, interleaved=True),
        # one chunk of a long YaRN prompt, queries in the expanded layout
        _latent("latent_append_chunk", op="latent_append", B=1, new=(2048, 2048),
                prior=(2048, 2048), H=40, R=512, rd=64, page=64, yarn=True, base=1e6),
        # one short conversation of a small model: the latency of a call
        _latent("absorbed_one", op="absorbed", B=1, new=(1, 1), prior=(332, 332), H=4, R=128,
                rd=32, page=16),
        # a serving batch of mixed lengths, one token each
        _latent("absorbed_b64", op="absorbed", B=64, new=(1, 1), prior=(511, 8191), H=32, R=512,
                rd=64, page=64),
        # a few long contexts
        _latent("absorbed_long", op="absorbed", B=4, new=(1, 1), prior=(50000, 131071), H=16,
                R=512, rd=64, page=32),
        # drafted tokens of a speculative step, a few per sequence
        _latent("absorbed_verify", op="absorbed", B=64, new=(2, 8), prior=(512, 8184), H=32,
                R=512, rd=64, page=64),
        # a mixed step: prompts of many lengths over histories
        _latent("expanded_varlen", op="expanded", B=16, new=(1, 512), prior=(0, 1000), H=32, dn=128,
                rd=64, dv=128),
        # one chunk of a long prompt: bound by the matrix products
        _latent("expanded_long", op="expanded", B=1, new=(2048, 2048), prior=(28672, 28672), H=40,
                dn=128, rd=64, dv=128),
        # a step of a beam search, bf16 pages
        _pages("fork_beams_bf16", op="fork", fmt="bf16", B=64, total=(512, 8192), KV=8, d=128,
               page=64),
        # an answer sampled many times from each prompt, pages of latents
        _pages("fork_samples_latent", op="fork", fmt="latent", B=256, total=(1, 1000), KV=1, d=576,
               page=16),
        # eviction by importance in a serving batch, a quarter kept, bf16 pages
        _pages("compact_bf16", op="compact", fmt="bf16", B=64, total=(512, 8192), keep=0.25, KV=8,
               d=128, rd=128, page=64),
        # eviction in a few short sequences, 8-bit pages
        _pages("compact_e4m3", op="compact", fmt="e4m3", B=4, total=(100, 1500), keep=0.5, KV=2,
               d=64, rd=64, page=32),
    ]


def _latent(name, op, B, H, rd, new=(1, 1), prior=(0, 0), R=512, dn=128, dv=128, page=64, lens=1,
            interleaved=False, yarn=False, base=1e4):
    """A case of latent attention as plain values; `lens` seeds the sequences' lengths."""
    c = dict(op=op, B=B, H=H, rd=rd, new_lo=new[0], new_hi=new[1], prior_lo=prior[0],
             prior_hi=prior[1], lens=lens)
    if op == "expanded":
        c.update(dn=dn, dv=dv)
    else:
        c.update(R=R, page=page)
    if op == "latent_append":
        c.update(interleaved=interleaved, yarn=yarn, base=base)
    if name is not None:
        c["name"] = name
    return c


def _pages(name, op, fmt, B, KV, d, page, total, keep=1.0, rd=0, lens=1, base=5e5):
    """A case of a cache's pages; a latent cache's rows have one head and no values."""
    c = dict(op=op, fmt=fmt, B=B, KV=KV, d=d, page=page, total_lo=total[0], total_hi=total[1],
             lens=lens)
    if op == "compact":
        c.update(keep=keep, rd=rd, base=base)
    if name is not None:
        c["name"] = name
    return c


def draw(rng):
    """One more case: any operator, head layout, page size and raggedness of the ranges above."""

    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def span(top, ragged, low=1):
        hi = log_int(low, max(low, top))
        return (rng.randint(low, hi), hi) if ragged else (hi, hi)

    op = rng.choice(("latent_append", "absorbed", "absorbed", "expanded", "fork", "compact"))
    ragged = rng.random() < 0.7
    lens = rng.randrange(1 << 30)
    page = rng.choice((16, 32, 64, 128))
    if op in ("latent_append", "absorbed"):
        B = log_int(1, 64)
        shape = dict(op=op, B=B, R=rng.choice((128, 256, 512, 512)), rd=rng.choice((32, 64, 64)),
                     page=page, lens=lens)
        if op == "latent_append":
            prior_hi = log_int(1, 2048)
            return _latent(None, H=log_int(1, 64), new=span(min(2048, max(1, 8192 // B)), ragged),
                           prior=(rng.randint(0, prior_hi), prior_hi),
                           interleaved=rng.random() < 0.5, yarn=rng.random() < 0.3,
                           base=rng.choice((1e4, 5e5, 1e6)), **shape)
        new = (1, 1) if rng.random() < 0.6 else span(max(1, 256 // B), ragged)
        H = log_int(1, 64)
        # at most the keys and the products of the listed batches
        top = max(64, min(131072, 262144 // B, (1 << 26) // (B * new[1] * H)))
        prior_hi = log_int(1, top)
        return _latent(None, H=H, new=new, prior=(rng.randint(0, prior_hi), prior_hi), **shape)
    if op == "expanded":
        B = log_int(1, 16)
        H = log_int(1, 40)
        new = span(min(1024, max(1, 4096 // B)), ragged)
        prior_hi = log_int(1, max(16, min(8192, 16384 // B)))
        return _latent(None, op=op, B=B, H=H, rd=rng.choice((32, 64, 64)),
                       dn=rng.choice((64, 128, 128)), dv=rng.choice((64, 128, 128)), new=new,
                       prior=(rng.randint(0, prior_hi), prior_hi), lens=lens)
    if op == "fork":
        fmt = rng.choice(("bf16", "e4m3", "latent"))
        B = log_int(1, 256)
        KV, d = (1, rng.choice((160, 320, 576))) if fmt == "latent" else (rng.choice((1, 2, 8)),
                                                                          rng.choice((64, 128)))
        return _pages(None, op=op, fmt=fmt, B=B, KV=KV, d=d, page=page,
                      total=span(max(16, 262144 // B // KV), ragged), lens=lens)
    B = log_int(1, 64)
    KV, d = rng.choice((1, 2, 8)), rng.choice((64, 128))
    return _pages(None, op=op, fmt=rng.choice(("bf16", "e4m3")), B=B, KV=KV, d=d, page=page,
                  total=span(max(16, min(65536, 262144 // B)), ragged),
                  keep=rng.choice((0.1, 0.25, 0.5, 0.9)), rd=rng.choice((0, d, d // 2)), lens=lens,
                  base=rng.choice((1e4, 5e5)))


def _lengths(c):
    """Per sequence: tokens before the call, and new tokens."""
    r = random.Random(c["lens"])
    prior = [r.randint(c["prior_lo"], c["prior_hi"]) for _ in range(c["B"])]
    return prior, [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["B"])]


def _totals(c):
    r = random.Random(c["lens"])
    return [r.randint(c["total_lo"], c["total_hi"]) for _ in range(c["B"])]


def _family(c):
    """Parents and the positions that every sequence needs room for beyond its parent's tokens:
    a third of the sequences end, their places are taken by children of others."""
    r = random.Random(c["lens"] + 1)
    B = c["B"]
    alive = sorted(r.sample(range(B), max(1, B - B // 3)))
    parents = [r.choice(alive) if r.random() < 0.5 else b for b in range(B)]
    return [p if r.random() < 0.95 else -1 for p in parents], [r.randint(0, 8) for _ in range(B)]


def _copied(c):
    """Pages that a fork copies."""
    lens, (parents, _) = _totals(c), _family(c)
    seen, n = set(), 0
    for p in parents:
        n += p in seen and lens[p] % c["page"] > 0
        seen.add(p)
    return n


def _row_bytes(c):
    """Bytes of one token in one kv head's pages, keys and values."""
    return {"bf16": 4, "e4m3": 2, "latent": 2}[c["fmt"]] * c["d"]


def work(c):
    if c["op"] == "fork":
        table = 4 * sum(-(-n // c["page"]) for n in _totals(c))
        return {"bytes": 2 * _copied(c) * c["KV"] * c["page"] * _row_bytes(c) + 2 * table, "flops": 0}
    if c["op"] == "compact":
        kept = sum(_kept(c, n) for n in _totals(c))
        return {"bytes": 2 * kept * c["KV"] * _row_bytes(c) + 4 * kept,
                "flops": 3 * kept * c["KV"] * c["rd"]}
    prior, new = _lengths(c)
    H, rd, T = c["H"], c["rd"], sum(new)
    if c["op"] == "latent_append":
        # a token's row in and out, the queries' rotated parts in and out
        return {"bytes": 4 * T * (c["R"] + rd + H * rd), "flops": 3 * T * (c["R"] + rd + H * rd)}
    pairs = sum(n * p + n * (n + 1) // 2 for p, n in zip(prior, new))
    keys = sum(prior) + T
    if c["op"] == "absorbed":
        wide = c["R"] + rd
        return {"bytes": 2 * keys * wide + 2 * T * H * (wide + c["R"]),
                "flops": 2 * H * pairs * (wide + c["R"])}
    wide = c["dn"] + rd
    return {"bytes": 2 * keys * (H * (c["dn"] + c["dv"]) + rd) + 2 * T * H * (wide + c["dv"]),
            "flops": 2 * H * pairs * (wide + c["dv"])}


def _kept(c, n):
    return max(1, round(n * c["keep"]))


# --------------------------------------------------------------- inputs ----

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pool(gen, n, KV, page, d, fmt):
    """Pages and, for 8-bit ones, their scales; every page and head with a magnitude of its own."""
    dev = "cuda"
    shape = (n, page, d) if fmt == "latent" else (n, KV, page, d)
    kind = torch.float8_e4m3fn if fmt == "e4m3" else torch.bfloat16
    pool = torch.empty(shape, dtype=kind, device=dev)
    scale = torch.empty(n, KV, dtype=torch.uint8, device=dev) if fmt == "e4m3" else None
    step = max(1, (1 << 27) // (KV * page * d))
    for i in range(0, n, step):
        x = torch.randn((min(step, n - i),) + shape[1:], generator=gen, device=dev)
        if fmt == "latent":
            pool[i:i + step] = x.to(kind)
            continue
        x *= torch.exp2(torch.randn(x.shape[0], KV, 1, 1, generator=gen, device=dev) * 0.7)
        if fmt == "e4m3":
            e = _exponent(x.abs().amax(dim=(2, 3)))
            scale[i:i + step] = (e + 127).to(torch.uint8)
            x *= torch.exp2(-e.float())[..., None, None]
        pool[i:i + step] = x.to(kind)
    return pool, scale


def _table(gen, per, pages):
    """A page table whose sequences have per[b] pages, out of `pages` in no order; the rest is -1.
    Also the pages that nobody has."""
    ids = torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int32)
    table = torch.full((len(per), max(per)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, ids[at:]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    make = {"latent_append": _prepare_latent, "absorbed": _prepare_latent,
            "expanded": _prepare_expanded, "fork": _prepare_fork, "compact": _prepare_compact}
    s = make[case["op"]](case, gen)
    s["case"] = case
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


def _bf16(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)


def _packed(c):
    prior, new = _lengths(c)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return prior, new, dict(T=cu[-1], cu=_ints(cu), prior=_ints(prior), max_new=max(new),
                            max_total=max(p + n for p, n in zip(prior, new)))


def _prepare_latent(c, gen):
    prior, new, s = _packed(c)
    T, H, R, rd, page = s["T"], c["H"], c["R"], c["rd"], c["page"]
    per = [-(-(p + n) // page) for p, n in zip(prior, new)]
    s["kv"], _ = _pool(gen, sum(per) + 3, 1, page, R + rd, "latent")
    s["table"], _ = _table(gen, per, sum(per) + 3)
    if c["op"] == "latent_append":
        s["new_kv"], s["q"] = _bf16(gen, T, R + rd), _bf16(gen, T, H, 2 * rd)
        s["norm_w"] = (1 + 0.1 * torch.randn(R, generator=gen, device="cuda")).to(torch.bfloat16)
        s["q_out"] = torch.zeros(T, H, R + rd, dtype=torch.bfloat16, device="cuda")
        return s
    s["q"] = _bf16(gen, T, H, R + rd)
    s["out"] = torch.zeros(T, H, R, dtype=torch.bfloat16, device="cuda")
    # scratch of the serving loop: room for the partial results of any split of these calls
    s["workspace"] = torch.empty(96 << 20, dtype=torch.uint8, device="cuda")
    return s


def _prepare_expanded(c, gen):
    prior, new, s = _packed(c)
    lens = [p + n for p, n in zip(prior, new)]
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    s["starts"], s["key_lens"] = _ints(at[:-1]), _ints(lens)
    s["q"] = _bf16(gen, s["T"], c["H"], c["dn"] + c["rd"])
    s["kv"] = _bf16(gen, at[-1], c["H"], c["dn"] + c["dv"])
    s["k_pe"] = _bf16(gen, at[-1], c["rd"])
    s["out"] = torch.zeros(s["T"], c["H"], c["dv"], dtype=torch.bfloat16, device="cuda")
    return s


def _prepare_fork(c, gen):
    lens, (parents, grow) = _totals(c), _family(c)
    page, B = c["page"], c["B"]
    per = [-(-n // page) for n in lens]
    most = -(-(max(lens) + max(grow)) // page) + 1
    pages = sum(per) + 2 * B + 5  # the server's pool has some pages free
    s = {}
    s["k"], s["k_scale"] = _pool(gen, pages, c["KV"], page, c["d"], c["fmt"])
    s["v"], s["v_scale"] = (None, None) if c["fmt"] == "latent" else _pool(
        gen, pages, c["KV"], page, c["d"], c["fmt"])
    table, _ = _table(gen, per, pages)
    s["table"] = torch.full((B, most), -1, dtype=torch.int32, device="cuda")
    s["table"][:, :table.shape[1]] = table
    s["ref"] = torch.zeros(pages, dtype=torch.int32, device="cuda")
    s["ref"][table[table >= 0].long()] = 1
    s["lens"], s["parents"], s["grow"] = _ints(lens), _ints(parents), _ints(grow)
    s["new_table"], s["new_ref"] = torch.empty_like(s["table"]), torch.empty_like(s["ref"])
    s["new_lens"], s["src"], s["dst"] = (torch.empty_like(s["lens"]) for _ in range(3))
    return s


def _prepare_compact(c, gen):
    lens, page = _totals(c), c["page"]
    kept = [_kept(c, n) for n in lens]
    per, new_per = [-(-n // page) for n in lens], [-(-n // page) for n in kept]
    pages = sum(per) + sum(new_per) + 3
    s = {}
    s["k"], s["k_scale"] = _pool(gen, pages, c["KV"], page, c["d"], c["fmt"])
    s["v"], s["v_scale"] = _pool(gen, pages, c["KV"], page, c["d"], c["fmt"])
    s["table"], rest = _table(gen, per, pages)
    s["new_table"] = torch.full((c["B"], max(new_per)), -1, dtype=torch.int32, device="cuda")
    s["keep"] = torch.zeros(c["B"], max(kept), dtype=torch.int32, device="cuda")
    at = 0
    for b, (n, m) in enumerate(zip(lens, kept)):
        s["new_table"][b, :new_per[b]] = rest[at:at + new_per[b]]
        at += new_per[b]
        # the last tokens and the most important of the others, in their order
        imp = torch.rand(n, generator=gen, device="cuda")
        imp[-max(1, m // 4):] += 1
        s["keep"][b, :m] = imp.topk(m).indices.sort().values
    s["kept"], s["max_kept"] = _ints(kept), max(kept)
    return s


# ----------------------------------------------------------- plain forms ----

def _exponent(amax):
    """Smallest e with amax <= 448 * 2^e, clamped to E8M0's range (-127 for 0)."""
    m, x = torch.frexp(amax)  # amax = m 2^x, m in [0.5, 1); 448 = 0.875 * 2^9
    e = x - 9 + (m > 0.875).to(x.dtype)
    return torch.where(amax > 0, e.clamp(-127, 127), torch.full_like(e, -127))


def _inv_freq(rd, base, yarn):
    """RoPE frequencies, with YaRN's ramp (factor 4 over 8192 positions, betas 32 and 1) where asked."""
    i = torch.arange(rd // 2, dtype=torch.float64, device="cuda")
    f = base ** (-2.0 * i / rd)
    if not yarn:
        return f, 1.0
    at = lambda rot: rd * math.log(8192 / (rot * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    low = max(math.floor(at(32.0)), 0)
    high = min(max(math.ceil(at(1.0)), 0), max(rd // 2 - 1, 0))
    ramp = ((i - low).clamp(min=0) / max(high - low, 1)).clamp(max=1)
    return f * (1 - ramp) + f / 4.0 * ramp, 0.1 * math.log(4.0) + 1.0


def _rotated(x, pos, rd, base, yarn=False, interleaved=False):
    """The first rd of x's last dimension turned, in 64 bits (angles of far positions, values next
    to a rounding border); pos broadcasts against x without its last dimension."""
    x = x.double()
    f, factor = _inv_freq(rd, base, yarn)
    a = pos.double()[..., None] * f
    cos, sin = torch.cos(a) * factor, torch.sin(a) * factor
    if interleaved:
        x0, x1 = x[..., 0:rd:2], x[..., 1:rd:2]
    else:
        x0, x1 = x[..., :rd // 2], x[..., rd // 2:rd]
    y0, y1 = x0 * cos - x1 * sin, x1 * cos + x0 * sin
    y = torch.stack([y0, y1], dim=-1).flatten(-2) if interleaved else torch.cat([y0, y1], dim=-1)
    return torch.cat([y, x[..., rd:]], dim=-1)


def _owners(s):
    """Of each new token: its sequence, its index there, its position."""
    cu, prior = s["cu"].long(), s["prior"].long()
    t = torch.arange(s["T"], device=cu.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    return b, t - cu[b], prior[b] + t - cu[b]


def _plain_latent_append(s):
    c = s["case"]
    R, rd, page = c["R"], c["rd"], c["page"]
    how = dict(rd=rd, base=c["base"], yarn=c["yarn"], interleaved=c["interleaved"])
    b, _, pos = _owners(s)
    x = s["new_kv"].double()
    latent = x[:, :R] / torch.sqrt(x[:, :R].square().mean(dim=-1, keepdim=True) + 1e-6)
    row = torch.cat([latent * s["norm_w"].double(), _rotated(x[:, R:], pos, **how)], dim=-1)
    s["kv"][s["table"][b, pos // page].long(), pos % page] = row.to(torch.bfloat16)
    s["q_out"][..., R:] = _rotated(s["q"][..., rd:], pos[:, None], **how).to(torch.bfloat16)
    return s["kv"], s["q_out"]


def _softmax_(x, seen):
    """Softmax over the last dimension, in place; a row that sees nothing becomes zeros."""
    x.masked_fill_(~seen, float("-inf"))
    top = x.amax(dim=-1, keepdim=True)
    x.sub_(torch.where(torch.isfinite(top), top, torch.zeros_like(top))).exp_()
    total = x.sum(dim=-1, keepdim=True)
    return x.div_(torch.where(total > 0, total, torch.ones_like(total)))


def _plain_absorbed(s):
    c = s["case"]
    B, H, R, N = c["B"], c["H"], c["R"], s["max_new"]
    wide = R + c["rd"]
    b, i, pos = _owners(s)
    rows = s["kv"][s["table"].clamp(min=0).long()].float().view(B, -1, wide)
    q = torch.zeros(B, N, H, wide, device="cuda")
    q[b, i] = s["q"].float()
    lim = torch.zeros(B, N, dtype=torch.long, device="cuda")
    lim[b, i] = pos + 1
    x = torch.matmul(q.view(B, N * H, wide), rows.transpose(1, 2)).mul_(_scale(c))
    seen = torch.arange(rows.shape[1], device="cuda") < lim.repeat_interleave(H, dim=1)[..., None]
    o = torch.matmul(_softmax_(x, seen), rows[..., :R])
    s["out"].copy_(o.view(B, N, H, R)[b, i])
    return (s["out"],)


def _scale(c):
    """The scale of scores over nope and rotated dimensions (128 and rd in the absorbed cases)."""
    return 1.0 / math.sqrt(c.get("dn", 128) + c["rd"])


def _plain_expanded(s):
    c = s["case"]
    B, H, dn, rd, dv, N, K = c["B"], c["H"], c["dn"], c["rd"], c["dv"], s["max_new"], s["max_total"]
    b, i, pos = _owners(s)
    q = torch.zeros(B, H, N, dn + rd, device="cuda")
    q[b, :, i] = s["q"].float()
    lim = torch.zeros(B, N, dtype=torch.long, device="cuda")
    lim[b, i] = pos + 1
    j = torch.arange(K, device="cuda")
    at = (s["starts"].long()[:, None] + j).clamp(max=s["kv"].shape[0] - 1)
    kv = s["kv"][at].permute(0, 2, 1, 3)  # [B, H, K, dn + dv]
    x = torch.matmul(q[..., :dn], kv[..., :dn].float().transpose(-1, -2))
    x += torch.matmul(q[..., dn:], s["k_pe"][at].float().transpose(-1, -2)[:, None])
    x = _softmax_(x.mul_(_scale(c)), (j < lim[..., None])[:, None])
    o = torch.matmul(x, kv[..., dn:].float())
    s["out"].copy_(o.permute(0, 2, 1, 3)[b, i])
    return (s["out"],)


def _plain_fork(s):
    c = s["case"]
    page, (B, P) = c["page"], s["table"].shape
    dev = s["table"].device
    parents, b, j = s["parents"].long(), torch.arange(B, device=dev), torch.arange(P, device=dev)
    has = parents >= 0
    p = parents.clamp(min=0)
    elder = (parents[:, None] == parents) & (b < b[:, None])
    first = has & ~elder.any(dim=1)
    n = torch.where(has, s["lens"].long()[p], torch.zeros_like(p))
    held = torch.where(has[:, None], s["table"][p], torch.full_like(s["table"], -1))
    ids = torch.where(first[:, None] | (j < (n // page)[:, None]), held, torch.full_like(held, -1))
    count = lambda t: torch.zeros(len(s["ref"]) + 1, dtype=torch.int32, device=dev).index_add_(  # noqa: E731
        0, torch.where(t >= 0, t, torch.full_like(t, len(s["ref"]))).flatten().long(),
        torch.ones(t.numel(), dtype=torch.int32, device=dev))[:-1]
    ref = s["ref"] - count(s["table"]) + count(ids)
    # the pages that are missing, from the free ones in order
    need = (j < ((n + s["grow"].long() + page - 1) // page)[:, None]) & (ids < 0)
    free = (ref == 0).nonzero()[:, 0].to(torch.int32)
    rank = need.flatten().long().cumsum(0).view(B, P) - 1
    got = need & (rank < len(free))
    ids = torch.where(got, free[rank.clamp(0, len(free) - 1)], ids)
    ref[ids[got].long()] = 1
    copied = has & ~first & (n % page > 0)
    at = (n // page).clamp(max=P - 1)[:, None]
    none = torch.full_like(s["src"], -1)
    s["dst"].copy_(torch.where(copied, ids.gather(1, at)[:, 0], none))
    s["src"].copy_(torch.where(copied & (s["dst"] >= 0), held.gather(1, at)[:, 0], none))
    s["new_table"].copy_(ids)
    s["new_ref"].copy_(ref)
    s["new_lens"].copy_(n)
    real = s["src"] >= 0
    src, dst = s["src"][real].long(), s["dst"][real].long()
    pools = [t for t in (s["k"], s["v"], s["k_scale"], s["v_scale"]) if t is not None]
    for t in pools:
        t.view(torch.uint8)[dst] = t.view(torch.uint8)[src]
    return [s["new_table"], s["new_ref"], s["new_lens"], s["src"], s["dst"]] + pools


def _plain_compact(s):
    c = s["case"]
    page = c["page"]
    j = torch.arange(s["max_kept"], device="cuda")
    b, j = (j < s["kept"][:, None]).nonzero(as_tuple=True)
    old = s["keep"][b, j].long()
    src, at = s["table"][b, old // page].long(), old % page
    dst, to = s["new_table"][b, j // page].long(), j % page
    for pool, scale, turn in ((s["k"], s["k_scale"], c["rd"]), (s["v"], s["v_scale"], 0)):
        x = pool[src, :, at].float()  # [kept, KV, d]
        if scale is not None:
            x *= torch.exp2(scale[src].float() - 127)[..., None]
        if turn:
            x = _rotated(x, (j - old)[:, None], turn, c["base"])
        if scale is not None:
            amax = torch.zeros(scale.shape, dtype=x.dtype, device=x.device)
            amax.scatter_reduce_(0, dst[:, None].expand(-1, c["KV"]), x.abs().amax(dim=-1), "amax")
            e = _exponent(amax)
            scale[dst] = (e[dst] + 127).to(torch.uint8)
            x = x * torch.exp2(-e[dst].to(x.dtype))[..., None]
        pool[dst, :, to] = x.float().to(pool.dtype) if scale is not None else x.to(pool.dtype)
    return [t for t in (s["k"], s["v"], s["k_scale"], s["v_scale"]) if t is not None]


# ------------------------------------------------------------------- run ----

def run(state):
    s = state
    c = s["case"]
    if not own:
        plain = {"latent_append": _plain_latent_append, "absorbed": _plain_absorbed,
                 "expanded": _plain_expanded, "fork": _plain_fork, "compact": _plain_compact}
        return plain[c["op"]](s)
    import causal_gqa_attention_rope_gb300 as na
    if c["op"] in ("latent_append", "absorbed"):
        cfg = na.LatentConfig(c["H"], kv_rank=c["R"], rope_dim=c["rd"], nope_dim=128,
                              rope_interleaved=c.get("interleaved", False))
        cache = na.PagedLatentCache(s["kv"], s["table"])
    if c["op"] == "latent_append":
        rope = na.RopeConfig(base=c["base"], yarn=c["yarn"], factor=4.0, orig_max_pos=8192)
        na.na_latent_append_paged(cfg, rope, s["cu"], s["prior"], s["new_kv"], s["q"][..., c["rd"]:],
                                  s["q_out"][..., c["R"]:], cache, kv_norm_w=s["norm_w"],
                                  status=s["status"])
        return s["kv"], s["q_out"]
    if c["op"] == "absorbed":
        na.na_attn_latent_paged(cfg, s["cu"], s["prior"], s["max_new"], s["max_total"], s["q"], cache,
                                s["out"], workspace=s["workspace"], status=s["status"])
        return (s["out"],)
    if c["op"] == "expanded":
        cfg = na.LatentConfig(c["H"], rope_dim=c["rd"], nope_dim=c["dn"], v_dim=c["dv"])
        na.na_attn_latent_expanded(cfg, s["cu"], s["starts"], s["key_lens"], s["max_new"],
                                   s["max_total"], s["q"], s["kv"], s["k_pe"], s["out"],
                                   status=s["status"])
        return (s["out"],)
    pools = [t for t in (s["k"], s["v"], s["k_scale"], s["v_scale"]) if t is not None]
    if c["op"] == "fork":
        na.na_pages_fork(s["parents"], s["lens"], s["table"], s["ref"], c["page"], s["new_table"],
                         s["new_ref"], s["new_lens"], s["src"], s["dst"], grow=s["grow"],
                         status=s["status"])
        if c["fmt"] == "latent":
            cache = na.PagedLatentCache(s["k"], s["new_table"])
        else:
            cache = na.PagedKVCache(s["k"], s["v"], s["new_table"], s["k_scale"], s["v_scale"])
        na.na_pages_copy(cache, s["src"], s["dst"], status=s["status"])
        return [s["new_table"], s["new_ref"], s["new_lens"], s["src"], s["dst"]] + pools
    cache = na.PagedKVCache(s["k"], s["v"], s["table"], s["k_scale"], s["v_scale"])
    new = na.PagedKVCache(s["k"], s["v"], s["new_table"], s["k_scale"], s["v_scale"])
    na.na_pages_compact(cache, new, s["kept"], s["max_kept"], keep=s["keep"],
                        rope=na.RopeConfig(base=c["base"]) if c["rd"] else None,
                        rotary_dim=c["rd"], status=s["status"])
    return pools


# ----------------------------------------------------------------- exact ----

def exact(case, seed):
    """The definition in 64 bits, sequence by sequence, unrounded (a fork computes no numbers)."""
    if case["op"] == "fork":
        return None
    s = prepare(case, seed)
    return {"latent_append": _exact_append, "absorbed": _exact_absorbed,
            "expanded": _exact_expanded, "compact": _exact_compact}[case["op"]](case, s)


def _angles(pos, rd, base, yarn):
    freq = []
    for i in range(rd // 2):
        f = base ** (-2.0 * i / rd)
        if yarn:
            edge = [rd * math.log(8192 / (r * 2 * math.pi)) / (2 * math.log(base)) for r in (32.0, 1.0)]
            lo = max(0, math.floor(edge[0]))
            hi = min(rd // 2 - 1, max(0, math.ceil(edge[1])))
            mix = min(1.0, max(0, i - lo) / max(1, hi - lo))
            f = f * (1 - mix) + f / 4.0 * mix
        freq.append(f)
    return pos.double()[..., None] * torch.tensor(freq, dtype=torch.float64, device=pos.device)


def _turned(x, angle, gain=1.0, interleaved=False):
    """Pairs as complex numbers, turned by the angle."""
    h = angle.shape[-1]
    z = x.reshape(*x.shape[:-1], h, 2) if interleaved else torch.stack((x[..., :h], x[..., h:]), dim=-1)
    z = torch.view_as_complex(z.contiguous()) * (gain * torch.polar(torch.ones_like(angle), angle))
    return torch.view_as_real(z).flatten(-2) if interleaved else torch.cat((z.real, z.imag), dim=-1)


def _spans(case):
    at = 0
    for b, (p, n) in enumerate(zip(*_lengths(case))):
        yield b, p, n, at
        at += n


def _exact_append(case, s):
    R, rd, page = case["R"], case["rd"], case["page"]
    gain = 0.1 * math.log(4.0) + 1.0 if case["yarn"] else 1.0
    pool, q = s["kv"].double(), s["q_out"].double()
    for b, p, n, at in _spans(case):
        pos = torch.arange(p, p + n, device="cuda")
        angle = _angles(pos, rd, case["base"], case["yarn"])
        x = s["new_kv"][at:at + n].double()
        c = x[:, :R] * torch.rsqrt(x[:, :R].square().sum(-1, keepdim=True) / R + 1e-6)
        row = torch.cat((c * s["norm_w"].double(), _turned(x[:, R:], angle, gain, case["interleaved"])), -1)
        pool[s["table"][b, pos // page].long(), pos % page] = row
        q[at:at + n, :, R:] = _turned(s["q"][at:at + n, :, rd:].double(), angle[:, None], gain,
                                      case["interleaved"])
    return pool, q


def _causal(x, p, n):
    """Softmax of x [..., n, p + n] where the i-th query sees keys up to p + i."""
    key = torch.arange(p + n, device=x.device)
    return torch.softmax(x.masked_fill(key > torch.arange(p, p + n, device=x.device)[:, None],
                                       float("-inf")), dim=-1)


def _exact_absorbed(case, s):
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for b, p, n, at in _spans(case):
        ids = s["table"][b, :-(-(p + n) // case["page"])].long()
        rows = s["kv"][ids].double().flatten(0, 1)[:p + n]
        x = torch.einsum("nhd,kd->hnk", s["q"][at:at + n].double(), rows) * _scale(case)
        out[at:at + n] = torch.einsum("hnk,kd->nhd", _causal(x, p, n), rows[:, :case["R"]])
    return (out,)


def _exact_expanded(case, s):
    dn = case["dn"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for b, p, n, at in _spans(case):
        k0 = int(s["starts"][b])
        pe = s["k_pe"][k0:k0 + p + n].double()
        for h in range(case["H"]):
            q, kv = s["q"][at:at + n, h].double(), s["kv"][k0:k0 + p + n, h].double()
            x = torch.cat((q[:, :dn] @ kv[:, :dn].T, q[:, dn:] @ pe.T)).view(2, n, p + n).sum(0)
            out[at:at + n, h] = _causal(x * _scale(case), p, n) @ kv[:, dn:]
    return (out,)


def _exact_compact(case, s):
    page, rd = case["page"], case["rd"]
    pools = [s["k"].double(), s["v"].double()]
    scales = [t if t is None else t.clone() for t in (s["k_scale"], s["v_scale"])]
    for b, m in enumerate(s["kept"].tolist()):
        old = s["keep"][b, :m].long()
        src = s["table"][b, old // page].long()
        new = torch.arange(m, device="cuda")
        for which in range(2):
            pool, scale = pools[which], scales[which]
            x = pool[src, :, old % page]  # [m, KV, d]
            if scale is not None:
                x = x * (2.0 ** (scale[src].double() - 127))[..., None]
            if which == 0 and rd:
                angle = _angles(new - old, rd, case["base"], False)[:, None]
                x = torch.cat((_turned(x[..., :rd], angle), x[..., rd:]), dim=-1)
            for lo in range(0, m, page):
                part = x[lo:lo + page]
                pid = int(s["new_table"][b, lo // page])
                if scale is not None:
                    # (a stored magnitude is often 448 times a power of two: no log decides those)
                    top = part.abs().amax(dim=(0, 2))
                    need = torch.round(torch.log2(top / E4M3_MAX))
                    need = (need + (top > E4M3_MAX * torch.exp2(need))).clamp(-127, 127)
                    part = part / torch.exp2(need)[:, None]
                    scale[pid] = (need + 127).to(torch.uint8)
                pool[pid, :, :part.shape[0]] = part.transpose(0, 1)
    return pools + [t for t in scales if t is not None]
