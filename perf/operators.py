"""Performance cases of the paged key/value cache: the fused append and the two attention calls.

The cache is a pool of pages, k and v [num_pages, KV, page, d], and a page
table [batch, pages a sequence] that says which page holds positions
[i * page, (i + 1) * page) of a sequence.  Pages hold bf16, or E4M3 with one
power-of-two scale (an E8M0 byte s: 2^(s - 127)) for each page and kv head.

  append   q_out = RoPE(norm(q)); K (normed, rotated) and V go into their pages.
           With E4M3 pages a page's scale is the smallest power of two 2^e with
           max |x| <= 448 * 2^e over the page's tokens; it only grows while the
           page fills, and when it does, the tokens that were there are rounded
           to the new scale.
  decode   one query per sequence against its pages, with the probabilities
           that importance-aware eviction reads where the case asks for them.
  prefill  a chunk of new tokens per sequence (already in the pages) against
           the pages, causal.

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
        # a decode step's new tokens into bf16 pages: 64 sequences, one token each
        _case("append_step_bf16", op="append", fmt="bf16", B=64, new=(1, 1), prior=(0, 1024),
              H=32, KV=8, d=128, rd=128, page=64),
        # the same step into 8-bit pages, a small model's heads
        _case("append_step_e4m3_d64", op="append", fmt="e4m3", B=32, new=(1, 1), prior=(0, 1024),
              H=4, KV=2, d=64, rd=64, page=32),
        # one chunk of a long YaRN prompt into 8-bit pages
        _case("append_chunk_e4m3", op="append", fmt="e4m3", B=1, new=(2048, 2048),
              prior=(2048, 2048), H=40, KV=8, d=128, rd=64, page=64, yarn=True, base=1e6),
        # a mixed batch of prompt chunks with normed q and k, small pages, ragged lengths
        _case("append_varlen_e4m3", op="append", fmt="e4m3", B=16, new=(1, 512), prior=(0, 1000),
              H=32, KV=4, d=128, rd=128, page=16, qk_norm=True, base=1e6),
        # one short conversation: the latency of a call
        _case("decode_one_e4m3_d64", op="decode", fmt="e4m3", B=1, total=(333, 333), H=4, KV=2,
              d=64, page=16),
        # a serving batch of mixed lengths with probabilities, 8-bit pages
        _case("decode_b64_e4m3_probs", op="decode", fmt="e4m3", B=64, total=(512, 8192), H=32,
              KV=8, d=128, page=64, probs=True),
        # the same batch without them, bf16 pages
        _case("decode_b64_bf16", op="decode", fmt="bf16", B=64, total=(512, 8192), H=32, KV=8,
              d=128, page=64),
        # a few long contexts, smallest pages, gated output
        _case("decode_long_e4m3", op="decode", fmt="e4m3", B=4, total=(50001, 131072), H=32, KV=4,
              d=128, page=16, gate=True),
        # a 128-token chunk in the middle of a prompt, bf16 pages
        _case("prefill_chunk_bf16", op="prefill", fmt="bf16", B=1, new=(128, 128),
              prior=(3968, 3968), H=32, KV=8, d=128, page=64),
        # drafted tokens of a speculative step, a few per sequence
        _case("prefill_verify_e4m3", op="prefill", fmt="e4m3", B=64, new=(2, 8), prior=(512, 8184),
              H=32, KV=8, d=128, page=64),
        # a mixed step: prompts of many lengths over cached histories, gated output
        _case("prefill_varlen_e4m3", op="prefill", fmt="e4m3", B=16, new=(1, 512),
              prior=(0, 16384), H=32, KV=4, d=128, page=64, gate=True),
        # one chunk of a long prompt: bound by the matrix products
        _case("prefill_long_e4m3", op="prefill", fmt="e4m3", B=1, new=(2048, 2048),
              prior=(28672, 28672), H=40, KV=8, d=128, page=128),
    ]


def _case(name, op, fmt, B, H, KV, d, page, new=(1, 1), prior=(0, 0), total=(1, 1), rd=0, lens=1,
          qk_norm=False, yarn=False, base=5e5, probs=False, gate=False, softcap=0.0, window=0):
    """A case as plain values; `lens` seeds the sequences' lengths."""
    c = dict(op=op, fmt=fmt, B=B, H=H, KV=KV, d=d, page=page, lens=lens)
    if op == "decode":
        c.update(total_lo=total[0], total_hi=total[1], probs=probs)
    else:
        c.update(new_lo=new[0], new_hi=new[1], prior_lo=prior[0], prior_hi=prior[1])
    if op == "append":
        c.update(rd=rd, qk_norm=qk_norm, yarn=yarn, base=base)
    else:
        c.update(gate=gate, softcap=softcap, window=window)
    if name is not None:
        c["name"] = name
    return c


def draw(rng):
    """One more case: any operator, head layout, page size and raggedness of the ranges above."""

    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def span(top, ragged):
        hi = log_int(1, top)
        return (rng.randint(1, hi), hi) if ragged else (hi, hi)

    op = rng.choice(("append", "decode", "prefill"))
    fmt = rng.choice(("e4m3", "e4m3", "bf16"))
    d = rng.choice((64, 128, 128))
    KV = rng.choice((1, 2, 4, 8))
    H = KV * rng.choice((1, 2, 3, 4, 5, 8))
    page = rng.choice((16, 32, 64, 128))
    B = log_int(1, 64)
    ragged = rng.random() < 0.7
    common = dict(op=op, fmt=fmt, B=B, H=H, KV=KV, d=d, page=page, lens=rng.randrange(1 << 30))
    if op == "append":
        new = span(min(2048, max(1, 8192 // B)), ragged)
        prior_hi = log_int(1, 2048)
        return _case(None, new=new, prior=(rng.randint(0, prior_hi), prior_hi),
                     rd=rng.choice((d, d // 2, d // 4 + 2)), qk_norm=rng.random() < 0.5,
                     yarn=rng.random() < 0.3, base=rng.choice((1e4, 5e5, 1e6)), **common)
    extra = dict(gate=rng.random() < 0.3, softcap=rng.choice((0.0, 0.0, 0.0, 30.0)),
                 window=rng.choice((0, 0, 0, log_int(16, 4096))))
    if op == "decode":
        # at most the keys of the listed batches
        return _case(None, total=span(max(64, min(65536, 262144 // B)), ragged),
                     probs=rng.random() < 0.5, **extra, **common)
    new = span(min(1024, max(1, 2048 // B)), ragged)
    prior_hi = log_int(1, max(64, min(16384, 131072 // B)))
    return _case(None, new=new, prior=(rng.randint(0, prior_hi), prior_hi), **extra, **common)


def _lengths(c):
    """Per sequence: cached tokens before the call, and new tokens (decode: the one attending)."""
    r = random.Random(c["lens"])
    if c["op"] == "decode":
        total = [r.randint(c["total_lo"], c["total_hi"]) for _ in range(c["B"])]
        return [n - 1 for n in total], [1] * c["B"]
    prior = [r.randint(c["prior_lo"], c["prior_hi"]) for _ in range(c["B"])]
    return prior, [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["B"])]


def work(c):
    prior, new = _lengths(c)
    H, KV, d, size = c["H"], c["KV"], c["d"], (1 if c["fmt"] == "e4m3" else 2)
    T = sum(new)
    if c["op"] == "append":
        # q in and out, k and v in, and out in the pages' type; a rotation is 3 operations an element
        return {"bytes": T * d * (4 * H + 4 * KV + 2 * KV * size), "flops": 3 * T * d * (H + KV)}
    w = c["window"]
    pairs = keys = 0  # (query, key) pairs that are seen, and keys that any query sees
    for p, n in zip(prior, new):
        if w == 0:
            pairs += n * p + n * (n + 1) // 2
            keys += p + n
        else:
            pairs += sum(min(w, p + i + 1) for i in range(n))
            keys += p + n - max(0, p - w + 1)
    data = 2 * keys * KV * d * size + (keys // c["page"] * KV * 2 if size == 1 else 0)
    data += T * H * d * (6 if c["gate"] else 4)
    if c.get("probs"):
        data += 4 * H * sum(p + 1 for p in prior)
    return {"bytes": data, "flops": 4 * H * d * pairs}


# --------------------------------------------------------------- inputs ----

def _pages(gen, n, KV, page, d, fmt):
    """A pool half a serving day old: every page and head with a magnitude of its own."""
    dev = "cuda"
    mag = torch.exp2(torch.randn(n, KV, 1, 1, generator=gen, device=dev) * 0.7)
    if fmt == "bf16":
        pool = torch.empty(n, KV, page, d, dtype=torch.bfloat16, device=dev)
    else:
        pool = torch.empty(n, KV, page, d, dtype=torch.float8_e4m3fn, device=dev)
    scale = torch.empty(n, KV, dtype=torch.uint8, device=dev)
    step = max(1, (1 << 27) // (KV * page * d))
    for i in range(0, n, step):
        m = mag[i:i + step]
        x = torch.randn(m.shape[0], KV, page, d, generator=gen, device=dev) * m
        if fmt == "bf16":
            pool[i:i + step] = x.to(torch.bfloat16)
        else:
            e = _exponent(x.abs().amax(dim=(2, 3)))
            pool[i:i + step] = (x * torch.exp2(-e.float())[..., None, None]).to(pool.dtype)
            scale[i:i + step] = (e + 127).to(torch.uint8)
    return pool, (scale if fmt == "e4m3" else None)


def prepare(case, seed):
    c = case
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    prior, new = _lengths(c)
    B, H, KV, d, page = c["B"], c["H"], c["KV"], c["d"], c["page"]
    T = sum(new)
    per = [-(-(p + n) // page) for p, n in zip(prior, new)]
    P = max(per)
    pages = sum(per) + 3  # the server's pool has a few pages that nobody uses now
    ids = torch.randperm(pages, generator=gen, device=dev, dtype=torch.int32)
    table = torch.full((B, P), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = ids[at:at + n]
        at += n
    s = dict(case=c, table=table, T=T, max_new=max(new), max_total=max(p + n for p, n in zip(prior, new)))
    s["k"], s["k_scale"] = _pages(gen, pages, KV, page, d, c["fmt"])
    s["v"], s["v_scale"] = _pages(gen, pages, KV, page, d, c["fmt"])
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["cu"], s["prior"] = ints(cu), ints(prior)
    s["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
    rnd = lambda *shape: torch.randn(*shape, generator=gen, device=dev).to(torch.bfloat16)  # noqa: E731
    s["q"] = rnd(T, H, d)
    s["out"] = torch.zeros(T, H, d, dtype=torch.bfloat16, device=dev)
    if c["op"] == "append":
        s["new_k"], s["new_v"] = rnd(T, KV, d), rnd(T, KV, d)
        s["qw"] = s["kw"] = None
        if c["qk_norm"]:
            s["qw"] = (1 + 0.1 * torch.randn(d, generator=gen, device=dev)).to(torch.bfloat16)
            s["kw"] = (1 + 0.1 * torch.randn(d, generator=gen, device=dev)).to(torch.bfloat16)
        return s
    s["gate"] = rnd(T, H, d) if c["gate"] else None
    if c["op"] == "decode":
        s["lens"] = s["prior"] + 1
        s["probs"] = torch.zeros(B, H, s["max_total"], device=dev) if c["probs"] else None
    # scratch of the serving loop: room for the partial results of any split of these calls
    s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device=dev)
    return s


# ----------------------------------------------------------- plain forms ----

def _exponent(amax):
    """Smallest e with amax <= 448 * 2^e, clamped to E8M0's range (-127 for 0)."""
    m, x = torch.frexp(amax)  # amax = m 2^x, m in [0.5, 1); 448 = 0.875 * 2^9
    e = x - 9 + (m > 0.875).to(x.dtype)
    return torch.where(amax > 0, e.clamp(-127, 127), torch.full_like(e, -127))


def _inv_freq(c, dev):
    """RoPE frequencies, with YaRN's ramp (factor 4 over 8192 positions, betas 32 and 1) where asked."""
    rd, base = c["rd"], c["base"]
    i = torch.arange(rd // 2, dtype=torch.float64, device=dev)
    f = base ** (-2.0 * i / rd)
    if not c["yarn"]:
        return f, 1.0
    at = lambda rot: rd * math.log(8192 / (rot * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    low = max(math.floor(at(32.0)), 0)
    high = min(max(math.ceil(at(1.0)), 0), max(rd // 2 - 1, 0))
    ramp = ((i - low).clamp(min=0) / max(high - low, 1)).clamp(max=1)
    return f * (1 - ramp) + f / 4.0 * ramp, 0.1 * math.log(4.0) + 1.0


def _normed_rotated(c, x, w, pos):
    """RMS norm over d where the case has it (eps 1e-6), then the rotation of the first rd dims."""
    x = x.double()  # angles of far positions, and values next to a rounding border
    if w is not None:
        x = x / torch.sqrt((x * x).mean(dim=-1, keepdim=True) + 1e-6) * w.double()
    f, factor = _inv_freq(c, x.device)
    a = (pos.double()[:, None] * f)[:, None, :]
    cos, sin = torch.cos(a) * factor, torch.sin(a) * factor
    h = c["rd"] // 2
    x0, x1 = x[..., :h], x[..., h:2 * h]
    return torch.cat([x0 * cos - x1 * sin, x1 * cos + x0 * sin, x[..., 2 * h:]], dim=-1)


def _store_bf16(pool, pid, slot, x):
    pool[pid.long(), :, slot.long()] = x.to(torch.bfloat16)


def _store_e4m3(pool, scale, first, off, pid, slot, x):
    """New tokens' rows x [T, KV, d] into pages pid at slot; first [B] and off [B]: each sequence's
    first page of this call and how many of its tokens are there already."""
    n, KV = scale.shape
    pid = pid.long()
    amax = torch.zeros(n, KV, dtype=x.dtype, device=x.device)
    amax.scatter_reduce_(0, pid[:, None].expand(-1, KV), x.abs().amax(dim=-1), "amax")
    e = _exponent(amax)
    old = torch.full_like(e, -127)
    held = off > 0
    old[first[held].long()] = scale[first[held].long()].to(e.dtype) - 127
    e = torch.maximum(e, old)
    # tokens that were there already, rounded to a scale that grew
    fp = first[held].long()
    rows = pool[fp].float() * torch.exp2((old[fp] - e[fp]).float())[..., None, None]
    there = torch.arange(pool.shape[2], device=x.device) < off[held][:, None]
    pool[fp] = torch.where(there[:, None, :, None], rows, pool[fp].float()).to(pool.dtype)
    y = x * torch.exp2(-e[pid].to(x.dtype))[..., None]
    pool[pid, :, slot.long()] = y.to(torch.float32).to(pool.dtype)
    scale[pid] = (e[pid] + 127).to(torch.uint8)


def _plain_append(s):
    c = s["case"]
    page = c["page"]
    cu, prior, table = s["cu"].long(), s["prior"].long(), s["table"]
    t = torch.arange(s["T"], device=cu.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = prior[b] + t - cu[b]
    pid, slot = table[b, pos // page], pos % page
    s["out"].copy_(_normed_rotated(c, s["q"], s["qw"], pos).to(torch.bfloat16))
    k = _normed_rotated(c, s["new_k"], s["kw"], pos)
    if c["fmt"] == "bf16":
        _store_bf16(s["k"], pid, slot, k)
        _store_bf16(s["v"], pid, slot, s["new_v"])
        return s["out"], s["k"], s["v"]
    first = table.gather(1, (prior // page)[:, None])[:, 0]
    off = prior % page
    _store_e4m3(s["k"], s["k_scale"], first, off, pid, slot, k)
    _store_e4m3(s["v"], s["v_scale"], first, off, pid, slot, s["new_v"].double())
    return s["out"], s["k"], s["v"], s["k_scale"], s["v_scale"]


def _gathered(pool, scale, table):
    """The sequences' keys or values, [B, KV, P * page, d] fp32 (pages past a sequence: page 0)."""
    ids = table.clamp(min=0).long()
    x = pool[ids].float()  # [B, P, KV, page, d]
    if scale is not None:
        x = x * torch.exp2(scale[ids].float() - 127)[..., None, None]
    B, P, KV, page, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, KV, P * page, d)


def _attend(c, q, k, v, lim):
    """Softmax attention of q [B, KV, R, d] over keys below lim [B, R] (0: none); (out, probs)."""
    x = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(c["d"]))
    if c["softcap"] > 0:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    j = torch.arange(k.shape[2], device=q.device)
    seen = j < lim[..., None]
    if c["window"] > 0:
        seen = seen & (j >= lim[..., None] - c["window"])
    x.masked_fill_(~seen[:, None], float("-inf"))
    top = x.amax(dim=-1, keepdim=True)
    x.sub_(torch.where(torch.isfinite(top), top, torch.zeros_like(top))).exp_()
    total = x.sum(dim=-1, keepdim=True)
    x.div_(torch.where(total > 0, total, torch.ones_like(total)))
    return torch.matmul(x, v), x


def _gated(o, gate):
    return o if gate is None else o * torch.sigmoid(gate.float())


def _plain_decode(s):
    c = s["case"]
    B, H, KV, d = c["B"], c["H"], c["KV"], c["d"]
    k = _gathered(s["k"], s["k_scale"], s["table"])
    v = _gathered(s["v"], s["v_scale"], s["table"])
    G = H // KV
    lim = s["lens"].long()[:, None].expand(B, G)
    o, p = _attend(c, s["q"].float().view(B, KV, G, d), k, v, lim)
    s["out"].copy_(_gated(o.reshape(B, H, d), s["gate"]))
    if s["probs"] is None:
        return (s["out"],)
    s["probs"].copy_(p.reshape(B, H, -1)[..., :s["probs"].shape[-1]])
    return s["out"], s["probs"]


def _plain_prefill(s):
    c = s["case"]
    B, H, KV, d = c["B"], c["H"], c["KV"], c["d"]
    G, N = H // KV, s["max_new"]
    cu, prior = s["cu"].long(), s["prior"].long()
    t = torch.arange(s["T"], device=cu.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[b]
    q = torch.zeros(B, N, H, d, device=cu.device)
    q[b, i] = s["q"].float()
    q = q.view(B, N, KV, G, d).permute(0, 2, 1, 3, 4).reshape(B, KV, N * G, d)
    lim = torch.zeros(B, N, dtype=torch.long, device=cu.device)
    lim[b, i] = prior[b] + i + 1
    k = _gathered(s["k"], s["k_scale"], s["table"])
    v = _gathered(s["v"], s["v_scale"], s["table"])
    o, _ = _attend(c, q, k, v, lim.repeat_interleave(G, dim=1))
    o = o.view(B, KV, N, G, d).permute(0, 2, 1, 3, 4).reshape(B, N, H, d)[b, i]
    s["out"].copy_(_gated(o, s["gate"]))
    return (s["out"],)


# ------------------------------------------------------------------- run ----

def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"append": _plain_append, "decode": _plain_decode, "prefill": _plain_prefill}[c["op"]](s)
    import causal_gqa_attention_rope_gb300 as na
    cache = na.PagedKVCache(s["k"], s["v"], s["table"], s["k_scale"], s["v_scale"])
    if c["op"] == "append":
        cfg = na.AttnConfig(c["H"], c["KV"], c["d"], rotary_dim=c["rd"], qk_norm=c["qk_norm"])
        rope = na.RopeConfig(base=c["base"], yarn=c["yarn"], factor=4.0, orig_max_pos=8192)
        na.na_rope_append_kv_paged(cfg, rope, s["cu"], s["prior"], s["q"], s["new_k"], s["new_v"],
                                   s["out"], cache, q_norm_w=s["qw"], k_norm_w=s["kw"],
                                   status=s["status"])
        if c["fmt"] == "bf16":
            return s["out"], s["k"], s["v"]
        return s["out"], s["k"], s["v"], s["k_scale"], s["v_scale"]
    cfg = na.AttnConfig(c["H"], c["KV"], c["d"], out_gate=c["gate"], softcap=c["softcap"],
                        window=c["window"])
    if c["op"] == "decode":
        na.na_attn_decode_paged(cfg, s["q"], cache, s["lens"], s["max_total"], s["out"],
                                probs=s["probs"], gate=s["gate"], workspace=s["workspace"],
                                status=s["status"])
        return (s["out"],) if s["probs"] is None else (s["out"], s["probs"])
    na.na_attn_prefill_chunk_paged(cfg, s["cu"], s["prior"], s["max_new"], s["max_total"], s["q"],
                                   cache, s["out"], gate=s["gate"], workspace=s["workspace"],
                                   status=s["status"])
    return (s["out"],)


# ----------------------------------------------------------------- exact ----

def exact(case, seed):
    """The definition in 64 bits, sequence by sequence, unrounded."""
    s = prepare(case, seed)
    return _exact_append(case, s) if case["op"] == "append" else _exact_attend(case, s)


def _spans(case):
    at = 0
    for b, (p, n) in enumerate(zip(*_lengths(case))):
        yield b, p, n, at
        at += n


def _exact_append(case, s):
    rd, page, d = case["rd"], case["page"], case["d"]
    dev = s["q"].device
    freq = []
    for i in range(rd // 2):
        f = case["base"] ** (-2.0 * i / rd)
        if case["yarn"]:
            edge = [rd * math.log(8192 / (r * 2 * math.pi)) / (2 * math.log(case["base"]))
                    for r in (32.0, 1.0)]
            lo = max(0, math.floor(edge[0]))
            hi = min(rd // 2 - 1, max(0, math.ceil(edge[1])))
            mix = min(1.0, max(0, i - lo) / max(1, hi - lo))
            f = f * (1 - mix) + f / 4.0 * mix
        freq.append(f)
    gain = 0.1 * math.log(4.0) + 1.0 if case["yarn"] else 1.0

    def turned(x, w, pos):
        """Pairs as complex numbers, turned by e^(i pos f)."""
        x = x.double()
        if w is not None:
            x = x * torch.rsqrt(x.square().sum(-1, keepdim=True) / d + 1e-6) * w.double()
        angle = pos[:, None].double() * torch.tensor(freq, dtype=torch.float64, device=dev)
        z = torch.complex(x[..., :rd // 2], x[..., rd // 2:rd])
        z = z * (gain * torch.polar(torch.ones_like(angle), angle))[:, None]
        return torch.cat((z.real, z.imag, x[..., rd:]), dim=-1)

    q = torch.empty(s["q"].shape, dtype=torch.float64, device=dev)
    pools = [s["k"].double(), s["v"].double()]
    scales = [None, None]
    if case["fmt"] == "e4m3":
        scales = [s["k_scale"].clone(), s["v_scale"].clone()]
    for b, p, n, at in _spans(case):
        pos = torch.arange(p, p + n, device=dev)
        q[at:at + n] = turned(s["q"][at:at + n], s["qw"], pos)
        for which, x in enumerate((turned(s["new_k"][at:at + n], s["kw"], pos),
                                   s["new_v"][at:at + n].double())):
            pool, scale = pools[which], scales[which]
            for pg in range(p // page, (p + n - 1) // page + 1):
                lo, hi = max(p, pg * page), min(p + n, (pg + 1) * page)
                pid = int(s["table"][b, pg])
                rows = x[lo - p:hi - p].transpose(0, 1)  # [KV, tokens, d]
                a, z = lo - pg * page, hi - pg * page
                if scale is not None:
                    need = torch.ceil(torch.log2(rows.abs().amax(dim=(1, 2)) / E4M3_MAX)).clamp(-127, 127)
                    if a > 0:
                        was = scale[pid].double() - 127
                        need = torch.maximum(need, was)
                        pool[pid, :, :a] *= torch.exp2(was - need)[:, None, None]
                    rows = rows / torch.exp2(need)[:, None, None]
                    scale[pid] = (need + 127).to(torch.uint8)
                pool[pid, :, a:z] = rows
    if case["fmt"] == "bf16":
        return q, pools[0], pools[1]
    return q, pools[0], pools[1], scales[0], scales[1]


def _exact_attend(case, s):
    H, KV, d, page = case["H"], case["KV"], case["d"], case["page"]
    G = H // KV
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    probs = None
    if case.get("probs"):
        probs = torch.zeros(s["probs"].shape, dtype=torch.float64, device=out.device)
    for b, p, n, at in _spans(case):
        ids = s["table"][b, :-(-(p + n) // page)].long()
        for g in range(KV):
            kv = []
            for pool, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
                x = pool[ids, g].double()
                if scale is not None:
                    x = x * (2.0 ** (scale[ids, g].double() - 127))[:, None, None]
                kv.append(x.reshape(-1, d)[:p + n])
            rows = s["q"][at:at + n, g * G:(g + 1) * G].double()  # [n, G, d]
            x = torch.einsum("ngd,kd->gnk", rows, kv[0]) / math.sqrt(d)
            if case["softcap"] > 0:
                x = torch.tanh(x / case["softcap"]) * case["softcap"]
            key = torch.arange(p + n, device=out.device)[None, :]
            own_pos = torch.arange(p, p + n, device=out.device)[:, None]
            hidden = key > own_pos
            if case["window"] > 0:
                hidden = hidden | (key <= own_pos - case["window"])
            w = torch.softmax(x.masked_fill(hidden, float("-inf")), dim=-1)
            out[at:at + n, g * G:(g + 1) * G] = torch.einsum("gnk,kd->ngd", w, kv[1])
            if probs is not None:
                probs[b, g * G:(g + 1) * G, :p + n] = w[:, 0]
    if s["gate"] is not None:
        out = out / (1 + torch.exp(-s["gate"].double()))
    return (out,) if probs is None else (out, probs)
