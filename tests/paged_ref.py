"""Paged caches for the tests, and the paged operators in 64 bits.

The pages of a test cache that no sequence owns, and the slots past a
sequence's tokens, hold NaN bit patterns (bf16 0x7FC1, E4M3 0x7F) and their
scale bytes 255 (E8M0's NaN); page-table entries past a sequence are -1.
"""
from __future__ import annotations

import math
from dataclasses import dataclass
from typing import List, Optional

import torch

NAN_BF16, NAN_E4M3, NAN_SCALE = 0x7FC1, 0x7F, 255


@dataclass
class Paged:
    """Host tensors of a paged cache."""
    k: torch.Tensor
    v: torch.Tensor
    table: torch.Tensor
    k_scale: Optional[torch.Tensor]
    v_scale: Optional[torch.Tensor]

    @property
    def page(self):
        return int(self.k.shape[2])

    def to(self, device):
        import causal_gqa_attention_rope_gb300 as na
        mv = lambda t: None if t is None else t.to(device)  # noqa: E731
        return na.PagedKVCache(mv(self.k), mv(self.v), mv(self.table), mv(self.k_scale),
                               mv(self.v_scale))

    @staticmethod
    def back(cache):
        mv = lambda t: None if t is None else t.cpu()  # noqa: E731
        return Paged(mv(cache.k), mv(cache.v), mv(cache.page_table), mv(cache.k_scale),
                     mv(cache.v_scale))


def bits(t: torch.Tensor) -> torch.Tensor:
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.uint8)


def exponent(amax: torch.Tensor) -> torch.Tensor:
    """Smallest e with amax <= 448 2^e, within E8M0's range; -127 for 0 (fp64 amax)."""
    e = torch.ceil(torch.log2(amax.double() / 448.0))
    return torch.where(amax > 0, e.clamp(-127, 127), torch.full_like(e, -127.0))


def make_paged(lens: List[int], KV: int, d: int, page: int, fmt: str, seed: int, spare: int = 3,
               room: int = 0, mag: float = 1.0, spread: float = 1.0) -> Paged:
    """Sequence b holds lens[b] tokens ~ mag * N(0, 1), every (page, head) times
    2^(spread * N(0, 1)), in pages scattered over the pool; the table has room
    for `room` more tokens each (their pages assigned too)."""
    g = torch.Generator().manual_seed(seed)
    per = [max(1, -(-(n + room) // page)) for n in lens]
    P, n_pages = max(per), sum(per) + spare
    ids = torch.randperm(n_pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), P), -1, dtype=torch.int32)
    at = 0
    out = []
    for b, n in enumerate(per):
        table[b, :n] = ids[at:at + n]
        at += n
    for _ in range(2):
        if fmt == "bf16":
            pool = torch.full((n_pages, KV, page, d), NAN_BF16, dtype=torch.int16).view(torch.bfloat16)
            scale = None
        else:
            pool = torch.full((n_pages, KV, page, d), NAN_E4M3, dtype=torch.uint8).view(torch.float8_e4m3fn)
            scale = torch.full((n_pages, KV), NAN_SCALE, dtype=torch.uint8)
        for b, n in enumerate(lens):
            for i in range(-(-n // page)):
                m = min(page, n - i * page)
                x = torch.randn(KV, m, d, generator=g) * mag
                x *= torch.exp2(spread * torch.randn(KV, 1, 1, generator=g))
                pid = int(table[b, i])
                if fmt == "bf16":
                    pool[pid, :, :m] = x.to(torch.bfloat16)
                else:
                    e = exponent(x.abs().amax(dim=(1, 2)))
                    q = (x.double() / torch.exp2(e)[:, None, None]).float().to(torch.float8_e4m3fn)
                    u = pool.view(torch.uint8)
                    u[pid, :, :m] = q.view(torch.uint8)
                    scale[pid] = (e + 127).to(torch.uint8)
        out.append((pool, scale))
    return Paged(out[0][0], out[1][0], table, out[0][1], out[1][1])


def values(pool, scale, ids) -> torch.Tensor:
    """fp64 values of pages `ids`, as [KV, tokens, d]."""
    x = pool[ids.long()] if scale is None else pool.view(torch.uint8)[ids.long()].view(pool.dtype)
    x = x.double()
    if scale is not None:
        x = x * torch.exp2(scale[ids.long()].double() - 127)[..., None, None]
    return x.permute(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3])


@dataclass
class Rows:
    out: torch.Tensor     # [T, H, d] fp64
    tol: torch.Tensor     # [T, H, d] how far a kernel may be off (see attend)
    probs: list           # per token [H, keys] fp64
    probs_tol: list


def attend(c: Paged, q: torch.Tensor, spans, scale=None, softcap=0.0, window=0, gate=None) -> Rows:
    """spans: per sequence (first token row, cached tokens before it, new tokens).

    Tolerance, from the roundings of the kernels (bf16 rounds by at most 2^-8 of
    the value, fp32 by 2^-24): the output's own rounding, 2^-8 |o|; the
    probabilities' to bf16, 2^-8 A with A = sum p |v|; and the scores', summed in
    fp32 over d terms in any order, (d + 8) 2^-24 S with S the largest
    scale * sum |q k| of the row, which is a relative error of p, entering
    numerator and sum: 2 (d + 8) 2^-24 S A.  exp2 and the sigmoid on the special
    function unit, the sum of p and the merge: 2^-16 A.  The soft cap's tanh adds
    an absolute 2^-19 cap to a score.  Over E4M3 pages the chunk call takes a query
    as the sum of two E4M3 numbers per element: exact, or below 2^-10 of the row's
    largest within 2^-17 of that, which adds 2^-17 max|q| scale sum |k| to a score;
    and V values with a scale below 2^-40 are multiples of 2^-64 (2^-65 of output).
    The weights' rounding to f16 there is finer than bf16's."""
    T, H, d = q.shape
    KV = c.k.shape[1]
    G = H // KV
    sc = 1.0 / math.sqrt(d) if scale is None else scale
    out = torch.zeros(T, H, d, dtype=torch.float64)
    tol = torch.zeros(T, H, d, dtype=torch.float64)
    probs, probs_tol = [None] * T, [None] * T
    for b, (row, prior, new) in enumerate(spans):
        total = prior + new
        if new == 0 or total == 0:
            continue
        first_page = 0 if window == 0 else max(0, prior - window + 1) // c.page
        ids = c.table[b, first_page:-(-total // c.page)]
        base = first_page * c.page
        kk = values(c.k, c.k_scale, ids)[:, :total - base]
        vv = values(c.v, c.v_scale, ids)[:, :total - base]
        for i in range(new):
            pos = prior + i
            lo = max(0, pos - window + 1) if window > 0 else 0
            k1, v1 = kk[:, lo - base:pos + 1 - base], vv[:, lo - base:pos + 1 - base]
            qi = q[row + i].double().view(KV, G, d)
            s = torch.einsum("kgd,knd->kgn", qi, k1) * sc
            eps = (d + 8) * 2.0 ** -24 * sc * torch.einsum("kgd,knd->kgn", qi.abs(), k1.abs()).amax(-1)
            if c.k_scale is not None:
                eps = eps + 2.0 ** -17 * sc * qi.abs().amax(-1) * k1.abs().sum(-1).amax(-1)[:, None]
            if softcap > 0:
                s = softcap * torch.tanh(s / softcap)
                eps = eps + 2.0 ** -19 * softcap
            p = torch.softmax(s, dim=-1)
            o = torch.einsum("kgn,knd->kgd", p, v1)
            a = torch.einsum("kgn,knd->kgd", p, v1.abs())
            rel = (2 * eps + 2.0 ** -16)[..., None]
            t = 2.0 ** -8 * o.abs() + a * (2.0 ** -8 + rel)
            if c.v_scale is not None:
                t = t + 2.0 ** -65
            if gate is not None:
                g = torch.sigmoid(gate[row + i].double()).view(KV, G, d)
                o, t = o * g, t * g
            out[row + i], tol[row + i] = o.reshape(H, d), t.reshape(H, d)
            pr = torch.zeros(H, pos + 1, dtype=torch.float64)
            pr[:, lo:] = p.reshape(H, -1)
            probs[row + i] = pr
            probs_tol[row + i] = pr * rel.reshape(H, 1) + 2.0 ** -120
    return Rows(out, tol, probs, probs_tol)


def inv_freq(rope, rd) -> tuple:
    """fp64 frequencies and the factor on cos and sin, for a RopeConfig."""
    i = torch.arange(rd // 2, dtype=torch.float64)
    f = rope.base ** (-2.0 * i / rd)
    if not rope.yarn:
        return f, rope.attn_factor if rope.attn_factor > 0 else 1.0

    def dim_at(rot):
        return rd * math.log(rope.orig_max_pos / (rot * 2 * math.pi)) / (2 * math.log(rope.base))
    low = max(math.floor(dim_at(rope.beta_fast)), 0)
    high = min(max(math.ceil(dim_at(rope.beta_slow)), 0), max(rd // 2 - 1, 0))
    ramp = ((i - low).clamp(min=0) / max(high - low, 1)).clamp(max=1)
    factor = rope.attn_factor if rope.attn_factor > 0 else (
        0.1 * math.log(rope.factor) + 1.0 if rope.factor > 1 else 1.0)
    return f * (1 - ramp) + f / rope.factor * ramp, factor


def normed_rotated(x, pos, rope, rd, w=None, eps=1e-6, zero_centered=False):
    """RMS norm (with weights w) and rotation of x [T, heads, d] at pos [T], fp64."""
    x = x.double()
    if w is not None:
        ww = w.double() + 1 if zero_centered else w.double()
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * ww
    f, factor = inv_freq(rope, rd)
    a = (pos.double()[:, None] * f)[:, None, :]
    c, s = torch.cos(a) * factor, torch.sin(a) * factor
    h = rd // 2
    return torch.cat([x[..., :h] * c - x[..., h:rd] * s, x[..., :h] * s + x[..., h:rd] * c,
                      x[..., rd:]], dim=-1)


def v_normed(x, eps):
    x = x.double()
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
