"""Latent attention in 64 bits, on the host, and pages of latent rows for the tests.

Pages that no sequence owns and slots past a sequence's tokens hold NaN bits;
page-table entries past a sequence are -1.
"""
from __future__ import annotations

import torch

from paged_ref import NAN_BF16, inv_freq


def nan_bf16(*shape):
    return torch.full(shape, NAN_BF16, dtype=torch.int16).view(torch.bfloat16)


def make_latent(lens, wide, page, seed, room=0, spare=3, mag=1.0):
    """(pages [n, page, wide], table): lens[b] tokens ~ mag N(0, 1) in scattered pages, with pages for
    `room` more tokens each."""
    g = torch.Generator().manual_seed(seed)
    per = [max(1, -(-(n + room) // page)) for n in lens]
    ids = torch.randperm(sum(per) + spare, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(per)), -1, dtype=torch.int32)
    pool, at = nan_bf16(len(ids), page, wide), 0
    for b, n in enumerate(per):
        table[b, :n] = ids[at:at + n]
        at += n
        x = (torch.randn(lens[b], wide, generator=g) * mag).to(torch.bfloat16)
        for i in range(-(-lens[b] // page)):
            part = x[i * page:(i + 1) * page]
            pool[int(table[b, i]), :len(part)] = part
    return pool, table


def rows_of(pool, table, b, n):
    page = pool.shape[1]
    return pool[table[b, :-(-n // page)].long()].flatten(0, 1)[:n]


def turn(x, pos, rope, interleaved):
    """fp64 x [T, ..., rd] turned by pos [T]."""
    rd = x.shape[-1]
    f, factor = inv_freq(rope, rd)
    a = (pos.double()[:, None] * f).view(len(pos), *([1] * (x.dim() - 2)), rd // 2)
    c, s = torch.cos(a) * factor, torch.sin(a) * factor
    x = x.double()
    if interleaved:
        x0, x1 = x[..., 0::2], x[..., 1::2]
        return torch.stack([x0 * c - x1 * s, x0 * s + x1 * c], dim=-1).flatten(-2)
    x0, x1 = x[..., :rd // 2], x[..., rd // 2:]
    return torch.cat([x0 * c - x1 * s, x0 * s + x1 * c], dim=-1)


def attend(q, k, v, lim, scale):
    """q [n, H, d], k [H or 1, keys, d], v [H or 1, keys, dv], lim [n] keys that each row sees:
    (out, tolerance) [n, H, dv] in fp64.

    The tolerance counts the kernels' roundings: the output's to bf16, 2^-8 |o|; the weights' to
    bf16, 2^-8 A with A = sum p |v|; the scores', d products summed in fp32 in any order,
    eps = (d + 8) 2^-24 S with S the largest scale sum |q k| of the row, an error of the weight's
    exponent that enters numerator and sum: 2 eps A; and 2^-16 A for exp2 on the special function
    unit, the sums and a merge of pieces."""
    q, k, v = q.double(), k.double(), v.double()
    n, H, d = q.shape
    k, v = k.expand(H, -1, -1), v.expand(H, -1, -1)
    s = torch.einsum("nhd,hkd->nhk", q, k) * scale
    big = torch.einsum("nhd,hkd->nhk", q.abs(), k.abs()) * scale
    hidden = torch.arange(k.shape[1]) >= lim[:, None]
    s = s.masked_fill(hidden[:, None], float("-inf"))
    big = big.masked_fill(hidden[:, None], 0.0).amax(-1, keepdim=True) if k.shape[1] else s.sum(-1, keepdim=True)
    p = torch.nan_to_num(torch.softmax(s, dim=-1), nan=0.0)  # a row that sees nothing: zeros
    o = torch.einsum("nhk,hkd->nhd", p, v)
    a = torch.einsum("nhk,hkd->nhd", p, v.abs())
    eps = (d + 8) * 2.0 ** -24 * big
    return o, 2.0 ** -8 * o.abs() + a * (2.0 ** -8 + 2 * eps + 2.0 ** -16)
