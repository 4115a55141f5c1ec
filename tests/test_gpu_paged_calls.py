"""The compiled route of the three paged calls (csrc/paged_calls.cpp): it takes the plain
call, leaves anything else to the Python checks, and both give the same bits."""
import os
import re

import pytest
import torch

import causal_gqa_attention_rope_gb300 as na
from paged_ref import bits, make_paged

pytestmark = pytest.mark.gpu
DEV = "cuda"
H, KV, D, PAGE = 4, 2, 64, 16


class Spy:
    """na's compiled calls, their answers noted; `off` answers None for all of them."""
    def __init__(self, calls, off=False):
        self.calls, self.off, self.answers = calls, off, []

    def __getattr__(self, name):
        def call(*args):
            got = None if self.off else getattr(self.calls, name)(*args)
            self.answers.append(got)
            return got
        return call


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def steps(fmt, **change):
    """One append, chunk call and decode call on the same data; their outputs."""
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    prior, new = [5, 30], [3, 4]
    cache = make_paged(prior, KV, D, PAGE, fmt, 3, room=4).to(DEV)
    cache = na.PagedKVCache(cache.k, cache.v, cache.page_table, cache.k_scale, cache.v_scale)
    a = dict(rope=na.RopeConfig(base=1e4), cu=ints([0, 3, 7]), prior=ints(prior), q=rnd(7, H, D),
             k=rnd(7, KV, D), v=rnd(7, KV, D), qw=rnd(D), kw=rnd(D), gate=rnd(7, H, D),
             max_new=4, max_total=34, lens=ints([8, 34]), status=ints([0]),
             ws=na.workspace(1 << 20, DEV), probs=torch.zeros(2, H, 40, device=DEV),
             q1=rnd(2, H, D), gate1=rnd(2, H, D), total=None, splits=0, stream=None, cache=cache)
    a["cfg"] = na.AttnConfig(H, KV, D, qk_norm=True, out_gate=True)
    a.update({n: f(a) for n, f in change.items()})
    cache = a["cache"]
    q_out, out = torch.zeros(7, H, D, dtype=torch.bfloat16, device=DEV), rnd(7, H, D)
    out1 = rnd(2, H, D)
    na.na_rope_append_kv_paged(a["cfg"], a["rope"], a["cu"], a["prior"], a["q"], a["k"], a["v"],
                               q_out, cache, q_norm_w=a["qw"], k_norm_w=a["kw"],
                               status=a["status"], total_tokens=a["total"], stream=a["stream"])
    na.na_attn_prefill_chunk_paged(a["cfg"], a["cu"], a["prior"], a["max_new"], a["max_total"],
                                   q_out, cache, out, gate=a["gate"], workspace=a["ws"],
                                   status=a["status"], total_tokens=a["total"],
                                   stream=a["stream"])
    na.na_attn_decode_paged(a["cfg"], a["q1"], cache, a["lens"], a["max_total"], out1,
                            probs=a["probs"], gate=a["gate1"], workspace=a["ws"],
                            num_splits=a["splits"], status=a["status"], stream=a["stream"])
    torch.cuda.synchronize()
    assert int(a["status"].item()) == 0
    return [bits(t.cpu()) for t in (q_out, out, out1, cache.k, cache.v)] + [a["probs"].cpu()]


def spied(monkeypatch, off=False):
    spy = Spy(na._calls(), off)
    monkeypatch.setattr(na, "_native", spy)
    return spy


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_both_routes_give_the_same_bits(fmt, monkeypatch):
    want = steps(fmt)
    spy = spied(monkeypatch)
    got = steps(fmt)
    assert spy.answers == [na.NA_OK] * 3
    spy = spied(monkeypatch, off=True)
    slow = steps(fmt)
    assert spy.answers == [None] * 3
    for a, b, c in zip(want, got, slow):
        assert torch.equal(a, b) and torch.equal(a, c)


class Number:
    """An integer of another kind."""
    def __init__(self, x):
        self.x = x

    def __index__(self):
        return self.x

    __int__ = __index__


class Config(na.AttnConfig):
    pass


UNUSUAL = [
    dict(cfg=lambda a: Config(H, KV, D, qk_norm=True, out_gate=True)),
    dict(cfg=lambda a: na.AttnConfig(H, KV, D, qk_norm=1, out_gate=1)),
    dict(max_total=lambda a: Number(34), total=lambda a: Number(7)),
]


@pytest.mark.parametrize("change", UNUSUAL, ids=["subclass", "flags", "integers"])
def test_unusual_arguments_take_the_other_route(change, monkeypatch):
    want = steps("e4m3")
    spy = spied(monkeypatch)
    got = steps("e4m3", **change)
    assert None in spy.answers
    for a, b in zip(want, got):
        assert torch.equal(a, b)


PLAIN = [
    dict(total=lambda a: 7),
    dict(q=lambda a: torch.cat([a["q"], a["q"]])[:9], gate=lambda a: torch.cat([a["gate"]] * 2),
         total=lambda a: 7),  # more rows than the call reads
    dict(prior=lambda a: ints([5, 30, 99])),  # and more sequences
    dict(cache=lambda a: na.PagedKVCache(a["cache"].k, a["cache"].v,
                                         torch.cat([a["cache"].page_table] * 2),
                                         a["cache"].k_scale, a["cache"].v_scale)),
    dict(qw=lambda a: torch.nn.Parameter(a["qw"])),
    dict(stream=lambda a: torch.cuda.current_stream()),
    dict(cfg=lambda a: na.AttnConfig(H, KV, D, rotary_dim=D, sm_scale=D ** -0.5, qk_norm=True,
                                     out_gate=True, window=0, softcap=0)),
]


@pytest.mark.parametrize("change", PLAIN, ids=["total", "rows", "lens", "table", "parameter",
                                               "stream", "spelt"])
def test_what_the_compiled_route_takes(change, monkeypatch):
    want = steps("e4m3")
    spy = spied(monkeypatch)
    got = steps("e4m3", **change)
    assert spy.answers == [na.NA_OK] * 3
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def strided(t):
    return torch.stack([t, t], dim=-1)[..., 0]


BAD = [
    (dict(q=lambda a: strided(a["q"])), "contiguous"),
    (dict(q=lambda a: a["q"].float()), "q"),
    (dict(q=lambda a: a["q"][:6], total=lambda a: 7), "q"),
    (dict(k=lambda a: a["k"][:, :1].contiguous()), "k"),
    (dict(v=lambda a: a["v"].half()), "v"),
    (dict(qw=lambda a: a["qw"][:8]), "q_norm_w"),
    (dict(kw=lambda a: torch.cat([a["kw"]] * 2)), "k_norm_w"),
    (dict(gate=lambda a: a["gate"][:6]), "gate"),
    (dict(gate1=lambda a: a["gate"][:3]), "gate"),
    (dict(probs=lambda a: torch.zeros(3, H, 40, device=DEV)), "probs"),
    (dict(probs=lambda a: strided(a["probs"])), "contiguous"),
    (dict(lens=lambda a: ints([8])), "kv_lens"),
    (dict(lens=lambda a: a["lens"].long()), "kv_lens"),
    (dict(prior=lambda a: ints([5])), "cache_lens"),
    (dict(cu=lambda a: a["cu"].long()), "cu_seqlens"),
    (dict(status=lambda a: a["status"].long()), "status"),
    (dict(ws=lambda a: strided(a["ws"])), "contiguous"),
    (dict(ws=lambda a: a["ws"].cpu()), "CUDA"),
    (dict(lens=lambda a: a["lens"].cpu()), "CUDA"),
    (dict(cache=lambda a: na.PagedKVCache(a["cache"].k, a["cache"].v[:1], a["cache"].page_table,
                                          a["cache"].k_scale, a["cache"].v_scale)), "cache.v"),
    (dict(cache=lambda a: na.PagedKVCache(a["cache"].k, torch.cat([a["cache"].v.view(torch.uint8)] * 2)
                                          .view(torch.float8_e4m3fn), a["cache"].page_table,
                                          a["cache"].k_scale, a["cache"].v_scale)), "cache.v"),
    (dict(cache=lambda a: na.PagedKVCache(a["cache"].k, a["cache"].v, a["cache"].page_table,
                                          a["cache"].k_scale[:1], a["cache"].v_scale)), "k_scale"),
    (dict(cache=lambda a: na.PagedKVCache(a["cache"].k, a["cache"].v, a["cache"].page_table[:1],
                                          a["cache"].k_scale, a["cache"].v_scale)), "page_table"),
    (dict(cache=lambda a: na.PagedKVCache(a["cache"].k, a["cache"].v, a["cache"].page_table,
                                          None, a["cache"].v_scale)), "k_scale"),
]


@pytest.mark.parametrize("change,word", BAD, ids=lambda x: x if isinstance(x, str) else "-".join(x))
def test_what_is_refused(change, word):
    with pytest.raises(ValueError, match=word):
        steps("e4m3", **change)


def test_the_library_refuses_through_the_compiled_route(monkeypatch):
    spy = spied(monkeypatch)
    with pytest.raises(na.NAError) as e:
        steps("bf16", max_total=lambda a: 10 ** 6)  # past the table
    assert e.value.code == na.NA_ERR_CAPACITY and spy.answers == [na.NA_OK, na.NA_ERR_CAPACITY]


def test_readme_examples_run():
    """The README's examples one after the other, the contiguous cache and the paged one."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
    with open(path) as fh:
        blocks = re.findall(r"```python\n(.*?)```", fh.read(), re.S)
    assert len(blocks) == 2
    names = {}
    for block in blocks:
        exec(block, names)
    torch.cuda.synchronize()
    assert int(names["status"].item()) == 0
    for out in (names["out"], names["out1"]):
        assert torch.isfinite(out.float()).all() and out.abs().max() > 0
    total = names["probs"][0, :, :129].double().sum(-1)
    assert (total - 1).abs().max() < 129 * 2.0 ** -16
