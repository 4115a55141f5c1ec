"""Latent calls over rows of size-1 dimensions: through the compiled calls and through Python's checks."""
import types

import pytest
import torch

from latent_ref import make_latent, nan_bf16
from paged_ref import bits
from test_gpu_latent import DEV, ints, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["compiled", "python"])
def way(request, monkeypatch):
    """Both ways of a call: the compiled one has to take it itself, or declines all."""
    import causal_gqa_attention_rope_gb300 as na
    real = na._calls()

    def taken(f):
        def call(*a):
            rc = f(*a)
            assert rc is not None
            return rc
        return call

    names = ("latent_append", "expanded")
    calls = {n: taken(getattr(real, n)) if request.param == "compiled" else lambda *a: None for n in names}
    monkeypatch.setattr(na, "_native", types.SimpleNamespace(**calls))


def append(cfg, T, kv, q, out):
    import causal_gqa_attention_rope_gb300 as na
    pool, table = make_latent([20], cfg.kv_rank + cfg.rope_dim, 16, 1, room=T)
    cache, status = na.PagedLatentCache(pool.to(DEV), table.to(DEV)), ints([0])
    na.na_latent_append_paged(cfg, na.RopeConfig(), ints([0, T]), ints([20]), kv, q, out, cache, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return bits(cache.kv.cpu()), bits(out.cpu().contiguous())


@pytest.mark.parametrize("T", [1, 5])
def test_append_of_one_head(way, T):
    import causal_gqa_attention_rope_gb300 as na
    cfg = na.LatentConfig(1, 128, 64, kv_norm=False)
    kv, wide = randn(1, T, 192).to(DEV), randn(2, T, 192).to(DEV)
    want = append(cfg, T, kv, wide[:, 128:].unsqueeze(1).contiguous(), nan_bf16(T, 1, 64).to(DEV))
    rows = torch.full((T, 256), 3.0, dtype=torch.bfloat16, device=DEV)
    got = append(cfg, T, kv, wide[:, 128:].unsqueeze(1), rows[:, 64:128].unsqueeze(1))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert (rows[:, :64] == 3.0).all() and (rows[:, 128:] == 3.0).all()


def test_append_of_one_token(way):
    """Rows whose stride is 0 or 1: there is no second one."""
    import causal_gqa_attention_rope_gb300 as na
    cfg = na.LatentConfig(4, 128, 64, kv_norm=False)
    kv, q = randn(1, 1, 192).to(DEV), randn(2, 1, 4, 64).to(DEV)
    want = append(cfg, 1, kv, q, nan_bf16(1, 4, 64).to(DEV))
    for row in (kv.as_strided((1, 192), (0, 1)), kv.as_strided((1, 192), (1, 1))):
        assert row.stride(0) < 192
        got = append(cfg, 1, row, q, nan_bf16(1, 4, 64).to(DEV))
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_expanded_over_one_key(way):
    import causal_gqa_attention_rope_gb300 as na
    cfg = na.LatentConfig(3, 128, 64, 64, 64)
    q, kv, pe = randn(1, 1, 3, 128).to(DEV), randn(2, 1, 3, 128).to(DEV), randn(3, 64).to(DEV)
    for rows in (pe.as_strided((1, 64), (0, 1)), pe.as_strided((1, 64), (1, 1))):
        out = nan_bf16(1, 3, 64).to(DEV)
        na.na_attn_latent_expanded(cfg, ints([0, 1]), ints([0]), ints([1]), 1, 1, q, kv, rows, out)
        torch.cuda.synchronize()
        assert torch.equal(bits(out.cpu()), bits(kv[..., 64:].cpu().contiguous()))
