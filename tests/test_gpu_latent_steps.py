"""Absorbed latent attention as a server's steps meet it: loose bounds, one workspace for steps of many
sizes, many rows, the same step again."""
import pytest
import torch

from latent_ref import make_latent
from paged_ref import bits
from test_gpu_latent import absorbed, check_absorbed, randn

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("H,R,rd,most", [(32, 512, 64, 4), (16, 256, 64, 8), (40, 128, 32, 100)])
def test_a_bound_above_the_call_s_tokens(H, R, rd, most):
    """The workspace that the query names for the same arguments is enough."""
    check_absorbed(H, R, rd, 64, [8000, 10], [1, 1], bounds=(most, 8064))


@pytest.mark.parametrize("R,rd", [(512, 64), (128, 32)])
def test_one_workspace_for_steps_of_many_sizes(R, rd):
    """Sized for the largest step, dirty with what the step before left in it."""
    import causal_gqa_attention_rope_gb300 as na
    H, prior = 32, [4000, 70, 900]
    cfg = na.LatentConfig(H, R, rd)
    pool, table = make_latent([n + 8 for n in prior], R + rd, 32, 21)
    need = na.na_latent_paged_workspace_size(cfg, 3, 24, 8, 4008)
    shared = na.workspace(need, DEV)
    for step, new in enumerate(([8, 8, 8], [1, 1, 1], [2, 0, 3], [0, 1, 0])):
        q = randn(22 + step, sum(new), H, R + rd)
        alone, status = absorbed(cfg, pool, table, prior, new, q)
        assert status == 0
        got, status = absorbed(cfg, pool, table, prior, new, q, workspace=shared)
        assert status == 0 and torch.equal(bits(got), bits(alone))


@pytest.mark.parametrize("R,H,new", [(512, 32, 8), (512, 128, 1), (256, 40, 5), (128, 32, 8)])
def test_many_rows_again_and_again(R, H, new):
    """Units of two CTAs: the same bits from every call, next to the 64-bit statement once."""
    import causal_gqa_attention_rope_gb300 as na
    prior = [3000, 129, 1, 6000, 64, 777]
    check_absorbed(H, R, 64, 64, prior, [new] * 6, seed=31)
    cfg = na.LatentConfig(H, R, 64)
    pool, table = make_latent([n + new for n in prior], R + 64, 64, 32)
    q = randn(33, 6 * new, H, R + 64)
    first, status = absorbed(cfg, pool, table, prior, [new] * 6, q)
    assert status == 0
    for _ in range(20):
        got, status = absorbed(cfg, pool, table, prior, [new] * 6, q)
        assert status == 0 and torch.equal(bits(got), bits(first))
