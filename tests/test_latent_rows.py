"""Rows of tensors with dimensions of size 1, whose strides say nothing (no GPU needed)."""
import pytest
import torch

import causal_gqa_attention_rope_gb300 as na


class Device(torch.Tensor):
    """A host tensor that says it is on a GPU."""
    is_cuda = property(lambda self: True)


def wide(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16).as_subclass(Device)


@pytest.mark.parametrize("view,stride", [
    (lambda: wide(5, 192)[:, 128:].unsqueeze(1), 192),                # one head of wider rows
    (lambda: wide(5, 1, 192)[..., 128:], 192),
    (lambda: wide(5, 4, 192)[..., 128:], 192),
    (lambda: wide(1, 4, 192)[..., 128:], 192),                        # one token
    (lambda: wide(4, 192)[:, 128:].unsqueeze(0), 192),
    (lambda: wide(4, 3, 192)[:1].transpose(0, 1)[:, :, 128:], 192),   # [3, 1, 64], odd strides between
    (lambda: wide(1, 1, 64), 64),
    (lambda: wide(64, 1).t().unsqueeze(0), 64),                       # a row whose own stride is 1
    (lambda: wide(64).as_strided((1, 64), (0, 1)), 64),               # or 0
    (lambda: wide(7, 100)[::3, 20:84], 300),
])
def test_their_distance(view, stride):
    t = view()
    pointer, got = na._rows(t, "x", 64)
    assert (pointer, got) == (t.data_ptr(), stride)


@pytest.mark.parametrize("view", [
    lambda: wide(5, 4, 192).transpose(0, 1)[..., 128:],   # heads are not one behind the other
    lambda: wide(5, 8, 192)[:, :4, 128:],
    lambda: wide(5, 128)[:, ::2],
])
def test_rows_that_are_not_equally_far_apart(view):
    with pytest.raises(ValueError, match="equally far apart"):
        na._rows(view(), "x", 64)
