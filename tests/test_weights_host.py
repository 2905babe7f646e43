"""The cases that show the weights' rounding beside a 4-bit cache, without a GPU: they tell weights in two
bf16 parts from weights in one."""
import pytest
import torch

from tests import _weights as W


def one(w):
    return w.bfloat16().double()


def two(w):
    return one(w) + one(w - one(w))


@pytest.mark.parametrize("case", W.CASES)
def test_two_parts_pass_and_one_does_not(case):
    p = W.Problem(*case, seed=1, device="cpu")
    want, tol = p.attend(lambda w: w)
    assert torch.equal(p.v64.bfloat16().double(), p.v64)
    assert ((p.attend(two)[0].bfloat16().double() - want).abs() <= tol).all()
    over = (p.attend(one)[0].bfloat16().double() - want).abs() > tol
    assert over.double().mean() > 0.01, over.double().mean()
