"""The bounds that the tensor-core prefill's outputs are held to, on the CPU: they hold for the roundings that the kernel
makes, and see one more, one of the wrong sign, and a NaN."""
import functools

import pytest
import torch

from delta_outputs import output_bounds, outputs, parts, unit_keys, within
from delta_plain import inputs

BF16 = torch.bfloat16


def case(kind, dk=128):
    x = inputs([140], 2, 1, dk, 64, BF16, seed=41, init=kind != "scores", device="cpu")
    if kind == "state":
        x["beta"].zero_()
    if kind == "scores":
        x = unit_keys(x, 140)
    return x


def hold(n, sign=1.0):
    return functools.partial(parts, n=n, sign=sign)


@pytest.mark.parametrize("kind", ["state", "scores", "all"])
def test_what_the_kernel_rounds_is_within(kind):
    x = case(kind)
    want, bound = output_bounds(x, [140], 0.5 if kind == "all" else 1.0, exact_scores=kind == "scores")
    got, of_s, of_p = outputs(x, [140], 0.5 if kind == "all" else 1.0, hold(2), hold(2), hold(1))
    assert within(got, want, bound)
    assert (kind == "state") == (not bool(of_p.any()))
    if kind == "scores":                                  # nothing of P is rounded
        assert torch.equal(got, outputs(x, [140], 1.0, hold(2), hold(2))[0])


@pytest.mark.parametrize("kind,s,u", [("state", hold(1), None), ("state", hold(2, -1.0), None),
                                      ("scores", None, hold(1)), ("scores", None, hold(2, -1.0))])
def test_a_lost_part_is_seen(kind, s, u):
    """One part of the state or of u in place of two, or the second with the wrong sign."""
    x = case(kind)
    want, bound = output_bounds(x, [140], exact_scores=kind == "scores")
    assert not within(outputs(x, [140], 1.0, s, u)[0], want, bound)


def test_a_nan_is_seen():
    x = case("all")
    want, bound = output_bounds(x, [140])
    got = want.clone()
    assert within(got, want, bound)
    got[77, 1, 5] = float("nan")
    assert not within(got, want, bound)
