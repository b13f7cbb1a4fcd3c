"""The oracle's gradient of a routing against 60 decimal digits, where its terms cancel or lie far from 1."""
from decimal import Decimal, getcontext

import numpy as np
import pytest

from oracle import int8_oracle as O

getcontext().prec = 60


def sigmoid(x):
    return 1 / (1 + (-Decimal(float(x))).exp())


def gradient(x, ids, d, scoring, renormalize, scale):
    """Of one token, as sums over pairs; 60 digits leave what cancels."""
    x, d, scale = [Decimal(float(v)) for v in x], [Decimal(float(v)) for v in d], Decimal(float(scale))
    if scoring == "sigmoid":
        s = [sigmoid(v) for v in x]
        ds = [v * (1 - v) for v in s]
    else:
        top = max(x)
        e = [(v - top).exp() for v in x]
        s = [v / sum(e) for v in e]
    total = sum(s[i] for i in ids)
    out = []
    for i in range(len(x)):
        v = Decimal(0)
        for c, j in enumerate(ids):  # dw_c / dx_i
            if scoring == "sigmoid":
                if renormalize:
                    v += d[c] * ds[i] * ((j == i) * total - ids.count(i) * s[j]) / total ** 2
                else:
                    v += d[c] * ds[i] * (j == i)
            elif renormalize:
                v += d[c] * s[j] / total * ((j == i) - ids.count(i) * s[i] / total)
            else:
                v += d[c] * s[j] * ((j == i) - s[i])
        out.append(float(scale * v))
    return np.array(out)


@pytest.mark.parametrize("renormalize", [True, False])
def test_oracle_gradient_of_far_sigmoid_logits(renormalize):
    """Within a few 2^-53 of every sum's terms; values 0.6 or more of their size away from their mean."""
    g = np.random.default_rng(51)
    x = g.uniform(25, 80, (6, 9)) * (1.0 if renormalize else np.where(np.arange(6)[:, None] < 2, -1.0, 1.0))
    e = np.stack([g.permutation(9)[:4] for _ in range(6)])
    d = np.array([[1.0, -2.0, 4.0, -8.0]]) * (1 + g.random((6, 1)))
    got = O.route_backward(x, e, d, "sigmoid", renormalize, 1.5)
    for t in range(6):
        np.testing.assert_allclose(got[t], gradient(x[t], e[t].tolist(), d[t], "sigmoid", renormalize, 1.5), rtol=1e-13, atol=0)


def test_oracle_gradient_of_the_smallest_sigmoid_scores():
    g = np.random.default_rng(52)
    x, d = g.uniform(-696, -695, 5), np.array([1e20, -2e20, 4e20, -8e20])
    got = O.route_backward(x[None], np.array([[0, 2, 3, 4]]), d[None], "sigmoid", True, 1.5)
    # (the exponential of a number of this size is off by 2^-53 of it, relative)
    np.testing.assert_allclose(got[0], gradient(x, [0, 2, 3, 4], d, "sigmoid", True, 1.5), rtol=1e-12, atol=0)


@pytest.mark.parametrize("scoring,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True)])
def test_oracle_gradient_beside_a_weight_of_nearly_one(scoring, renormalize):
    """One logit 25 .. 60 above all others, with the largest of the positive values: no sum of shares cancels."""
    g = np.random.default_rng(53)
    for t in range(6):
        x, ids, d = -g.uniform(25, 60, 12), g.permutation(12)[:5], g.uniform(0.1, 1.0, 5)
        x[ids[t % 5]], d[t % 5] = g.normal(), 2.0
        got = O.route_backward(x[None], ids[None], d[None], scoring, renormalize, 1.5)
        np.testing.assert_allclose(got[0], gradient(x, ids.tolist(), d, scoring, renormalize, 1.5), rtol=1e-13, atol=0)
