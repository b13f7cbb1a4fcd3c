"""The 8-bit integer operators and the routing to experts without a GPU: their oracle against
worked values, differences and plain statements of its own, the refusals of the binding and of
the C ABI (checked before any HIP call), and the registers of the compiled kernels."""
from __future__ import annotations

import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch
from torch.autograd import forward_ad

from oracle import int8_oracle as O
from weight_only_quantization_quantize_amd import _lib, ops
from weight_only_quantization_quantize_amd import build as woq_build

# ---------------------------------------------------------------------------
# The oracle
# ---------------------------------------------------------------------------


def test_quantize_worked_rows():
    x = np.array([[127.0, 0.5, 1.5, -2.5, -126.5, 63.5], [0, 0, 0, 0, 0, 0], [1, np.inf, 0, 0, 0, 0], [2, np.nan, 1, 0, 0, 0]])
    q, s = O.quantize(x)
    assert q[0].tolist() == [127, 0, 2, -2, -126, 64] and s[0] == 1.0
    assert q[1].tolist() == [0] * 6 and s[1] == 0.0
    assert q[2].tolist() == [0] * 6 and np.isnan(s[2])
    assert q[3].tolist() == [0] * 6 and np.isnan(s[3])


def test_quantize_error_is_at_most_half_a_step():
    x = np.random.default_rng(1).normal(size=(20, 64))
    q, s = O.quantize(x)
    assert np.abs(x - q * s[:, None]).max(1).max() <= (s / 2).max() * (1 + 1e-12)
    assert np.all(np.abs(x - q * s[:, None]) <= s[:, None] / 2 * (1 + 1e-12))


def test_folds_cancel_in_a_product():
    g = np.random.default_rng(2)
    x, w, s = g.normal(size=(4, 64)), g.normal(size=(5, 64)), np.exp2(g.integers(-3, 4, 64)).astype(np.float64)
    a, b = O.fold(x, s, False), O.fold(w, s, True)
    np.testing.assert_allclose(a @ b.T, x @ w.T, rtol=1e-5, atol=1e-5)


def test_route_worked_rows():
    x = np.array([[1.0, 3.0, 3.0, -np.inf], [-np.inf] * 4, [0.0, np.nan, 5.0, 1.0]])
    e, w = O.route(x, 2)
    assert e.tolist() == [[1, 2], [0, 1], [2, 3]]
    np.testing.assert_allclose(w[0], [0.5, 0.5])
    assert w[1].tolist() == [0, 0]
    # a bias steers the choice, not the weights; a masked expert stays last whatever its bias
    e, w = O.route(x[:1], 3, "sigmoid", bias=[2.0, 0, 0, 9.0], renormalize=False, scale=2.0)
    assert e.tolist() == [[0, 1, 2]]
    np.testing.assert_allclose(w[0], 2 / (1 + np.exp(-x[0, :3])))
    # groups: of {0.9, 0.1}, {0.6, 0.5} the first has the best expert, the second the better pair
    x = np.log([[0.9, 0.1, 0.6, 0.5]])
    assert O.route(x, 2, groups=2, top_groups=1, group_top=1)[0].tolist() == [[0, 1]]
    assert O.route(x, 2, groups=2, top_groups=1, group_top=2)[0].tolist() == [[2, 3]]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradient_against_differences(scoring, renormalize):
    g = np.random.default_rng(3)
    x, d = g.normal(size=(3, 9)), g.normal(size=(3, 4))
    e, _ = O.route(x, 4, scoring)

    def loss(x):
        s = O.scores(x, scoring)
        w = np.array([O._weights(x[t], s[t], e[t], scoring, renormalize, 1.7) for t in range(3)])
        return (w * d).sum()

    got, step = O.route_backward(x, e, d, scoring, renormalize, 1.7), 1e-5
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += step
        down[i] -= step
        # a central difference is off by step^2 / 6 times a third derivative (below 10 here) and by 2^-52 / step
        assert abs((loss(up) - loss(down)) / (2 * step) - got[i]) < 1e-8


def test_moe_is_the_dense_layer_where_nothing_is_rounded():
    """Codes that are exact: one hot column of the activations, h's rows with one non-zero element."""
    x = np.zeros((2, 16))
    x[0, 3], x[1, 5] = 127.0, -127.0
    up, down = np.zeros((2, 32, 16), np.int8), np.zeros((2, 16, 16), np.int8)
    up[:, 2, :], up[:, 18, :] = 1, 2  # gate and up of column 2
    down[0, :, 2], down[1, :, 2] = np.arange(16), np.arange(16)[::-1]
    y, reach, _ = O.moe(x, np.array([[0, 1], [1, -1]]), np.array([[1.0, 2.0], [0.5, 7.0]]), up, np.ones((2, 32)), down,
                        np.ones((2, 16)))
    h0, h1 = 127.0 / (1 + np.exp(-127.0)) * 254.0, -127.0 / (1 + np.exp(127.0)) * -254.0
    np.testing.assert_allclose(y[0], h0 * (np.arange(16) + 2.0 * np.arange(16)[::-1]))
    np.testing.assert_allclose(y[1], 0.5 * h1 * np.arange(16)[::-1])
    assert not reach.any()


# ---------------------------------------------------------------------------
# Refusals of the binding
# ---------------------------------------------------------------------------
F16, F32, I8, I32 = torch.float16, torch.float32, torch.int8, torch.int32


def _x(m=3, k=32, dtype=F16):
    return torch.zeros(m, k, dtype=dtype)


def _w(n=5, k=32):
    return torch.zeros(n, k, dtype=I8), torch.zeros(n)


def _moe_args(**other):
    T, H, I, E, k = 3, 32, 16, 4, 2
    a = {"X": _x(T, H), "experts": torch.zeros(T, k, dtype=I32), "weights": torch.zeros(T, k),
         "up_codes": torch.zeros(E, 2 * I, H, dtype=I8), "up_scales": torch.zeros(E, 2 * I),
         "down_codes": torch.zeros(E, H, I, dtype=I8), "down_scales": torch.zeros(E, H)}
    return a | other


REFUSED = {
    "quantize rank": lambda: ops.int8_quantize(torch.zeros(32, dtype=F16)),
    "quantize type": lambda: ops.int8_quantize(torch.zeros(2, 32, dtype=torch.float64)),
    "quantize empty": lambda: ops.int8_quantize(_x(0)),
    "quantize K": lambda: ops.int8_quantize(_x(2, 24)),
    "quantize long": lambda: ops.int8_quantize(_x(1, 131072)),
    "quantize act_scale": lambda: ops.int8_quantize(_x(), torch.ones(16)),
    "quantize out": lambda: ops.int8_quantize(_x(), out=(torch.zeros(3, 32, dtype=torch.uint8), torch.zeros(3))),
    "quantize out scales": lambda: ops.int8_quantize(_x(), out=(torch.zeros(3, 32, dtype=I8), torch.zeros(3, dtype=F16))),
    "gemm codes": lambda: ops.int8_gemm(_x(), torch.zeros(3), *_w()),
    "gemm scales": lambda: ops.int8_gemm(_w(3)[0], torch.zeros(4), *_w()),
    "gemm K": lambda: ops.int8_gemm(*_w(3, 48), *_w()),
    "gemm dtype": lambda: ops.int8_gemm(*_w(3), *_w(), dtype=torch.float64),
    "gemm bias": lambda: ops.int8_gemm(*_w(3), *_w(), bias=torch.zeros(5, dtype=F16)),
    "gemm empty": lambda: ops.int8_gemm(*_w(0), *_w()),
    "gemm out": lambda: ops.int8_gemm(*_w(3), *_w(), dtype=F16, out=torch.zeros(3, 5)),
    "linear type": lambda: ops.int8_linear(_x(dtype=F32), *_w()),
    "linear K": lambda: ops.int8_linear(_x(3, 48), *_w()),
    "linear empty": lambda: ops.int8_linear(_x(0), *_w()),
    "route scoring": lambda: ops.moe_route(_x(), 2, "relu"),
    "route top_k": lambda: ops.moe_route(_x(), 33),
    "route no top_k": lambda: ops.moe_route(_x(), 0),
    "route top_k of groups": lambda: ops.moe_route(_x(), 9, groups=4, top_groups=1),
    "route groups": lambda: ops.moe_route(_x(), 2, groups=5),
    "route top_groups": lambda: ops.moe_route(_x(), 2, groups=4, top_groups=5),
    "route group_top": lambda: ops.moe_route(_x(), 2, groups=32, group_top=2),
    "route experts": lambda: ops.moe_route(torch.zeros(2, 513), 2),
    "route bias": lambda: ops.moe_route(_x(), 2, bias=torch.zeros(31)),
    "route out": lambda: ops.moe_route(_x(), 2, out=(torch.zeros(3, 2), torch.zeros(3, 2))),
    "backward experts": lambda: ops.moe_route_backward(_x(), torch.zeros(3, 2, dtype=torch.int64), torch.zeros(3, 2)),
    "backward dweights": lambda: ops.moe_route_backward(_x(), torch.zeros(3, 2, dtype=I32), torch.zeros(3, 3)),
    "moe down": lambda: ops.int8_moe(**_moe_args(down_codes=torch.zeros(4, 32, 32, dtype=I8))),
    "moe X": lambda: ops.int8_moe(**_moe_args(X=_x(3, 48))),
    "moe experts": lambda: ops.int8_moe(**_moe_args(experts=torch.zeros(2, 2, dtype=I32))),
    "moe weights": lambda: ops.int8_moe(**_moe_args(weights=torch.zeros(3, 2, dtype=F16))),
    "moe top_k": lambda: ops.int8_moe(**_moe_args(experts=torch.zeros(3, 65, dtype=I32), weights=torch.zeros(3, 65))),
    "moe no choices": lambda: ops.int8_moe(**_moe_args(experts=torch.zeros(3, 0, dtype=I32), weights=torch.zeros(3, 0))),
    "moe out": lambda: ops.int8_moe(**_moe_args(), out=torch.zeros(3, 32)),
    "moe empty": lambda: ops.int8_moe(**_moe_args(X=_x(0), experts=torch.zeros(0, 2, dtype=I32), weights=torch.zeros(0, 2))),
    # all in order, but not on a GPU
    "host tensors": lambda: ops.int8_moe(**_moe_args()),
}


@pytest.mark.parametrize("name", REFUSED)
def test_refused(name):
    with pytest.raises(ValueError):
        REFUSED[name]()


DERIVED = {
    "quantize": lambda x: ops.int8_quantize(x),
    "linear": lambda x: ops.int8_linear(x, *_w()),
    "route": lambda x: ops.moe_route(x, 2),
    "backward": lambda x: ops.moe_route_backward(x, torch.zeros(3, 2, dtype=I32), torch.zeros(3, 2)),
    "moe": lambda x: ops.int8_moe(**_moe_args(X=x)),
}


@pytest.mark.parametrize("name", DERIVED)
def test_derivatives_are_refused(name):
    with pytest.raises(ValueError, match="gradient"):
        DERIVED[name](_x().requires_grad_(True))
    with forward_ad.dual_level(), pytest.raises(ValueError, match="gradient"):
        DERIVED[name](forward_ad.make_dual(_x(), torch.ones(3, 32, dtype=F16)))
    with torch.no_grad(), pytest.raises(ValueError, match="GPU tensors only"):
        DERIVED[name](_x().requires_grad_(True))


# ---------------------------------------------------------------------------
# Refusals of the C ABI.  The addresses are never dereferenced.
# ---------------------------------------------------------------------------
MB = 1 << 20
INVALID, UNSUPPORTED = _lib.WOQ_ERR_INVALID_ARGUMENT, _lib.WOQ_ERR_UNSUPPORTED


def P(i):
    return (i + 1) * MB


QUANTIZE = dict(x=P(0), xdtype=0, act_scale=P(1), multiply=0, M=4, K=64, codes=P(2), scales=P(3), stream=None)
GEMM = dict(a=P(0), sa=P(1), w=P(2), sw=P(3), bias=P(4), M=4, N=5, K=64, ydtype=0, Y=P(5), stream=None)
LINEAR = dict(X=P(0), xdtype=0, act_scale=P(1), w=P(2), sw=P(3), bias=P(4), M=4, N=5, K=64, Y=P(5), ws=P(6), ws_bytes=MB, stream=None)
ROUTE = dict(logits=P(0), dtype=0, T=4, E=8, top_k=2, scoring=0, bias=P(1), groups=2, top_groups=1, group_top=1, renormalize=1,
             scale=1.0, experts=P(2), weights=P(3), stream=None)
BACKWARD = dict(logits=P(0), dtype=0, experts=P(1), dweights=P(2), T=4, E=8, top_k=2, scoring=0, renormalize=1, scale=1.0,
                dlogits=P(3), stream=None)
MOE = dict(X=P(0), xdtype=0, experts=P(1), weights=P(2), up=P(3), su=P(4), down=P(5), sd=P(6), T=4, H=64, I=32, E=8, top_k=2,
           Y=P(7), ws=P(8), ws_bytes=MB, stream=None)
ABI = [
    ("woq_int8_quantize", QUANTIZE, INVALID, [dict(x=None), dict(x=P(0) + 8), dict(xdtype=3), dict(M=0), dict(K=24), dict(K=0),
                                              dict(codes=None), dict(codes=P(2) + 8), dict(scales=None), dict(scales=P(3) + 2),
                                              dict(act_scale=P(1) + 4), dict(codes=P(0)), dict(scales=P(1)),
                                              dict(scales=P(2) + 64), dict(codes=P(0) + 496)]),
    ("woq_int8_quantize", QUANTIZE, UNSUPPORTED, [dict(K=131072), dict(M=(1 << 28) + 1)]),
    ("woq_int8_gemm", GEMM, INVALID, [dict(a=None), dict(sa=None), dict(w=None), dict(sw=None), dict(Y=None), dict(Y=P(5) + 8),
                                      dict(w=P(2) + 4), dict(bias=P(4) + 2), dict(M=0), dict(N=0), dict(K=8), dict(ydtype=5),
                                      dict(Y=P(0)), dict(Y=P(1)), dict(Y=P(2) + 304), dict(Y=P(3)), dict(Y=P(4))]),
    ("woq_int8_gemm", GEMM, UNSUPPORTED, [dict(K=131072), dict(M=1 << 28, N=1 << 28), dict(M=1 << 22, N=1 << 16)]),
    ("woq_int8_linear", LINEAR, INVALID, [dict(X=None), dict(xdtype=2), dict(Y=None), dict(ws=None), dict(ws=P(6) + 16),
                                          dict(ws_bytes=100), dict(Y=P(0)), dict(ws=P(5)), dict(ws=P(0)), dict(act_scale=P(1) + 8)]),
    ("woq_moe_route", ROUTE, INVALID, [dict(logits=None), dict(logits=P(0) + 1), dict(dtype=9), dict(T=0), dict(E=0), dict(top_k=0),
                                       dict(top_k=5), dict(scoring=2), dict(groups=3), dict(groups=0), dict(top_groups=3),
                                       dict(top_groups=0), dict(group_top=3), dict(group_top=0), dict(groups=8, group_top=2),
                                       dict(bias=P(1) + 1), dict(experts=None), dict(weights=None), dict(experts=P(0)),
                                       dict(weights=P(2) + 28)]),
    ("woq_moe_route", ROUTE, UNSUPPORTED, [dict(E=1024), dict(E=512, groups=1, top_k=65), dict(T=(1 << 24) + 1)]),
    ("woq_moe_route_backward", BACKWARD, INVALID, [dict(logits=None), dict(experts=None), dict(dweights=None), dict(dlogits=None),
                                                   dict(dlogits=P(0)), dict(dlogits=P(1)), dict(dlogits=P(2)), dict(dtype=1, dlogits=P(3) + 1)]),
    ("woq_int8_moe", MOE, INVALID, [dict(X=None), dict(xdtype=2), dict(experts=None), dict(weights=P(2) + 2), dict(up=None), dict(su=None),
                                    dict(down=P(5) + 8), dict(sd=None), dict(T=0), dict(H=40), dict(I=8), dict(top_k=0), dict(Y=P(0)),
                                    dict(Y=P(3)), dict(ws=P(7)), dict(ws=None), dict(ws_bytes=1000), dict(Y=None)]),
    ("woq_int8_moe", MOE, UNSUPPORTED, [dict(E=513), dict(top_k=65), dict(H=1 << 16, I=1 << 16), dict(T=1 << 20, H=1 << 16),
                                        dict(T=1 << 23, H=16, I=16, top_k=64), dict(T=(1 << 24) + 1, H=16, I=16, top_k=1)]),
]


@pytest.mark.parametrize("name,base,status,change", [(n, b, s, c) for n, b, s, cs in ABI for c in cs],
                         ids=lambda v: v if isinstance(v, str) else ("-".join(v) if isinstance(v, dict) and len(v) < 4 else ""))
def test_abi_refuses(name, base, status, change):
    assert _lib.call(name, *(base | change).values()) == status
    assert _lib.load().woq_last_error()


def test_workspace_sizes_of_invalid_sizes_are_zero():
    assert _lib.call("woq_int8_linear_workspace_bytes", 0, 5, 64) == 0
    assert _lib.call("woq_int8_linear_workspace_bytes", 4, 5, 60) == 0
    assert _lib.call("woq_int8_moe_workspace_bytes", 4, 64, 32, 8, 0) == 0
    assert _lib.call("woq_int8_moe_workspace_bytes", 4, 64, 32, 600, 2) == 0
    assert _lib.call("woq_int8_moe_workspace_bytes", 4, 64, 32, 8, 2) > 0


# ---------------------------------------------------------------------------
# Registers: a spill would wait for all loads on their way whenever it is read back
# ---------------------------------------------------------------------------
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
FILES = {
    "int8_quantize.hip": ["int8_quantize_kernel"],
    "int8_gemv.hip": ["int8_gemv_kernel"],
    "int8_gemm.hip": ["int8_gemm_kernel"],
    "moe_route.hip": ["moe_route_kernel", "moe_route_wide_kernel", "moe_route_backward_kernel"],
    "int8_moe_row.hip": ["int8_moe_row_up_kernel", "int8_moe_row_down_kernel"],
    "int8_moe.hip": ["int8_moe_prepare_kernel", "int8_moe_product_kernel", "int8_moe_combine_kernel"],
}


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("src", sorted(FILES))
def test_kernels_do_not_spill(src, tmp_path):
    out = str(tmp_path / "k.s")
    cmd = [HIPCC, "-x", "hip", *woq_build.COMMON_FLAGS, "--cuda-device-only", "-S", os.path.join(woq_build.CSRC, src), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    private = {}
    for m in re.finditer(r"\.amdhsa_kernel (\S+)\n(.*?)\.end_amdhsa_kernel", open(out).read(), re.S):
        private[m.group(1)] = int(re.search(r"\.amdhsa_private_segment_fixed_size (\d+)", m.group(2)).group(1))
    for name in FILES[src]:
        assert any(name in k for k in private), f"no {name} in {src}"
    assert not {k: n for k, n in private.items() if n}
