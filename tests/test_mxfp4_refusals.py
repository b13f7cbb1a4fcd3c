"""Refusals of the microscaled operators that need no GPU: derivatives asked of
them in either mode, and outputs that share memory with another argument (the C
ABI checks them before any HIP call)."""
import pytest
import torch
from torch.autograd import forward_ad

from weight_only_quantization_quantize_amd import _lib, ops

N, K = 16, 256
H, I, E = 64, 32, 4


def _w(n=N, k=K):
    return torch.zeros(n, k // 2, dtype=torch.uint8), torch.zeros(n, k // 32, dtype=torch.uint8)


def _moe_args():
    return [torch.zeros(3, H, dtype=torch.float16), torch.zeros(E, H, dtype=torch.float16),
            torch.zeros(E, 2 * I, H // 2, dtype=torch.uint8), torch.zeros(E, 2 * I, H // 32, dtype=torch.uint8),
            torch.zeros(E, H, I // 2, dtype=torch.uint8), torch.zeros(E, H, I // 32, dtype=torch.uint8), 2]


def _moe_with(at, t):
    a = _moe_args()
    a[at] = t
    return a


DERIVED = {
    "quantize": (3, K, lambda x: ops.mxfp4_quantize(x)),
    "gemm": (3, K, lambda x: ops.mxfp4_gemm(x, *_w())),
    "moe": (3, H, lambda x: ops.mxfp4_moe(*_moe_with(0, x))),
    "router": (E, H, lambda x: ops.mxfp4_moe(*_moe_with(1, x))),
}


@pytest.mark.parametrize("name", DERIVED)
def test_forward_mode_tangents_are_refused(name):
    M, k, call = DERIVED[name]
    x = torch.zeros(M, k, dtype=torch.float16)
    with forward_ad.dual_level():
        with pytest.raises(ValueError, match="no gradient"):
            call(forward_ad.make_dual(x, torch.ones_like(x)))
        with pytest.raises(ValueError, match="GPU tensors only"):  # one without a tangent passes
            call(x)
    # under torch.no_grad() a tangent is still asked for
    with forward_ad.dual_level(), torch.no_grad():
        with pytest.raises(ValueError, match="no gradient"):
            call(forward_ad.make_dual(x, torch.ones_like(x)))


@pytest.mark.parametrize("name", DERIVED)
def test_function_transforms_are_refused(name):
    M, k, call = DERIVED[name]
    x = torch.zeros(M, k, dtype=torch.float16)
    with pytest.raises(ValueError, match="no gradient"):
        torch.func.jvp(call, (x,), (torch.ones_like(x),))
    with pytest.raises(ValueError, match="no gradient"):
        torch.func.grad(lambda t: call(t).sum())(x)


def test_outputs_that_ask_for_a_gradient_are_refused():
    x = torch.zeros(3, K, dtype=torch.float16)
    for call in (lambda o: ops.mxfp4_gemm(x, *_w(), out=o), lambda o: ops.mxfp4_gemm_mx(*_w(3), *_w(), torch.float16, out=o)):
        with pytest.raises(ValueError, match="no gradient"):
            call(torch.zeros(3, N, dtype=torch.float16, requires_grad=True))
    with pytest.raises(ValueError, match="no gradient"):
        ops.mxfp4_moe(*_moe_args(), out=torch.zeros(3, H, dtype=torch.float16, requires_grad=True))
    with torch.no_grad(), pytest.raises(ValueError, match="GPU tensors only"):
        ops.mxfp4_gemm(x, *_w(), out=torch.zeros(3, N, dtype=torch.float16, requires_grad=True))


# ---------------------------------------------------------------------------
# Outputs that share memory with another argument.  The addresses are never
# dereferenced: a refused call returns before any HIP call.
# ---------------------------------------------------------------------------

MB = 1 << 20


def _place(sizes):
    """Addresses 16 MB apart, none overlapping, for arguments of these sizes."""
    assert max(sizes.values()) < 16 * MB
    return {name: 16 * MB * (i + 1) for i, name in enumerate(sizes)}


def _assert_overlaps_refused(call, sizes, outputs, allowed=()):
    lib = _lib.load()
    base = _place(sizes)
    for out in outputs:
        for other in sizes:
            if other == out or (out, other) in allowed:
                continue
            for at in (base[other],                                                    # the same start
                       base[other] + (sizes[other] - 1) // 256 * 256,                  # its last bytes
                       base[other] - (sizes[out] - 1) // 256 * 256):                   # the output's last bytes
                places = dict(base)
                places[out] = at
                assert call(lib, places) == _lib.WOQ_ERR_INVALID_ARGUMENT, (out, other, at)
                assert b"overlap" in lib.woq_last_error(), (out, other, lib.woq_last_error())


def test_quantize_refuses_overlap():
    M, k = 1024, 1024
    sizes = {"x": 2 * M * k, "codes": M * k // 2, "scales": M * k // 32}
    _assert_overlaps_refused(lambda lib, p: lib.woq_mxfp4_quantize(p["x"], 0, M, k, p["codes"], p["scales"], None), sizes,
                             ["codes", "scales"])


def test_dequantize_refuses_overlap():
    M, k = 512, 1024
    sizes = {"codes": M * k // 2, "scales": M * k // 32, "out": 4 * M * k}
    _assert_overlaps_refused(lambda lib, p: lib.woq_mxfp4_dequantize(p["codes"], p["scales"], M, k, 2, p["out"], None), sizes,
                             ["out"])


@pytest.mark.parametrize("M, n, k", [(1, 4096, 1024), (16, 1024, 1024), (300, 1024, 1024)])
def test_gemm_refuses_overlap(M, n, k):
    need = _lib.load().woq_mxfp4_gemm_workspace_bytes(M, n, k)
    sizes = {"x": 2 * M * k, "codes": n * k // 2, "scales": n * k // 32, "y": 2 * M * n}
    if need:
        sizes["ws"] = need
    _assert_overlaps_refused(lambda lib, p: lib.woq_mxfp4_gemm(p["x"], 0, p["codes"], p["scales"], M, n, k, p["y"], p.get("ws"),
                                                               need, None), sizes, ["y"] + (["ws"] if need else []))


@pytest.mark.parametrize("M, n, k", [(16, 1024, 1024), (1000, 2048, 4096)])
def test_gemm_mx_refuses_overlap(M, n, k):
    need = _lib.load().woq_mxfp4_gemm_mx_workspace_bytes(M, n, k)
    sizes = {"a": M * k // 2, "as": M * k // 32, "codes": n * k // 2, "scales": n * k // 32, "y": 2 * M * n}
    if need:
        sizes["ws"] = need
    _assert_overlaps_refused(lambda lib, p: lib.woq_mxfp4_gemm_mx(p["a"], p["as"], p["codes"], p["scales"], M, n, k, 0, p["y"],
                                                                  p.get("ws"), need, None), sizes, ["y"] + (["ws"] if need else []))


def test_moe_refuses_overlap():
    T, h, i, e, k = 40, 1024, 512, 8, 2
    need = _lib.load().woq_mxfp4_moe_workspace_bytes(T, h, i, e, k)
    sizes = {"x": 2 * T * h, "router": 2 * e * h, "up": e * i * h, "ups": e * i * h // 16, "down": e * h * i // 2,
             "downs": e * h * i // 32, "y": 2 * T * h, "ws": need}
    _assert_overlaps_refused(lambda lib, p: lib.woq_mxfp4_moe(p["x"], 0, p["router"], p["up"], p["ups"], p["down"], p["downs"], T,
                                                              h, i, e, k, p["y"], p["ws"], need, None), sizes, ["y", "ws"],
                             allowed=[("y", "x")])  # in place: x is read before y is written


def test_products_of_too_many_rows_are_refused():
    # 2^28 rows: past it the scales' row stride (4 bytes a row) and the grid's threads would
    # pass 32 bits
    lib = _lib.load()
    at = 1 << 44  # never dereferenced: refused, or (the last rows that are taken) for its workspace
    for M in ((1 << 28) + 1, (1 << 30) - 1):
        assert lib.woq_mxfp4_gemm_workspace_bytes(M, 8, 32) == 0
        assert lib.woq_mxfp4_gemm_mx_workspace_bytes(M, 8, 32) == 0
        assert lib.woq_mxfp4_gemm(at, 0, 2 * at, 3 * at, M, 8, 32, 4 * at, 5 * at, 1 << 42, None) == _lib.WOQ_ERR_UNSUPPORTED
        assert lib.woq_mxfp4_gemm_mx(at, 6 * at, 2 * at, 3 * at, M, 8, 32, 0, 4 * at, 5 * at, 1 << 42, None) == _lib.WOQ_ERR_UNSUPPORTED
    M = 1 << 28
    need = lib.woq_mxfp4_gemm_workspace_bytes(M, 8, 32)
    assert need > 0
    assert lib.woq_mxfp4_gemm(at, 0, 2 * at, 3 * at, M, 8, 32, 4 * at, 5 * at, need - 1, None) == _lib.WOQ_ERR_INVALID_ARGUMENT
