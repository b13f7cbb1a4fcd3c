"""The microscaled 4-bit float operators on the host: the oracle's own pins,
the binding's refusals (CPU tensors: each fails before any library call) and
the C ABI's (each call returns during validation, before any HIP call)."""
import numpy as np
import pytest
import torch

from oracle import mxfp4_oracle as O
from weight_only_quantization_quantize_amd import _lib, ops

FAKE = 0x10000  # an aligned address that is never dereferenced


def test_oracle_worked_block():
    x = np.zeros((1, 32))
    # top 6 -> scale 2^0: every grid value, the ties, and what rounds to them
    x[0, :12] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.3, 0.2, -6.0]
    codes, scales = O.quantize(x)
    assert scales[0, 0] == 127
    n = np.stack([codes & 15, codes >> 4], -1).reshape(-1)
    assert list(n[:12]) == [7, 0, 2, 2, 4, 4, 6, 6, 8, 9, 0, 15]
    assert list(O.dequantize(codes, scales)[0, :8]) == [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]


@pytest.mark.parametrize("top, byte", [(1.0, 125), (1.99, 125), (2.0, 126), (6.0, 127), (7.9, 127), (8.0, 128),
                                       (2.0 ** -24, 101), (2.0 ** -126, 0), (2.0 ** 127, 252)])
def test_oracle_scale_byte(top, byte):
    x = np.zeros((1, 32))
    x[0, 3] = -top
    assert O.quantize(x)[1][0, 0] == byte


def test_oracle_special_blocks():
    x = np.zeros((1, 128))
    x[0, 32], x[0, 64], x[0, 97] = np.inf, np.nan, -0.0
    codes, scales = O.quantize(x)
    assert list(scales[0]) == [0, 255, 255, 0]
    assert codes[0, 48] == 0x80 and codes.sum() == 0x80
    v = O.dequantize(codes, scales)
    assert np.isnan(v[0, 32:96]).all() and not np.isnan(v[0, :32]).any() and not np.isnan(v[0, 96:]).any()


def test_oracle_quantization_is_nearest_and_idempotent():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((4, 64)).astype(np.float16).astype(np.float64)
    codes, scales = O.quantize(x)
    v = O.dequantize(codes, scales)
    s = np.repeat(np.exp2(scales.astype(np.float64) - 127), 32, axis=1)
    every = np.concatenate([O.GRID, -O.GRID])
    best = np.abs(x[..., None] - every * s[..., None]).min(-1)
    assert np.array_equal(np.abs(x - v), best)
    again, scales2 = O.quantize(v)
    keep = np.repeat(np.abs(v).reshape(4, 2, 32).max(-1) >= 4 * np.exp2(scales.astype(np.float64) - 127), 32, axis=1)
    assert np.array_equal(O.dequantize(again, scales2)[keep], v[keep])


def test_oracle_top_k_ties_take_the_lower_index():
    assert O.top_k(np.array([[1.0, 3.0, 3.0, 2.0, 3.0]]), 3).tolist() == [[1, 2, 4]]


# ---------------------------------------------------------------------------
# Refusals of the binding
# ---------------------------------------------------------------------------

N, K = 16, 256
H, I, E = 64, 32, 4


def _w(n=N, k=K):
    return torch.zeros(n, k // 2, dtype=torch.uint8), torch.zeros(n, k // 32, dtype=torch.uint8)


def _moe_args():
    return [torch.zeros(3, H, dtype=torch.float16), torch.zeros(E, H, dtype=torch.float16),
            torch.zeros(E, 2 * I, H // 2, dtype=torch.uint8), torch.zeros(E, 2 * I, H // 32, dtype=torch.uint8),
            torch.zeros(E, H, I // 2, dtype=torch.uint8), torch.zeros(E, H, I // 32, dtype=torch.uint8), 2]


def test_valid_calls_reach_the_device_check():
    x = torch.zeros(3, K, dtype=torch.bfloat16)
    for call in (lambda: ops.mxfp4_quantize(x), lambda: ops.mxfp4_dequantize(*_w()),
                 lambda: ops.mxfp4_gemm(x, *_w()), lambda: ops.mxfp4_gemm_mx(*_w(3), *_w()),
                 lambda: ops.mxfp4_moe(*_moe_args())):
        with pytest.raises(ValueError, match="GPU tensors only"):
            call()


@pytest.mark.parametrize("x, needle", [
    (torch.zeros(3, K), "fp16/bf16"),
    (torch.zeros(K, dtype=torch.float16), "fp16/bf16"),
    (torch.zeros(3, 48, dtype=torch.float16), "multiple of 32"),
    (torch.zeros(3, 0, dtype=torch.float16), "multiple of 32"),
    (torch.zeros(0, K, dtype=torch.float16), "M >= 1"),
    (torch.zeros(3, K, dtype=torch.float16, requires_grad=True), "no gradient"),
])
def test_quantize_refuses(x, needle):
    with pytest.raises(ValueError, match=needle):
        ops.mxfp4_quantize(x)


def test_quantize_refuses_wrong_outputs():
    x = torch.zeros(N, K, dtype=torch.float16)
    codes, scales = _w()
    with pytest.raises(ValueError, match="out codes"):
        ops.mxfp4_quantize(x, out=(codes[:, :-1], scales))
    with pytest.raises(ValueError, match="out scales"):
        ops.mxfp4_quantize(x, out=(codes, scales.to(torch.int8)))


@pytest.mark.parametrize("case, needle", [
    ("codes_dtype", "weight codes"), ("codes_dim", "weight codes"), ("codes_cols", "weight codes"),
    ("scales_dtype", "weight scales"), ("scales_shape", "weight scales"), ("x_dtype", "fp16/bf16"),
    ("x_cols", "fp16/bf16"), ("x_empty", "at least one row"), ("w_empty", "at least one row"), ("out", "out must be"),
    ("grad", "no gradient"),
])
def test_gemm_refuses(case, needle):
    x, (codes, scales), out = torch.zeros(3, K, dtype=torch.float16), _w(), None
    if case == "codes_dtype":
        codes = codes.to(torch.int8)
    elif case == "codes_dim":
        codes = codes.view(-1)
    elif case == "codes_cols":
        codes = codes[:, :-8]
    elif case == "scales_dtype":
        scales = scales.to(torch.float16)
    elif case == "scales_shape":
        scales = scales[:, :-1]
    elif case == "x_dtype":
        x = x.float()
    elif case == "x_cols":
        x = x[:, :-32]
    elif case == "x_empty":
        x = x[:0]
    elif case == "w_empty":
        codes, scales = codes[:0], scales[:0]
    elif case == "out":
        out = torch.zeros(3, N + 1, dtype=torch.float16)
    elif case == "grad":
        x.requires_grad_()
    with pytest.raises(ValueError, match=needle):
        ops.mxfp4_gemm(x, codes, scales, out=out)


def test_gemm_mx_refuses():
    with pytest.raises(ValueError, match="share K"):
        ops.mxfp4_gemm_mx(*_w(3, 128), *_w())
    with pytest.raises(ValueError, match="dtype must be"):
        ops.mxfp4_gemm_mx(*_w(3), *_w(), torch.float32)
    with pytest.raises(ValueError, match="activation codes"):
        ops.mxfp4_gemm_mx(torch.zeros(3, K // 2), _w(3)[1], *_w())
    with pytest.raises(ValueError, match="at least one row"):
        ops.mxfp4_gemm_mx(*_w(0), *_w())


@pytest.mark.parametrize("case, needle", [
    ("tokens", "1 to 64 tokens"), ("no_tokens", "1 to 64 tokens"), ("router_shape", "router must be"),
    ("router_dtype", "router must be"), ("x_cols", "X must be"), ("down", "up must be"), ("odd_up", "up must be"),
    ("top_k_0", "top_k"), ("top_k_5", "top_k"), ("experts", "512 experts"), ("top_k_65", "top_k of up to 64"), ("grad", "no gradient"),
])
def test_moe_refuses(case, needle):
    a = _moe_args()
    if case == "tokens":
        a[0] = torch.zeros(65, H, dtype=torch.float16)
    elif case == "no_tokens":
        a[0] = a[0][:0]
    elif case == "router_shape":
        a[1] = a[1][:-1]
    elif case == "router_dtype":
        a[1] = a[1].bfloat16()
    elif case == "x_cols":
        a[0] = a[0][:, :32]
    elif case == "down":
        a[4], a[5] = a[4][:, :-1], a[5][:, :-1]
    elif case == "odd_up":
        a[2], a[3] = a[2][:, :-1], a[3][:, :-1]
    elif case == "top_k_0":
        a[6] = 0
    elif case == "top_k_5":
        a[6] = 5
    elif case == "experts":
        for j in range(1, 6):
            a[j] = a[j][:1].expand(513, *a[j].shape[1:])
    elif case == "top_k_65":
        for j in range(1, 6):
            a[j] = a[j][:1].expand(100, *a[j].shape[1:])
        a[6] = 65
    elif case == "grad":
        a[0].requires_grad_()
    with pytest.raises(ValueError, match=needle):
        ops.mxfp4_moe(*a)


# ---------------------------------------------------------------------------
# Refusals of the C ABI
# ---------------------------------------------------------------------------

INVALID, UNSUPPORTED = _lib.WOQ_ERR_INVALID_ARGUMENT, _lib.WOQ_ERR_UNSUPPORTED


def _refused(name, good, changes):
    lib = _lib.load()
    for at, value, status in changes:
        a = list(good)
        a[at] = value
        assert getattr(lib, name)(*a) == status, (name, at, value)
        assert lib.woq_last_error()


def test_abi_quantize_and_dequantize_refuse():
    _refused("woq_mxfp4_quantize", [FAKE, 0, 4, 64, FAKE, FAKE, None],
             [(0, None, INVALID), (0, FAKE + 8, INVALID), (1, 2, INVALID), (1, -1, INVALID), (2, 0, INVALID),
              (3, 48, INVALID), (3, 0, INVALID), (3, -32, INVALID), (4, None, INVALID), (4, FAKE + 4, INVALID),
              (5, None, INVALID), (2, 1 << 40, UNSUPPORTED), (3, 1 << 40, UNSUPPORTED)])
    _refused("woq_mxfp4_dequantize", [FAKE, FAKE, 4, 64, 0, FAKE, None],
             [(0, None, INVALID), (1, None, INVALID), (2, -1, INVALID), (3, 33, INVALID), (4, 3, INVALID),
              (5, None, INVALID), (5, FAKE + 2, INVALID)])


def test_abi_gemm_refuses():
    lib = _lib.load()
    need = lib.woq_mxfp4_gemm_workspace_bytes(4, 64, 64)
    assert need > 0
    good = [FAKE, 0, FAKE, FAKE, 4, 64, 64, FAKE, FAKE, need, None]
    _refused("woq_mxfp4_gemm", good,
             [(0, None, INVALID), (0, FAKE + 2, INVALID), (1, 2, INVALID), (2, None, INVALID), (2, FAKE + 8, INVALID),
              (3, None, INVALID), (4, 0, INVALID), (5, 0, INVALID), (6, 40, INVALID), (7, None, INVALID),
              (7, FAKE + 2, INVALID), (8, None, INVALID), (8, FAKE + 128, INVALID), (9, need - 1, INVALID),
              (5, 1 << 29, UNSUPPORTED), (4, 1 << 40, UNSUPPORTED)])
    need = lib.woq_mxfp4_gemm_mx_workspace_bytes(600, 4096, 4096)  # tiles that read turned scales
    assert need > 0
    _refused("woq_mxfp4_gemm_mx", [FAKE, FAKE, FAKE, FAKE, 600, 4096, 4096, 0, FAKE, FAKE, need, None],
             [(0, None, INVALID), (1, None, INVALID), (2, FAKE + 8, INVALID), (3, None, INVALID), (4, 0, INVALID),
              (5, -5, INVALID), (6, 16, INVALID), (7, 2, INVALID), (8, None, INVALID),
              (9, None, INVALID), (9, FAKE + 64, INVALID), (10, need - 1, INVALID)])


def test_abi_workspace_queries():
    lib = _lib.load()
    assert lib.woq_mxfp4_gemm_workspace_bytes(1, 8192, 8192) == 0      # one row uses none
    assert lib.woq_mxfp4_gemm_workspace_bytes(1, 64, 16416) > 0        # but past the GEMV's K
    assert lib.woq_mxfp4_gemm_workspace_bytes(16, 4096, 4096) == 0     # split in the product's launch
    assert lib.woq_mxfp4_gemm_mx_workspace_bytes(4, 64, 64) == 0       # scales kept in LDS
    for bad in ((0, 64, 64), (4, 0, 64), (4, 64, 63), (4, 64, 0)):
        assert lib.woq_mxfp4_gemm_workspace_bytes(*bad) == 0
    assert lib.woq_mxfp4_moe_workspace_bytes(1, 64, 32, 4, 2) > 0
    for bad in ((0, 64, 32, 4, 2), (65, 64, 32, 4, 2), (1, 48, 32, 4, 2), (1, 64, 31, 4, 2), (1, 64, 32, 0, 2),
                (1, 64, 32, 513, 2), (1, 64, 32, 4, 0), (1, 64, 32, 4, 5), (1, 64, 32, 100, 65)):
        assert lib.woq_mxfp4_moe_workspace_bytes(*bad) == 0


def test_abi_moe_refuses():
    lib = _lib.load()
    need = lib.woq_mxfp4_moe_workspace_bytes(3, 64, 32, 4, 2)
    good = [FAKE, 0, FAKE, FAKE, FAKE, FAKE, FAKE, 3, 64, 32, 4, 2, FAKE, FAKE, need, None]
    _refused("woq_mxfp4_moe", good,
             [(0, None, INVALID), (1, 2, INVALID), (2, None, INVALID), (2, FAKE + 8, INVALID), (3, None, INVALID),
              (4, None, INVALID), (5, FAKE + 4, INVALID), (6, None, INVALID), (7, 0, INVALID), (7, 65, UNSUPPORTED),
              (8, 40, INVALID), (9, 0, INVALID), (10, 0, INVALID), (10, 513, UNSUPPORTED), (11, 0, INVALID),
              (11, 5, INVALID), (12, None, INVALID), (13, None, INVALID), (14, need - 1, INVALID)])
