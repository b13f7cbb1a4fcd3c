"""GPU parity of the 8-bit integer products: every tile that may take them, in every output type, and the bits of a row
between the kernels.

Tolerance of a product: the sum is exact; its conversion, the first scale's product, and the second's with the bias
round once each (2^-24), then the output.
"""
import numpy as np
import pytest
import torch

from tests.test_gpu_int8 import ABOVE, BF16, F16, F32, HALF, TINY, U, check_moe, gemm_inputs, layer, on_gpu, rng, tensor
from weight_only_quantization_quantize_amd import ops

pytestmark = pytest.mark.gpu


# Each tile with 1, 2, .. row blocks left for its last tile, all columns ragged; tests/test_int8_tiles.py reads the choice of tiles.
TILES = [(804, 13381, 672), (861, 13411, 656), (1164, 9333, 672), (2515, 4699, 656), (1030, 14573, 656), (1093, 14675, 688),
         (1182, 13573, 656), (1476, 10937, 656), (1155, 6479, 656), (647, 10857, 704), (517, 14277, 656), (258, 10911, 704),
         (321, 11047, 688), (141, 10909, 656), (197, 8487, 656), (65, 9267, 656), (5, 5, 848), (23, 9001, 2112), (5, 8597, 2112),
         (2139, 197, 2384), (333, 1001, 5168), (5, 7, 1248), (771, 13153, 208), (1153, 9267, 16), (1035, 13189, 144),
         (641, 10907, 112), (325, 10947, 144), (68, 8201, 192)]


@pytest.mark.parametrize("M,N,K", TILES)
def test_every_tile(M, N, K):
    a, sa, w, sw, b = gemm_inputs(M, N, K, True)
    a, sa, w, sw, b = tensor(a, torch.int8), tensor(sa), tensor(w, torch.int8), tensor(sw), tensor(b)
    plain = a.double() @ w.double().t().contiguous() * sa.double()[:, None] * sw.double()
    for bias in (None, b):
        ref = plain if bias is None else plain + bias.double()
        for dtype in (F16, BF16, F32):
            y = ops.int8_gemm(a, sa, w, sw, bias, dtype).double()
            bound = ((2 if bias is None else 1) * U * ref.abs() + 2 * U * plain.abs() + HALF[dtype] * ref.abs()) * ABOVE + TINY[dtype] + 2.0 ** -149
            worst = float(((y - ref).abs() / bound).max())
            print(f"{M} x {N} x {K} {dtype} bias {bias is not None}: worst element {worst:.3f} of its bound", flush=True)
            assert worst <= 1.0


def bits(t):
    return t.view(torch.int32 if t.dtype == F32 else torch.int16)


@pytest.mark.parametrize("N,K", [(1001, 4096), (260, 528), (77, 16), (500, 8192), (130, 20000)])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("bias", [False, True])
def test_a_row_has_the_same_bits_in_every_batch(N, K, dtype, bias):
    """Batches of one to four rows are streamed (up to K = 8192; one row past that), larger ones go to tiles."""
    a, sa, w, sw, b = gemm_inputs(300, N, K, bias)
    sa[2], sw[5], a[3] = -sa[2], -sw[5], 0  # (zeros of either sign)
    codes, scales, args = tensor(a, torch.int8), tensor(sa), (tensor(w, torch.int8), tensor(sw), tensor(b) if bias else None, dtype)
    y = ops.int8_gemm(codes, scales, *args)
    for at in (0, 3, 295):
        for M in (1, 2, 3, 4, 5):
            few = ops.int8_gemm(codes[at:at + M].contiguous(), scales[at:at + M].contiguous(), *args)
            assert torch.equal(bits(few), bits(y[at:at + M])), (at, M)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("K", [1024, 8192, 20000])
def test_a_row_of_a_linear_has_the_same_bits_in_every_batch(dtype, K):
    g, N = rng(41, K), 333
    x, w, s = tensor(g.normal(size=(60, K)), dtype), tensor(g.normal(size=(N, K)) * 0.02, dtype), tensor(np.exp(g.normal(size=K) / 2))
    codes, scales = ops.int8_quantize(w, s, weight=True)
    bias = tensor(g.normal(size=N))
    y = ops.int8_linear(x, codes, scales, s, bias)
    for M in (1, 2, 3, 4, 5):
        assert torch.equal(bits(ops.int8_linear(x[:M], codes, scales, s, bias)), bits(y[:M])), M


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_large_tiles_of_a_layer_of_long_rows(dtype):
    """Tiles of 320 rows with 1 .. 5 row blocks, whose products run for more stages than LDS holds: some tokens against the
    oracle, many against the same token alone, which another kernel takes."""
    g, H, I, counts = rng(42), 1040, 4112, (320, 64, 1, 128, 256, 192, 331)
    E, T = len(counts), sum(counts)
    x, weights = tensor(g.normal(size=(T, H)), dtype), layer(7, H, I, E)
    e = tensor(g.permutation(np.repeat(np.arange(E), counts)).astype(np.int32)[:, None], torch.int32)
    w = tensor(g.random((T, 1)).astype(np.float32))
    first = np.array([int(np.flatnonzero(e.cpu().numpy()[:, 0] == i)[0]) for i in range(E)])  # of each expert
    y = check_moe(x, e, w, weights, "long rows", np.concatenate([first, np.arange(0, T, 160)]))
    gpu = on_gpu(*weights)
    for t in range(0, T, 5):
        assert torch.equal(bits(y[t:t + 1]), bits(ops.int8_moe(x[t:t + 1], e[t:t + 1], w[t:t + 1], *gpu))), t
