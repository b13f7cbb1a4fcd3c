"""Cases of the microscaled 4-bit operators, in plain form and through the library.

Four kinds of call, over one number format: an element is a 4-bit float e2m1
(sign, values 0 0.5 1 1.5 2 3 4 6), 32 consecutive elements of a row share one
scale 2^(byte - 127), and two elements share a byte (even k in the low nibble).

  quantize  16-bit values to that format, and the values that it stands for
  gemm      16-bit activations times microscaled weights
  gemm_mx   activations quantised, then the product of two microscaled matrices
  moe       a mixture-of-experts layer on a few tokens with microscaled experts

With ``own`` false, run() computes them from elementary torch operations in 32
bits and rounds once at the end; with ``own`` true it calls the library.
"""
import torch

own = False

BLOCK = 32
DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # quantising one token's activations: a call whose latency counts
        {"name": "quantize_token", "kind": "quantize", "type": "bf16", "M": 1, "K": 4096},
        # quantising the weights of one large projection
        {"name": "quantize_weights", "kind": "quantize", "type": "f16", "M": 28672, "K": 8192},
        # decoding one token through a small odd projection: the smallest product
        {"name": "gemm_one_small", "kind": "gemm", "type": "bf16", "M": 1, "N": 1021, "K": 1056},
        # decoding one token through a square 8192 projection
        {"name": "gemm_one", "kind": "gemm", "type": "f16", "M": 1, "N": 8192, "K": 8192},
        # decoding a batch of 16 through a wide projection
        {"name": "gemm_batch", "kind": "gemm", "type": "bf16", "M": 16, "N": 28672, "K": 8192},
        # prefill of 2048 tokens
        {"name": "gemm_prefill", "kind": "gemm", "type": "f16", "M": 2048, "N": 11008, "K": 4096},
        # decoding a batch of 64 with quantised activations
        {"name": "gemm_mx_batch", "kind": "gemm_mx", "type": "bf16", "M": 64, "N": 8192, "K": 8192},
        # a ragged prompt through a projection of odd sizes
        {"name": "gemm_mx_ragged", "kind": "gemm_mx", "type": "f16", "M": 333, "N": 1001, "K": 5152},
        # prefill of 2048 tokens with quantised activations
        {"name": "gemm_mx_prefill", "kind": "gemm_mx", "type": "bf16", "M": 2048, "N": 11008, "K": 4096},
        # one token through a layer of 32 experts, 4 of them taken
        {"name": "moe_one", "kind": "moe", "type": "bf16", "M": 1, "K": 4096, "I": 2048, "E": 32, "k": 4},
        # a few tokens through a layer of many small experts of odd sizes
        {"name": "moe_few", "kind": "moe", "type": "f16", "M": 5, "K": 2080, "I": 1056, "E": 60, "k": 6},
        # a decoding batch of 64: every expert is taken by some token
        {"name": "moe_batch", "kind": "moe", "type": "bf16", "M": 64, "K": 4096, "I": 2048, "E": 32, "k": 4},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return min(high, max(low, int(round(low * (high / low) ** rng.random()))))


def draw(rng):
    kind = rng.choice(("quantize", "gemm", "gemm", "gemm_mx", "gemm_mx", "moe", "moe"))
    case = {"kind": kind, "type": rng.choice(("f16", "bf16"))}
    if kind == "quantize":
        K = BLOCK * _spread(rng, 2, 344)
        case |= {"M": _spread(rng, 1, min(28672, 28672 * 8192 // K)), "K": K}
    elif kind == "moe":
        K, I, E = BLOCK * _spread(rng, 8, 128), BLOCK * _spread(rng, 4, 64), _spread(rng, 4, 64)
        E = max(4, min(E, 32 * 4096 * 2048 // (K * I)))
        case |= {"M": _spread(rng, 1, 64), "K": K, "I": I, "E": E, "k": rng.randint(1, min(8, E))}
    else:
        N, K = _spread(rng, 64, 28672), BLOCK * _spread(rng, 2, 256)
        most = 2048 * 11008 * 4096 // (N * K)
        M = 1 if kind == "gemm" and rng.random() < 0.25 else _spread(rng, 1, max(1, min(2048, most)))
        case |= {"M": M, "N": N, "K": K}
    return case


def _pow2(byte):
    """2^(byte - 127) in 32 bits for a byte of 0 .. 254."""
    b = byte.to(torch.int32)
    return torch.where(b == 0, torch.full_like(b, 1 << 22), b << 23).view(torch.float32)


def _quantize(x):
    """Microscaled codes and scale bytes of a matrix, from elementary operations."""
    v = x.float().view(x.shape[0], -1, BLOCK)
    _, e = torch.frexp(v.abs().amax(-1))
    byte = torch.where(v.abs().amax(-1) > 0, (e - 1 - 2 + 127).clamp(0, 254), torch.zeros_like(e))
    a = v.abs() * _pow2(254 - byte)[..., None]
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code.to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
    pair = code.view(x.shape[0], -1, 2)
    return pair[..., 0] | (pair[..., 1] << 4), byte.to(torch.uint8)


def _values(codes, scales):
    """The 32-bit values that codes [..., K/2] and scales [..., K/32] stand for."""
    one = torch.tensor(GRID + tuple(-g for g in GRID), device=codes.device)
    byte = torch.arange(256, device=codes.device)
    table = torch.stack((one[byte & 15], one[byte >> 4]), -1)
    v = table[codes.to(torch.int32)].view(*scales.shape, BLOCK) * _pow2(scales)[..., None]
    return v.view(*codes.shape[:-1], -1)


def _activations(g, M, K, dtype):
    """Rows of a layer's input: a few channels are far larger than the others."""
    x = torch.randn(M, K, generator=g, device=DEV)
    far = torch.rand(K, generator=g, device=DEV) < 1 / 128
    return (x * torch.where(far, 16.0, 1.0)).to(dtype)


def _weights(g, rows, K, dtype):
    spread = torch.exp(0.25 * torch.randn(rows, 1, generator=g, device=DEV))
    return (torch.randn(rows, K, generator=g, device=DEV) * (0.02 * spread)).to(dtype)


def _inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dtype, M, K = TYPES[case["type"]], case["M"], case["K"]
    s = {"kind": case["kind"], "dtype": dtype}
    if case["kind"] == "quantize":
        s["x"] = _weights(g, M, K, dtype) if M > 64 else _activations(g, M, K, dtype)
        return s
    s["x"] = _activations(g, M, K, dtype)
    if case["kind"] != "moe":
        s["codes"], s["scales"] = _quantize(_weights(g, case["N"], K, dtype))
        return s
    E, I = case["E"], case["I"]
    s["top_k"] = case["k"]
    s["router"] = (torch.randn(E, K, generator=g, device=DEV) * (1.5 / K ** 0.5)).to(dtype)
    for name, rows, cols in (("up", 2 * I, K), ("down", K, I)):
        codes, scales = _quantize(_weights(g, E * rows, cols, dtype))
        s[name + "_codes"], s[name + "_scales"] = codes.view(E, rows, -1), scales.view(E, rows, -1)
    return s


def prepare(case, seed):
    return _inputs(case, seed)


def _moe(s):
    x, k, E = s["x"].float(), s["top_k"], s["router"].shape[0]
    T, I = x.shape[0], s["up_codes"].shape[1] // 2
    logits, ids = torch.sort(x @ s["router"].float().t(), dim=1, descending=True, stable=True)
    p, ids = torch.softmax(logits[:, :k], 1), ids[:, :k]
    if T * k < E:  # fewer expert rows than experts: only the chosen ones are decoded
        up = _values(s["up_codes"][ids], s["up_scales"][ids])
        gu = torch.matmul(up, x[:, None, :, None])[..., 0]
        h = torch.nn.functional.silu(gu[..., :I]) * gu[..., I:] * p[..., None]
        down = _values(s["down_codes"][ids], s["down_scales"][ids])
        return torch.matmul(down, h[..., None])[..., 0].sum(1).to(s["dtype"])
    share = torch.zeros(T, E, device=x.device).scatter_(1, ids, p)
    gu = (x @ _values(s["up_codes"], s["up_scales"]).view(E * 2 * I, -1).t()).view(T, E, 2 * I)
    h = torch.nn.functional.silu(gu[..., :I]) * gu[..., I:] * share[..., None]
    down = _values(s["down_codes"], s["down_scales"])
    return torch.matmul(h.transpose(0, 1).contiguous(), down.transpose(1, 2)).sum(0).to(s["dtype"])


def run(state):
    s, kind = state, state["kind"]
    if own:
        from weight_only_quantization_quantize_amd import ops

        if kind == "quantize":
            codes, scales = ops.mxfp4_quantize(s["x"])
            return {"codes": codes, "scales": scales, "values": ops.mxfp4_dequantize(codes, scales, torch.bfloat16)}
        if kind == "gemm":
            return ops.mxfp4_gemm(s["x"], s["codes"], s["scales"])
        if kind == "gemm_mx":
            codes, scales = ops.mxfp4_quantize(s["x"])
            return ops.mxfp4_gemm_mx(codes, scales, s["codes"], s["scales"], s["dtype"])
        return ops.mxfp4_moe(s["x"], s["router"], s["up_codes"], s["up_scales"], s["down_codes"], s["down_scales"],
                             s["top_k"])
    if kind == "quantize":
        codes, scales = _quantize(s["x"])
        return {"codes": codes, "scales": scales, "values": _values(codes, scales).to(torch.bfloat16)}
    if kind == "gemm":
        return (s["x"].float() @ _values(s["codes"], s["scales"]).t()).to(s["dtype"])
    if kind == "gemm_mx":
        return (_values(*_quantize(s["x"])) @ _values(s["codes"], s["scales"]).t()).to(s["dtype"])
    return _moe(s)


def work(case):
    M, K, packed = case["M"], case["K"], 0.5 + 1 / BLOCK
    if case["kind"] == "quantize":
        return {"bytes": M * K * (2 + packed + 2), "flops": M * K}
    if case["kind"] == "moe":
        # the experts that some token takes, at the least: as many as one token takes
        E, I, k = case["E"], case["I"], case["k"]
        taken = E * (1 - (1 - k / E) ** M)
        return {"bytes": taken * 3 * I * K * packed + 2 * E * K + 4 * M * K, "flops": 2.0 * M * k * 3 * I * K + 2.0 * M * E * K}
    N = case["N"]
    return {"bytes": N * K * packed + 2 * M * K + 2 * M * N, "flops": 2.0 * M * N * K}


def _exact_blocks(x):
    """The nearest microscaled values of a matrix in 64 bits, by the format's definition: the scale's exponent is that
    of the block's largest magnitude less 2, an element the nearest of the grid, ties to the even code."""
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    rows = max(1, (1 << 24) // x.shape[1])
    for at in range(0, x.shape[0], rows):
        v = x[at:at + rows].double().reshape(-1, BLOCK)
        top = v.abs().max(1, keepdim=True).values
        e = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
        e = e + (torch.exp2(e + 1) <= top).double() - (torch.exp2(e) > top).double()
        scale = torch.exp2((e - 2).clamp(-127, 127))
        u = (v.abs() / scale).clamp(max=6.0)
        hi = torch.searchsorted(grid, u).clamp(max=7)
        lo = (hi - 1).clamp(min=0)
        up, down = grid[hi] - u, u - grid[lo]
        near = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), grid[hi], grid[lo])
        out[at:at + rows] = (torch.sign(v) * near * scale).reshape(-1, x.shape[1])
    return out


def _exact_values(codes, scales):
    grid = torch.tensor(GRID, dtype=torch.float64, device=codes.device)
    low, high = (codes & 15).long(), (codes >> 4).long()
    both = torch.stack([grid[n & 7] * (1 - 2 * (n >> 3)).double() for n in (low, high)], -1).flatten(-2)
    return both * torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, -1)


def _exact_moe(s):
    x, k, E = s["x"].double(), s["top_k"], s["router"].shape[0]
    I = s["up_codes"].shape[1] // 2
    logits = x @ s["router"].double().t()
    y = torch.zeros_like(x)
    order = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    weight = torch.exp(logits.gather(1, order) - logits.gather(1, order).max(1, keepdim=True).values)
    weight = weight / weight.sum(1, keepdim=True)
    for e in range(E):
        t, slot = torch.nonzero(order == e, as_tuple=True)
        if t.numel():
            gu = x[t] @ _exact_values(s["up_codes"][e], s["up_scales"][e]).t()
            h = gu[:, :I] / (1 + torch.exp(-gu[:, :I])) * gu[:, I:]
            y[t] += weight[t, slot][:, None] * (h @ _exact_values(s["down_codes"][e], s["down_scales"][e]).t())
    return y


def exact(case, seed):
    s = _inputs(case, seed)
    if s["kind"] == "quantize":
        return {"codes": None, "scales": None, "values": _exact_blocks(s["x"])}
    if s["kind"] == "moe":
        return _exact_moe(s)
    x = s["x"].double() if s["kind"] == "gemm" else _exact_blocks(s["x"])
    return x @ _exact_values(s["codes"], s["scales"]).t()
