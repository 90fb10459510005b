"""The 8-bit layer's operators as measured cases: the plain torch form of each beside the library's call.

The format (include/svdq.h, "FP8 block-128"): E4M3 codes [rows][K] with one power-of-two scale (E8M0) per 128
consecutive elements along K, the scales in tiles of 128 rows x 4 blocks.  Cases come from the repository's own
layers (4608 tokens, widths 3072, 9216, 12288) and from generic sizes around them: one token, odd token counts,
widths whose last block is short.
"""

import math

import torch

own = False

BLOCK = 128
F32 = torch.float32
F64 = torch.float64


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one token between two layers: latency alone
        {"name": "rmsnorm_1x3072", "op": "rmsnorm", "M": 1, "K": 3072, "res": "bf16", "gamma": True, "y": False},
        # an odd batch of tokens, wide rows, a residual stream kept in fp32, bf16 output beside the codes
        {"name": "rmsnorm_333x8208_f32", "op": "rmsnorm", "M": 333, "K": 8208, "res": "f32", "gamma": True, "y": True},
        # the token stream of the DiT layers
        {"name": "rmsnorm_4608x3072", "op": "rmsnorm", "M": 4608, "K": 3072, "res": "bf16", "gamma": True, "y": False},
        # a few tokens entering the out-projection of a single-stream block
        {"name": "quantize_64x15360", "op": "quantize", "M": 64, "K": 15360, "ld": 15360, "gelu": False},
        # the MLP part of a single-stream block's fused projection: 12288 of 21504 columns, through GELU
        {"name": "quantize_gelu_4608x12288", "op": "quantize", "M": 4608, "K": 12288, "ld": 21504, "gelu": True},
        # weights of a small layer as fp32 masters, and of the MLP up-projection as bf16
        {"name": "pack_1040x1000_f32", "op": "pack", "K": 1040, "N": 1000, "w": "f32"},
        {"name": "pack_3072x12288_bf16", "op": "pack", "K": 3072, "N": 12288, "w": "bf16"},
        # one token through the QKV projection: the weights' bytes bound it
        {"name": "linear_1x3072x9216", "op": "linear", "M": 1, "K": 3072, "N": 9216, "bias": True},
        # an odd number of tokens, a width with a short last block
        {"name": "linear_77x2064x5000", "op": "linear", "M": 77, "K": 2064, "N": 5000, "bias": True},
        # the MLP down-projection of the full token stream
        {"name": "linear_4608x12288x3072", "op": "linear", "M": 4608, "K": 12288, "N": 3072, "bias": False},
        # the MLP up-projection with its GELU and the next layer's quantiser: a few tokens, then the full stream
        {"name": "linear_gelu_16x3072x12288", "op": "linear_gelu", "M": 16, "K": 3072, "N": 12288, "bias": True},
        {"name": "linear_gelu_4608x3072x12288", "op": "linear_gelu", "M": 4608, "K": 3072, "N": 12288, "bias": True},
    ]


def _log(rng, lo, hi, mult):
    """A multiple of `mult` in [lo, hi], spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(v / mult + 0.5) * mult))


def draw(rng):
    op = rng.choice(["rmsnorm", "quantize", "pack", "linear", "linear", "linear_gelu"])
    if op == "rmsnorm":
        return {"op": op, "M": _log(rng, 1, 4608, 1), "K": _log(rng, 64, 12288, 16),
                "res": rng.choice(["none", "bf16", "bf16", "f32"]), "gamma": rng.random() < 0.8,
                "y": rng.random() < 0.3}
    if op == "quantize":
        K = _log(rng, 64, 12288, 16)
        return {"op": op, "M": _log(rng, 1, 4608, 1), "K": K, "ld": K + rng.choice([0, 0, 8, 1024]),
                "gelu": rng.random() < 0.5}
    if op == "pack":
        return {"op": op, "K": _log(rng, 64, 8192, 16), "N": _log(rng, 64, 8192, 8), "w": rng.choice(["bf16", "f32"])}
    while True:
        c = {"op": op, "M": _log(rng, 1, 4608, 1), "K": _log(rng, 64, 12288, 16),
             "N": _log(rng, 64, 12288, 8 if op == "linear" else 16), "bias": rng.random() < 0.6}
        if c["M"] * c["K"] * c["N"] <= 4608 * 3072 * 12288:
            return c


def work(case):
    if case["op"] == "pack":
        K, N = case["K"], case["N"]
        return {"bytes": K * N * (2 if case["w"] == "bf16" else 4) + _packed_bytes(N, K), "flops": 2 * K * N}
    M, K = case["M"], case["K"]
    if case["op"] == "rmsnorm":
        r = {"none": 0, "bf16": 2, "f32": 4}[case["res"]]
        b = M * K * (2 + 2 * r + (2 if case["y"] else 0)) + _packed_bytes(M, K) + (2 * K if case["gamma"] else 0)
        return {"bytes": b, "flops": 6 * M * K}
    if case["op"] == "quantize":
        return {"bytes": 2 * M * K + _packed_bytes(M, K), "flops": (12 if case["gelu"] else 2) * M * K}
    N = case["N"]
    b = _packed_bytes(M, K) + _packed_bytes(N, K) + (2 * N if case["bias"] else 0)
    b += 2 * M * N if case["op"] == "linear" else _packed_bytes(M, N)
    return {"bytes": b, "flops": 2 * M * N * K}


def _packed_bytes(rows, K):
    return rows * K + rows * -(-K // BLOCK)


# ------------------------------------------------------------- plain form --
def _to_tiles(b):
    """Scale bytes [rows][blocks] -> the tiles' byte order (rows and blocks padded with 0)."""
    rows, n = b.shape
    R, C = -(-rows // 128), -(-n // 4)
    full = torch.zeros((R * 128, C * 4), dtype=torch.uint8, device=b.device)
    full[:rows, :n] = b
    return full.view(R, 4, 32, C, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _from_tiles(s, rows, K):
    """The tiles' bytes -> the scales' exponents as int32 [rows][blocks]."""
    n = -(-K // BLOCK)
    R, C = -(-rows // 128), -(-n // 4)
    b = s.view(torch.uint8).view(R, C, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(R * 128, C * 4)
    return b[:rows, :n].to(torch.int32) - 127


def _two(e):
    """2^e in fp32, from the bits (a library power of two may be off by an ulp, which moves ties)."""
    return ((e.to(torch.int64) + 1023) << 52).view(F64).to(F32)


def _blocks(v):
    rows, K = v.shape
    pad = -K % BLOCK
    if pad:
        v = torch.cat([v, v.new_zeros((rows, pad))], dim=1)
    return v.view(rows, -1, BLOCK)


def _quantise(v):
    """fp32 [rows][K] -> (codes float8_e4m3fn [rows][K], scales float8_e8m0fnu in tiles)."""
    rows, K = v.shape
    b = _blocks(v)
    amax = b.abs().amax(dim=2)
    m, x = torch.frexp(amax)                     # amax = m 2^x; 448 = 0.875 * 2^9
    e = x - 9 + (m > 0.875).to(x.dtype)
    e = torch.where(amax > 0, e, torch.full_like(e, -127)).clamp_min(-127)
    codes = (b * _two(-e)[:, :, None]).reshape(rows, -1)[:, :K].to(torch.float8_e4m3fn)
    return codes.contiguous(), _to_tiles((e + 127).to(torch.uint8)).view(torch.float8_e8m0fnu)


def _dequantise(codes, scales):
    rows, K = codes.shape
    b = _blocks(codes.to(F32))
    return (b * _two(_from_tiles(scales, rows, K))[:, :, None]).reshape(rows, -1)[:, :K]


def _gelu(v):
    return 0.5 * v * torch.special.erfc(v * -math.sqrt(0.5))


def _plain(state):
    op = state["op"]
    if op == "rmsnorm":
        h, out = state["X"].to(F32), {}
        if state["residual"] is not None:
            out["residual"] = (h + state["residual"].to(F32)).to(state["residual"].dtype)
            h = out["residual"].to(F32)
        y = h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + state["eps"])
        if state["gamma"] is not None:
            y = y * state["gamma"].to(F32)
        out["codes"], out["scales"] = _quantise(y)
        if state["y"]:
            out["Y"] = y.to(torch.bfloat16)
        return out
    if op == "quantize":
        v = state["X"].to(F32)
        return _quantise(_gelu(v) if state["gelu"] else v)
    if op == "pack":
        return _quantise(state["W"].to(F32).t())
    acc = _dequantise(state["x_codes"], state["x_scales"]) @ _dequantise(state["w_codes"], state["w_scales"]).t()
    if state["bias"] is not None:
        acc = acc + state["bias"].to(F32)
    return acc.to(torch.bfloat16) if op == "linear" else _quantise(_gelu(acc))


# ---------------------------------------------------------- library's call --
def _own(state):
    import bit_w4a4_quantized_smooth_b200 as svdq
    op = state["op"]
    if op == "rmsnorm":
        codes, scales, residual, Y = svdq.rmsnorm(state["X"], state["gamma"], state["residual"], eps=state["eps"],
                                                  bf16_out=state["y"])
        out = {"codes": codes, "scales": scales}
        if residual is not None:
            out["residual"] = residual
        if Y is not None:
            out["Y"] = Y
        return out
    if op == "quantize":
        return svdq.quantize_fp8(state["X"], gelu=state["gelu"])
    if op == "pack":
        return svdq.pack_weight_fp8(state["W"])
    fn = svdq.linear_fp8 if op == "linear" else svdq.linear_fp8_gelu
    return fn(state["x_codes"], state["x_scales"], state["w_codes"], state["w_scales"], state["bias"])


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------- inputs --
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda") * scale


def _activation(g, M, K):
    """Hidden states: N(0, 1) with 1 % of the channels 20 to 100 times larger."""
    hot = torch.rand(K, generator=g, device="cuda") < 0.01
    gain = torch.where(hot, 20.0 + 80.0 * torch.rand(K, generator=g, device="cuda"), torch.ones(K, device="cuda"))
    return _randn(g, M, K) * gain


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op == "pack":
        W = _randn(g, case["K"], case["N"], scale=0.02)
        return {"op": op, "W": W.to(torch.bfloat16) if case["w"] == "bf16" else W}
    M, K = case["M"], case["K"]
    if op == "rmsnorm":
        dt = {"none": None, "bf16": torch.bfloat16, "f32": F32}[case["res"]]
        return {"op": op, "X": _randn(g, M, K, scale=0.5).to(torch.bfloat16), "eps": 1e-6, "y": case["y"],
                "residual": None if dt is None else _activation(g, M, K).to(dt),
                "gamma": (1.0 + _randn(g, K, scale=0.1)).to(torch.bfloat16) if case["gamma"] else None}
    if op == "quantize":
        X = _randn(g, M, case["ld"], scale=1.5) if case["gelu"] else _activation(g, M, case["ld"])
        return {"op": op, "X": X.to(torch.bfloat16)[:, case["ld"] - K:], "gelu": case["gelu"]}
    N = case["N"]
    x_codes, x_scales = _quantise(_randn(g, M, K))
    w_codes, w_scales = _quantise(_randn(g, N, K, scale=1.0 / math.sqrt(K)))
    bias = _randn(g, N, scale=0.1).to(torch.bfloat16) if case["bias"] else None
    return {"op": op, "x_codes": x_codes, "x_scales": x_scales, "w_codes": w_codes, "w_scales": w_scales,
            "bias": bias}


# ------------------------------------------------- definition in 64 bits --
POWERS = [2.0 ** k for k in range(-200, 201)]  # exact, by index


def _power(k):
    return torch.tensor(POWERS, dtype=F64, device=k.device)[k.to(torch.int64) + 200]


def _exact_fp8(v):
    """The format's definition in fp64: per block the smallest 2^e (e >= -127) with amax <= 448 2^e; every value to
    the nearest multiple of its binade's step (8 steps a binade, 2^-9 at the least), ties to even."""
    rows, K = v.shape
    codes = torch.empty((rows, K), dtype=torch.float8_e4m3fn, device=v.device)
    n = -(-K // BLOCK)
    grid = torch.zeros((-(-rows // 128) * 128, -(-n // 4) * 4), dtype=torch.int64, device=v.device)
    for j in range(n):
        part = v[:, j * BLOCK:(j + 1) * BLOCK]
        top = part.abs().amax(dim=1)
        e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 448.0)).clamp(-127, 127)
        e = torch.where(top > 448.0 * _power(e), e + 1, e)  # log2 may be off by one next to a power of two
        e = torch.where((top <= 448.0 * _power(e - 1)) & (e > -127), e - 1, e)
        e = torch.where(top > 0, e, torch.full_like(e, -127.0))
        u = part * _power(-e)[:, None]
        binade = torch.floor(torch.log2(u.abs().clamp_min(2.0 ** -6)))
        binade = torch.where(u.abs() < _power(binade), binade - 1, binade)
        binade = torch.where(u.abs() >= _power(binade + 1), binade + 1, binade).clamp_min(-6)
        step = _power(binade - 3)
        codes[:, j * BLOCK:(j + 1) * BLOCK] = (torch.round(u / step) * step).to(torch.float8_e4m3fn)
        grid[:rows, j] = e.to(torch.int64) + 127
    row = torch.arange(grid.shape[0], device=v.device)[:, None]
    blk = torch.arange(grid.shape[1], device=v.device)[None, :]
    at = ((row // 128) * (grid.shape[1] // 4) + blk // 4) * 512 + (row % 32) * 16 + (row % 128 // 32) * 4 + blk % 4
    scales = torch.empty(grid.numel(), dtype=torch.uint8, device=v.device)
    scales[at.reshape(-1)] = grid.reshape(-1).to(torch.uint8)
    return codes, scales.view(torch.float8_e8m0fnu)


def _exact_values(codes, scales):
    rows, K = codes.shape
    n4 = -(-(-(-K // BLOCK)) // 4)
    row = torch.arange(rows, device=codes.device)[:, None]
    k = torch.arange(K, device=codes.device)[None, :] // BLOCK
    at = ((row // 128) * n4 + k // 4) * 512 + (row % 32) * 16 + (row % 128 // 32) * 4 + k % 4
    return codes.to(F64) * _power(scales.view(torch.uint8)[at].to(torch.int64) - 127)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "rmsnorm":
        out = {}
        h = s["X"].to(F64)
        if s["residual"] is not None:
            out["residual"] = (h + s["residual"].to(F64)).to(s["residual"].dtype)
            h = out["residual"].to(F64)
        y = h / torch.sqrt((h * h).sum(dim=1, keepdim=True) / h.shape[1] + s["eps"])
        if s["gamma"] is not None:
            y = y * s["gamma"].to(F64)[None, :]
        out["codes"], out["scales"] = _exact_fp8(y)
        if s["y"]:
            out["Y"] = y
        return out
    if op == "pack":
        return _exact_fp8(s["W"].to(F64).t())
    if op == "quantize":
        v = s["X"].to(F64)
        return _exact_fp8(v * torch.special.ndtr(v) if s["gelu"] else v)
    acc = _exact_values(s["x_codes"], s["x_scales"]) @ _exact_values(s["w_codes"], s["w_scales"]).t()
    if s["bias"] is not None:
        acc = acc + s["bias"].to(F64)
    return acc if op == "linear" else _exact_fp8(acc * torch.special.ndtr(acc))
