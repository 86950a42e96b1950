"""Cases of the microscaled 4-bit floating point operators: quantisation, product and linear layer.

Formats (elements e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives):
  "mx"  blocks of 32 along K share one power-of-two scale (e8m0);
  "nv"  blocks of 16 along K share one e4m3 scale, the tensor one fp32 scale g.
A value is element * block scale * g.  Quantising takes z = fl32(x * fl32(1 / g)) and, per block,
  mx: s = 2^(floor(log2(max|z|)) - 2),  nv: s = e4m3(max|z| / 6),  element = e2m1(z / s),
all round to nearest even with saturation; the product is y = ga * gw * sum_k (a sa)(w sw).

Layouts (the framework's): codes are rows of K_pad / 2 bytes, K_pad = 128 ceil(K / 128), the even k of a byte in its
low half; scales are 512-byte tiles of 128 rows x 4 blocks, row r and block c of a tile at 16 (r % 32) + 4 (r / 32) + c,
the tiles of a row band one after another.
"""
import math

import torch

own = False

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
# between code i and i + 1: the midpoint, and whether the tie goes up (to the even code)
MIDS = [(0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)]
BLOCK = {"mx": 32, "nv": 16}
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def pad_up(n, m):
    return (n + m - 1) // m * m


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode token quantised and read back: the smallest call
        {"name": "quant_mx_token", "op": "quant", "fmt": "mx", "rows": 1, "K": 2560, "ld": 2560, "x": "bf16", "y": "bf16"},
        # a ragged fp16 batch that is a slice of a wider tensor (one part of a fused projection)
        {"name": "quant_nv_slice", "op": "quant", "fmt": "nv", "rows": 997, "K": 6910, "ld": 13824, "x": "fp16", "y": "fp32"},
        # a weight matrix prepared offline: its tensor scale, codes, and the values read back
        {"name": "quant_nv_weight", "op": "quant", "fmt": "nv", "rows": 13824, "K": 5120, "ld": 5120, "x": "bf16", "y": "bf16"},
        # a prefill's activations kept in fp32
        {"name": "quant_mx_prefill", "op": "quant", "fmt": "mx", "rows": 2048, "K": 6912, "ld": 6912, "x": "fp32", "y": "fp16"},
        # single-token decode of a small and of a large layer
        {"name": "gemm_mx_token", "op": "gemm", "fmt": "mx", "M": 1, "N": 2560, "K": 6912, "y": "bf16"},
        {"name": "gemm_nv_token_large", "op": "gemm", "fmt": "nv", "M": 1, "N": 55296, "K": 5120, "y": "bf16"},
        # a ragged batch: nothing is a multiple of a tile
        {"name": "gemm_nv_ragged", "op": "gemm", "fmt": "nv", "M": 77, "N": 3211, "K": 4801, "y": "fp16"},
        # prefill products
        {"name": "gemm_nv_prefill", "op": "gemm", "fmt": "nv", "M": 2048, "N": 13824, "K": 2560, "y": "bf16"},
        {"name": "gemm_mx_large", "op": "gemm", "fmt": "mx", "M": 4096, "N": 27648, "K": 5120, "y": "bf16"},
        # the linear layer as a decode step, a small batch and a prefill call it
        {"name": "linear_nv_token", "op": "linear", "fmt": "nv", "M": 1, "N": 6912, "K": 2560, "x": "bf16", "y": "bf16"},
        {"name": "linear_mx_batch", "op": "linear", "fmt": "mx", "M": 12, "N": 13824, "K": 2560, "x": "bf16", "y": "bf16"},
        {"name": "linear_nv_prefill", "op": "linear", "fmt": "nv", "M": 2048, "N": 2560, "K": 6912, "x": "fp16", "y": "fp16"},
    ]


MOST_MACS = 4096 * 27648 * 5120  # of one product
MOST_VALUES = 13824 * 5120       # of one quantised tensor


def draw(rng):
    def size(lo, hi):
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        if rng.random() < 0.5 and n >= 64:  # half of them whole tiles, half odd
            n = n // 64 * 64
        return max(lo, min(hi, n))

    op, fmt = rng.choice(["quant", "gemm", "linear"]), rng.choice(["mx", "nv"])
    if op == "quant":
        K = size(16, 27648)
        rows = size(1, min(16384, MOST_VALUES // K))
        return {"op": op, "fmt": fmt, "rows": rows, "K": K, "ld": K + rng.choice([0, 0, 1, 8, 2560]),
                "x": rng.choice(["bf16", "fp16", "fp32"]), "y": rng.choice(["bf16", "fp16", "fp32"])}
    N, K = size(64, 55296), size(64, 27648)
    if N * K > 55296 * 5120:
        K = 55296 * 5120 // N
    M = size(1, max(1, min(4096, MOST_MACS // (N * K))))
    if rng.random() < 0.35:  # decode: one token up to a small batch
        M = rng.choice([1, 1, 2, 3, 4, 7, 8, 16])
    c = {"op": op, "fmt": fmt, "M": M, "N": N, "K": K, "y": rng.choice(["bf16", "fp16"])}
    if op == "linear":
        c["x"] = rng.choice(["bf16", "fp16", "fp32"])
    return c


# ------------------------------------------------------------------ plain forms

def divided(x, by):
    """x / by, correctly rounded (a division by a Python number multiplies by its reciprocal on the GPU)."""
    return x / torch.full((), by, dtype=x.dtype, device=x.device)


def quantise(z, fmt):
    """Codes (0..7, with their signs) and block scales of z, fp32 [rows, K_pad]: every step is exact in fp32."""
    rows, Kp = z.shape
    zb = z.view(rows, Kp // BLOCK[fmt], BLOCK[fmt])
    amax = zb.abs().amax(dim=2)
    if fmt == "mx":
        e = torch.where(amax > 0, torch.frexp(amax)[1] - 3, -127).clamp(-127, 127)
        s = torch.ldexp(torch.ones_like(amax, dtype=torch.float64), e).float()
    else:
        s = divided(amax, 6.0).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    a, t = zb.abs(), s.unsqueeze(2)
    m = [(a >= mid * t) if up else (a > mid * t) for mid, up in MIDS]
    code = torch.stack(m, 0).sum(0, dtype=torch.uint8)
    code = torch.where(t > 0, code, 0)
    return code.view(rows, Kp), torch.signbit(z), s


def padded(x, Kp):
    z = torch.zeros(x.shape[0], Kp, dtype=torch.float32, device=x.device)
    z[:, :x.shape[1]] = x
    return z


def lay_out(code, sign, s, fmt):
    """The framework's code rows and scale tiles."""
    n = code | (sign.to(torch.uint8) << 3)
    codes = (n[:, 0::2] | (n[:, 1::2] << 4)).contiguous()
    b = (torch.where(s > 0, torch.frexp(s)[1] + 126, 0).to(torch.uint8) if fmt == "mx"
         else s.to(torch.float8_e4m3fn).view(torch.uint8))
    rows, nb = b.shape
    t = torch.zeros(pad_up(rows, 128), pad_up(nb, 4), dtype=torch.uint8, device=b.device)
    t[:rows, :nb] = b
    t = t.view(t.shape[0] // 128, 4, 32, t.shape[1] // 4, 4).permute(0, 3, 2, 1, 4)
    return codes, t.contiguous().view(-1)


def values(codes, scales, fmt):
    """element * block scale, fp32 [rows, K_pad] (exact), from the framework's layouts."""
    rows, Kp = codes.shape[0], 2 * codes.shape[1]
    nb = Kp // BLOCK[fmt]
    lut = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float32, device=codes.device)
    v = lut[torch.stack([codes & 15, codes >> 4], dim=2).view(rows, Kp).int()]
    kt, rt = pad_up(nb, 4) // 4, pad_up(rows, 128) // 128
    b = scales.view(rt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)[:rows, :nb].contiguous()
    if fmt == "mx":
        s = torch.ldexp(torch.ones_like(b, dtype=torch.float64), b.int() - 127).float()
    else:
        s = b.view(torch.float8_e4m3fn).float()
    return (v.view(rows, nb, BLOCK[fmt]) * s.unsqueeze(2)).view(rows, Kp)


def plain_quant(x, fmt, g):
    z = padded(x.float() * (1.0 / g), pad_up(x.shape[1], 128))
    return lay_out(*quantise(z, fmt), fmt)


def plain_tensor_scale(x):
    return divided(x.float().abs().amax(), 2688.0).clamp(min=2.0 ** -126).view(1)


def plain_gemm(a, sa, ga, w, sw, gw, fmt, dtype):
    return (torch.matmul(values(a, sa, fmt), values(w, sw, fmt).t()) * (ga * gw)).to(dtype)


# ------------------------------------------------------------------ inputs

def activations(rows, K, ld, dtype, gen):
    """N(0, 1) with one value in a hundred 20 times as large, each row at a level of its own."""
    x = torch.randn(rows, ld, generator=gen, device="cuda")
    x *= torch.where(torch.rand(rows, ld, generator=gen, device="cuda") < 0.01, 20.0, 1.0)
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=gen, device="cuda"))
    return x.to(dtype)[:, :K]


def weights(N, K, gen):
    return torch.randn(N, K, generator=gen, device="cuda") * 0.02


def inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    fmt = case["fmt"]
    if case["op"] == "quant":
        return {"x": activations(case["rows"], case["K"], case["ld"], DTYPES[case["x"]], gen)}
    M, N, K = case["M"], case["N"], case["K"]
    w = weights(N, K, gen)
    x = activations(M, K, K, DTYPES[case.get("x", "bf16")], gen)
    # the tensor scales that a calibrated "nv" layer keeps; "mx" has none
    ga = plain_tensor_scale(x) * 1.25 if fmt == "nv" else torch.ones(1, device="cuda")
    gw = plain_tensor_scale(w) if fmt == "nv" else torch.ones(1, device="cuda")
    return {"x": x, "w": w, "ga": ga, "gw": gw}


def prepare(case, seed):
    d = inputs(case, seed)
    state = {"case": case, "x": d["x"]}
    if case["op"] == "quant":
        return state
    fmt = case["fmt"]
    state["w"], state["sw"] = plain_quant(d["w"], fmt, d["gw"])
    state["ga"], state["gw"] = d["ga"], d["gw"]
    if case["op"] == "gemm":
        state["a"], state["sa"] = plain_quant(d["x"], fmt, d["ga"])
        del state["x"]
    return state


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    fmt, dtype = case["fmt"], DTYPES[case["y"]]
    if own:
        import ternary_weight_bit_w2a8_b200 as bn
        f = bn.BITNET_FP4_MX if fmt == "mx" else bn.BITNET_FP4_NV
        if case["op"] == "quant":
            g = bn.bitnet_fp4_tensor_scale(state["x"]) if fmt == "nv" else None
            codes, scales = bn.bitnet_fp4_quant(state["x"], f, g=g)
            y = bn.bitnet_fp4_dequant(codes, scales, case["K"], f, g=g, dtype=dtype)
            return {"y": y} if g is None else {"y": y, "g": g}
        ga, gw = (state["ga"], state["gw"]) if fmt == "nv" else (None, None)
        if case["op"] == "gemm":
            return {"y": bn.bitnet_fp4_gemm(state["a"], state["sa"], state["w"], state["sw"], case["K"], f,
                                            ga=ga, gw=gw, dtype=dtype)}
        return {"y": bn.bitnet_fp4_linear(state["x"], state["w"], state["sw"], f, ga=ga, gw=gw, dtype=dtype)}
    if case["op"] == "quant":
        x = state["x"]
        g = plain_tensor_scale(x) if fmt == "nv" else torch.ones(1, device=x.device)
        codes, scales = plain_quant(x, fmt, g)
        y = (values(codes, scales, fmt) * g)[:, :case["K"]].to(dtype)
        return {"y": y, "g": g} if fmt == "nv" else {"y": y}
    if case["op"] == "gemm":
        a, sa = state["a"], state["sa"]
    else:
        a, sa = plain_quant(state["x"], fmt, state["ga"])
    return {"y": plain_gemm(a, sa, state["ga"], state["w"], state["sw"], state["gw"], fmt, dtype)}


def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    bits = 0.5 + 1.0 / BLOCK[case["fmt"]]  # bytes of a quantised value with its share of the scale
    if case["op"] == "quant":
        n = case["rows"] * case["K"]
        # x is read and its quantised form written; reading back, that form is read and y written
        return {"bytes": n * (size[case["x"]] + 2 * bits + size[case["y"]]), "flops": 0}
    M, N, K = case["M"], case["N"], case["K"]
    x = M * K * (size[case["x"]] if case["op"] == "linear" else bits)
    return {"bytes": x + N * K * bits + M * N * size[case["y"]], "flops": 2 * M * N * K}


# ------------------------------------------------------------------ 64 bits

def exact_round(v):
    """e2m1 of v >= 0 by its spacing: 1/2 below 2, 1 below 4, then 2; saturates at 6."""
    step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0)).double()
    return (torch.round(v / step) * step).clamp(max=6.0)


def power_below(v):
    """2^floor(log2 v) of normal v > 0 in 64 bits: v without its mantissa."""
    return (v.view(torch.int64) & 0x7FF0000000000000).view(torch.float64)


def exact_values(x, fmt, inv):
    """What quantising x stands for, without the tensor scale, in 64 bits (z itself is defined in 32)."""
    rows, K = x.shape
    B = BLOCK[fmt]
    z = torch.zeros(rows, pad_up(K, B), dtype=torch.float64, device=x.device)
    z[:, :K] = (x.float() * inv).double()
    z = z.view(rows, -1, B)
    top = z.abs().amax(dim=2, keepdim=True)
    if fmt == "mx":
        s = (power_below(top.clamp(min=2.0 ** -160)) / 4).clamp(min=2.0 ** -127)
    else:
        t = (top / torch.full_like(top, 6.0)).clamp(max=448.0)
        step = power_below(t.clamp(min=2.0 ** -6)) / 8  # three mantissa bits, down to 2^-9
        s = torch.round(t / step) * step
    v = exact_round(z.abs() / torch.where(s > 0, s, 1.0)) * s * torch.sign(z)
    return v.view(rows, -1)[:, :K]


def exact(case, seed):
    d, fmt = inputs(case, seed), case["fmt"]
    if case["op"] == "quant":
        x = d["x"]
        if fmt != "nv":
            return {"y": exact_values(x, fmt, 1.0)}
        g = (x.double().abs().max() / torch.full((), 2688.0, dtype=torch.float64, device=x.device)).clamp(min=2.0 ** -126)
        g32 = g.float()  # what quantising takes
        return {"y": exact_values(x, fmt, torch.reciprocal(g32)) * g32.double(), "g": g.view(1)}
    a = exact_values(d["x"], fmt, 1.0 / d["ga"])
    w = exact_values(d["w"], fmt, 1.0 / d["gw"])
    return {"y": (a @ w.t()) * (d["ga"].double() * d["gw"].double())}
