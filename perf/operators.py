"""Workloads of the MXFP4 operators: quantising, multiplying and training with
microscaled 4-bit floating point.

An MXFP4 operand of `rows` rows of K values is a pair: packed e2m1 codes, (rows, K/2)
bytes with the even k in the low nibble, rows of a multiple of 16 bytes; and e8m0
block scales, one byte (exponent + 127) per 32 values of K, stored by block:
scales[b, i] belongs to block b of row i, rows of a multiple of 16 bytes.

Kinds of cases:
  roundtrip  quantise a tensor (and, for training, its transpose in the same call), and
             read the values back
  product    C = A * B of two MXFP4 operands
  a16        C = A * B of 16-bit activations and MXFP4 weights
  train      one step of a linear layer: forward product, gradients of its input and of
             its weight, every product in MXFP4
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one decoded token's activations
        {"name": "roundtrip token", "kind": "roundtrip", "rows": 1, "K": 4096, "type": "bf16",
         "both": False, "rule": "floor", "out": "bf16"},
        # a prefill's activations
        {"name": "roundtrip prefill", "kind": "roundtrip", "rows": 8192, "K": 8192, "type": "f16",
         "both": False, "rule": "floor", "out": "bf16"},
        # fp32 master weights of an odd shape, scales that never saturate
        {"name": "roundtrip ragged master", "kind": "roundtrip", "rows": 2999, "K": 5003, "type": "f32",
         "both": False, "rule": "fit", "out": "f32"},
        # a training tensor: both contraction axes from one read
        {"name": "roundtrip both axes", "kind": "roundtrip", "rows": 4096, "K": 8192, "type": "bf16",
         "both": True, "rule": "floor", "out": "bf16"},
        # one decoded token against a layer's weights
        {"name": "product token", "kind": "product", "M": 1, "N": 8192, "K": 8192, "out": "bf16"},
        # a short batch of decoded sequences, odd in every dimension
        {"name": "product ragged", "kind": "product", "M": 333, "N": 2081, "K": 4133, "out": "f32"},
        # a prefill chunk
        {"name": "product chunk", "kind": "product", "M": 1024, "N": 8192, "K": 8192, "out": "f16"},
        # the largest product of the library's own sweep
        {"name": "product 8192", "kind": "product", "M": 8192, "N": 8192, "K": 8192, "out": "f32"},
        # decoding with 16-bit activations: one sequence, then an odd batch
        {"name": "a16 token", "kind": "a16", "M": 1, "N": 8192, "K": 8192, "type": "bf16", "out": "bf16"},
        {"name": "a16 batch", "kind": "a16", "M": 37, "N": 4096, "K": 8192, "type": "f16", "out": "f32"},
        # a prefill with 16-bit activations
        {"name": "a16 prefill", "kind": "a16", "M": 2048, "N": 8192, "K": 8192, "type": "bf16", "out": "bf16"},
        # a training step of one layer, tokens of ragged sequences packed together
        {"name": "train step", "kind": "train", "M": 4001, "N": 4096, "K": 4096, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["roundtrip", "product", "a16", "train"])
    if kind == "roundtrip":
        return {"kind": kind, "rows": _log(rng, 1, 8192), "K": _log(rng, 17, 8192),
                "type": rng.choice(["f32", "f16", "bf16"]), "both": rng.random() < 0.4,
                "rule": rng.choice(["floor", "fit"]), "out": rng.choice(["f32", "bf16"])}
    if kind == "product":
        return {"kind": kind, "M": _log(rng, 1, 8192), "N": _log(rng, 17, 8192), "K": _log(rng, 33, 8192),
                "out": rng.choice(["f32", "f16", "bf16"])}
    if kind == "a16":
        return {"kind": kind, "M": _log(rng, 1, 4096), "N": _log(rng, 17, 8192), "K": _log(rng, 33, 8192),
                "type": rng.choice(["f16", "bf16"]), "out": rng.choice(["f32", "f16", "bf16"])}
    return {"kind": kind, "M": _log(rng, 15, 4096), "N": _log(rng, 64, 4096), "K": _log(rng, 64, 4096),
            "type": rng.choice(["f16", "bf16"])}


def _up(x, m):
    return (x + m - 1) // m * m


# ---- plain forms: elementary operations in fp32 ----

def _scaled(x, e):
    """fp32 x * 2^e for integers e in [-252, 252], by two exact powers of two made from their
    bits (a power function need not return them exactly)."""
    h = torch.div(e, 2, rounding_mode="floor")
    lower = ((h.to(torch.int32) + 127) << 23).view(torch.float32)
    upper = (((e - h).to(torch.int32) + 127) << 23).view(torch.float32)
    return x * lower * upper


def _plain_quantize(x, rule):
    """(codes, exponents) of fp32 rows x (rows, K): e2m1 codes (rows, blocks, 32) with the
    sign in bit 3, and the blocks' exponents (rows, blocks).  K is padded with zeros."""
    rows, K = x.shape
    blocks = (K + 31) // 32
    padded = torch.zeros((rows, blocks * 32), dtype=torch.float32, device=x.device)
    padded[:, :K] = x
    v = padded.view(rows, blocks, 32)
    mant, ex = torch.frexp(v.abs().amax(dim=2))        # amax = mant * 2^ex, mant in [0.5, 1)
    e = ex - 3
    if rule == "fit":
        e = e + (mant > 0.75).to(e.dtype)
    e = torch.where(mant == 0, torch.full_like(e, -127), e.clamp(min=-127))
    s = _scaled(v, -e.unsqueeze(2))
    a = s.abs()
    # codes passed on the way up; a value halfway goes to the even code
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5)
            + (a > 5.0))
    return code + 8 * (s < 0).to(torch.uint8), e


def _plain_values(code, e, K):
    """fp32 values (rows, K) of codes (rows, blocks, 32) and exponents (rows, blocks)."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=code.device)
    v = _scaled(table[code.to(torch.int64)], e.unsqueeze(2))
    return v.view(code.shape[0], -1)[:, :K]


def _plain_unpack(packed, scales, K):
    """fp32 values (rows, K) of a stored operand."""
    rows, blocks = packed.shape[0], (K + 31) // 32
    code = torch.stack((packed & 15, packed >> 4), dim=2).view(rows, blocks, 32)
    return _plain_values(code, scales[:, :rows].t().to(torch.int32) - 127, K)


def _plain_product(a, b, out):
    """a (M, K) times b (N, K) transposed, fp32, rounded once."""
    return (a @ b.t()).to(TYPES[out])


# ---- inputs ----

def _store(x, rule="floor"):
    """The stored operand (packed, scales) of fp32 rows, as the library keeps it."""
    code, e = _plain_quantize(x, rule)
    rows, blocks = e.shape
    flat = code.view(rows, blocks * 32)
    packed = flat[:, 0::2] | (flat[:, 1::2] << 4)
    scales = torch.zeros((blocks, _up(rows, 16)), dtype=torch.uint8, device=x.device)
    scales[:, :rows] = (e + 127).t().to(torch.uint8)
    return packed.contiguous(), scales


def _activations(g, rows, K, dtype):
    """Activations: normal values, channels of unequal spread, a few of them far out."""
    x = torch.randn((rows, K), generator=g, device="cuda")
    spread = torch.exp(0.7 * torch.randn((K,), generator=g, device="cuda"))
    spread = torch.where(torch.rand((K,), generator=g, device="cuda") < 0.004, spread * 20, spread)
    return (x * spread).to(dtype)


def _rows16(x):
    """x in a buffer whose rows span a multiple of 16 bytes, as the library takes them."""
    rows, K = x.shape
    buf = torch.zeros((rows, _up(K, 16 // x.element_size())), dtype=x.dtype, device=x.device)
    buf[:, :K] = x
    return buf[:, :K]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind = case["kind"]
    state = dict(case)
    if kind == "roundtrip":
        state["x"] = _rows16(_activations(g, case["rows"], case["K"], TYPES[case["type"]]))
        return state
    M, N, K = case["M"], case["N"], case["K"]
    x = _activations(g, M, K, torch.float32)
    w = 0.02 * torch.randn((N, K), generator=g, device="cuda")
    if kind == "product":
        state["a"], state["sa"] = _store(x)
        state["b"], state["sb"] = _store(w)
    elif kind == "a16":
        state["x"] = _rows16(x.to(TYPES[case["type"]]))
        state["b"], state["sb"] = _store(w)
    else:
        state["x"] = _rows16(x.to(TYPES[case["type"]]))
        state["w"] = _rows16(w.to(TYPES[case["type"]]))
        grad = 0.01 * torch.randn((M, N), generator=g, device="cuda")
        state["g"] = _rows16(grad.to(TYPES[case["type"]]))
    return state


# ---- one pass ----

def run(state):
    if own:
        return _run_own(state)
    kind = state["kind"]
    if kind == "roundtrip":
        x, rule = state["x"].float(), state["rule"]
        rows, K = x.shape
        out = {"values": _plain_values(*_plain_quantize(x, rule), K).to(TYPES[state["out"]])}
        if state["both"]:
            out["values_t"] = _plain_values(*_plain_quantize(x.t(), rule), rows).to(TYPES[state["out"]])
        return out
    K = state["K"]
    if kind == "product":
        return _plain_product(_plain_unpack(state["a"], state["sa"], K), _plain_unpack(state["b"], state["sb"], K),
                              state["out"])
    if kind == "a16":
        return _plain_product(state["x"].float(), _plain_unpack(state["b"], state["sb"], K), state["out"])
    x, w, grad = state["x"].float(), state["w"].float(), state["g"].float()

    def quantized(t):
        return _plain_values(*_plain_quantize(t, "floor"), t.shape[1])

    return {"y": _plain_product(quantized(x), quantized(w), state["type"]),
            "dx": _plain_product(quantized(grad), quantized(w.t()), state["type"]),
            "dw": _plain_product(quantized(grad.t()), quantized(x.t()), "f32")}


def _run_own(state):
    import precision_dense_gemm_amd as pd

    kind = state["kind"]
    if kind == "roundtrip":
        x, out = state["x"], TYPES[state["out"]]
        rows, K = x.shape
        if state["both"]:
            (q, s), (qt, st) = pd.mxf4_quantize_both(x, scale_rule=state["rule"])
            return {"values": pd.mxf4_dequantize(q, s, K, out_dtype=out),
                    "values_t": pd.mxf4_dequantize(qt, st, rows, out_dtype=out)}
        q, s = pd.mxf4_quantize(x, scale_rule=state["rule"])
        return {"values": pd.mxf4_dequantize(q, s, K, out_dtype=out)}
    K = state["K"]
    if kind == "product":
        return pd.gemm_mxf4(state["a"], state["sa"], state["b"], state["sb"], K, out_dtype=TYPES[state["out"]])
    if kind == "a16":
        return pd.gemm_a16_mxf4(state["x"], state["b"], state["sb"], out_dtype=TYPES[state["out"]])
    M, N = state["M"], state["N"]
    out = TYPES[state["type"]]
    (x, sx), (xt, sxt) = pd.mxf4_quantize_both(state["x"])
    (w, sw), (wt, swt) = pd.mxf4_quantize_both(state["w"])
    (g, sg), (gt, sgt) = pd.mxf4_quantize_both(state["g"])
    return {"y": pd.gemm_mxf4(x, sx, w, sw, K, out_dtype=out),
            "dx": pd.gemm_mxf4(g, sg, wt, swt, N, out_dtype=out),
            "dw": pd.gemm_mxf4(gt, sgt, xt, sxt, M)}


# ---- what a pass cannot do without ----

def work(case):
    kind = case["kind"]

    def stored(rows, K):
        return rows * ((K + 1) // 2) + rows * ((K + 31) // 32)

    if kind == "roundtrip":
        n, o = case["rows"] * case["K"], SIZE[case["out"]]
        return {"bytes": n * SIZE[case["type"]] + n * o * (2 if case["both"] else 1), "flops": 0}
    M, N, K = case["M"], case["N"], case["K"]
    if kind == "product":
        return {"bytes": stored(M, K) + stored(N, K) + M * N * SIZE[case["out"]], "flops": 2 * M * N * K}
    if kind == "a16":
        return {"bytes": 2 * M * K + stored(N, K) + M * N * SIZE[case["out"]], "flops": 2 * M * N * K}
    return {"bytes": 2 * (M * K + N * K + M * N) + 2 * (M * N + M * K) + 4 * N * K, "flops": 6 * M * N * K}


# ---- the definition in 64 bits, written apart from the plain forms ----

def _pow2(e):
    """fp64 2^e of whole-numbered e in [-1022, 1023], from its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_quantized(x, rule):
    """fp64 values that rows x (rows, K) have in MXFP4, by arithmetic on the values."""
    rows, K = x.shape
    x = torch.nn.functional.pad(x.double(), (0, -K % 32)).reshape(rows, -1, 32)
    top = x.abs().amax(dim=2, keepdim=True)
    # floor(log2 top): the logarithm's floor, put right where it lands beside a power of two
    safe = torch.where(top > 0, top, torch.ones_like(top))
    f = torch.floor(torch.log2(safe))
    f = torch.where(_pow2(f) > safe, f - 1, torch.where(_pow2(f + 1) <= safe, f + 1, f))
    e = f - 2
    if rule == "fit":
        e = torch.where(6.0 * _pow2(e) < safe, e + 1, e)
    scale = _pow2(e.clamp(min=-127))
    y = x / scale
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    y = torch.sign(y) * (torch.round(a / step) * step).clamp(max=6.0)   # torch.round: ties to even
    return (y * scale * (top > 0)).reshape(rows, -1)[:, :K]


def _exact_stored(packed, scales, K):
    """fp64 values of a stored operand, from the bits of each code."""
    k = torch.arange(K, device=packed.device)
    nib = (packed[:, k // 2].to(torch.int64) >> (4 * (k % 2))) & 15
    exponent, mantissa = (nib >> 1) & 3, (nib & 1).double()
    mag = torch.where(exponent == 0, mantissa / 2, (1 + mantissa / 2) * _pow2(exponent - 1))
    sign = 1.0 - 2.0 * (nib >> 3).double()
    byte = scales[k // 32][:, :packed.shape[0]].t().to(torch.int64)
    return sign * mag * _pow2(byte - 127)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "roundtrip":
        out = {"values": _exact_quantized(s["x"], case["rule"])}
        if case["both"]:
            out["values_t"] = _exact_quantized(s["x"].t().contiguous(), case["rule"])
        return out
    K = case["K"]
    if kind == "product":
        return torch.matmul(_exact_stored(s["a"], s["sa"], K), _exact_stored(s["b"], s["sb"], K).t())
    if kind == "a16":
        return torch.matmul(s["x"].double(), _exact_stored(s["b"], s["sb"], K).t())
    x, w, g = s["x"], s["w"], s["g"]
    q = lambda t: _exact_quantized(t.contiguous(), "floor")  # noqa: E731
    return {"y": torch.matmul(q(x), q(w).t()), "dx": torch.matmul(q(g), q(w.t()).t()),
            "dw": torch.matmul(q(g.t()), q(x.t()).t())}
