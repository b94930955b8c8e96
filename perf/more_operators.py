"""Workloads of the operators around a quantised model's products: the root-mean-square
norm that makes the INT8 products' operand, its gradient, products of 16-bit activations
with group-scaled INT4 weights, and a mixture-of-experts layer of such weights.

INT4 weights of N rows of K values are (N, ceil(K/2)) bytes, two signed 4-bit values per
byte with the even k in the low nibble, and one scale per `group` consecutive k of a row,
stored by group: scales[g, n] belongs to group g of row n.  The value is code * scale.

Kinds of cases:
  norm      h = x + residual, and the norm of h: 16-bit or fp32, or INT8 with row scales
  gradient  the norm's gradients: of its input (with the residual stream's gradient added)
            and of its weight
  product   C = A * B of 16-bit activations and INT4 weights
  experts   a mixture-of-experts layer for a few tokens: the choice of experts from the
            router's logits, both products of the chosen experts, their weighted sum
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "i8": 1}
EPS = 1e-5


def listed():
    return [
        # one decoded token's residual stream, quantised for an INT8 projection
        {"name": "norm token", "kind": "norm", "rows": 1, "cols": 8192, "type": "bf16", "out": "i8", "residual": True},
        # a prefill's
        {"name": "norm prefill", "kind": "norm", "rows": 8192, "cols": 8192, "type": "f16", "out": "i8",
         "residual": True},
        # an fp32 stream of an odd width, no residual: a model's first norm
        {"name": "norm ragged", "kind": "norm", "rows": 2999, "cols": 5003, "type": "f32", "out": "bf16",
         "residual": False},
        # a training step's gradient through the norm
        {"name": "gradient", "kind": "gradient", "rows": 4096, "cols": 8192, "type": "bf16", "residual": True},
        # a small odd batch in fp32
        {"name": "gradient ragged", "kind": "gradient", "rows": 333, "cols": 2081, "type": "f32", "residual": False},
        # one decoded token against a layer's weights
        {"name": "product token", "kind": "product", "M": 1, "N": 8192, "K": 8192, "group": 128, "type": "bf16",
         "scales": "bf16", "out": "bf16"},
        # a few sequences, odd in every dimension, the shortest groups
        {"name": "product ragged", "kind": "product", "M": 5, "N": 2081, "K": 4133, "group": 32, "type": "f16",
         "scales": "f32", "out": "f32"},
        # an odd batch of decoded tokens
        {"name": "product batch", "kind": "product", "M": 37, "N": 4096, "K": 8192, "group": 64, "type": "f16",
         "scales": "f16", "out": "f16"},
        # a prefill
        {"name": "product prefill", "kind": "product", "M": 2048, "N": 8192, "K": 8192, "group": 128, "type": "bf16",
         "scales": "bf16", "out": "bf16"},
        # one decoded token through a layer of a few large experts
        {"name": "experts token", "kind": "experts", "T": 1, "H": 4096, "I": 2048, "E": 32, "top": 4, "group": 128,
         "type": "bf16", "scales": "bf16", "pad": 0},
        # a decode batch through many small experts
        {"name": "experts batch", "kind": "experts", "T": 16, "H": 2048, "I": 768, "E": 128, "top": 8, "group": 64,
         "type": "f16", "scales": "f16", "pad": 0},
        # a larger one, padded at its end with rows that have no expert, odd sizes
        {"name": "experts padded", "kind": "experts", "T": 61, "H": 2000, "I": 1001, "E": 60, "top": 6, "group": 32,
         "type": "bf16", "scales": "f32", "pad": 5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "gradient", "product", "experts"])
    case = {"kind": kind}
    if kind in ("norm", "gradient"):
        case |= {"rows": _log(rng, 1, 8192), "cols": _log(rng, 64, 8192), "type": rng.choice(["f32", "f16", "bf16"]),
                 "residual": rng.random() < 0.6}
        if kind == "norm":
            case["out"] = rng.choice(["i8", "i8", "f32", "f16", "bf16"])
        return case
    case |= {"group": rng.choice([32, 64, 128]), "type": rng.choice(["f16", "bf16"])}
    case["scales"] = rng.choice(["f32", case["type"]])
    if kind == "product":
        return case | {"M": _log(rng, 1, 2048), "N": _log(rng, 64, 8192), "K": _log(rng, 64, 8192),
                       "out": rng.choice(["f32", "f16", "bf16"])}
    E = rng.choice([8, 16, 32, 60, 128])
    H, I, T = _log(rng, 256, 4096), _log(rng, 64, 2048), _log(rng, 1, 64)
    while E * H * I > 1 << 28:
        E //= 2
    return case | {"T": T, "H": H, "I": I, "E": E, "top": rng.randint(1, min(8, E)),
                   "pad": rng.choice([0, 0, T // 3])}


# ---- plain forms: elementary operations in fp32 ----

def _plain_inverse(h):
    return torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS)


def _plain_norm(s):
    x, w, out = s["x"], s["w"].float(), s["out"]
    result = {}
    if s["residual"]:
        x = (x.float() + s["res"].float()).to(x.dtype)
        result["h"] = x
    h = x.float()
    t, r = h * w, _plain_inverse(h)
    if out == "i8":
        # the row's scale cancels in the codes
        m = t.abs().amax(dim=1, keepdim=True)
        result["q"] = torch.round(t * (127.0 / m)).to(torch.int8)
        result["scale"] = (m * r / 127.0)[:, 0]
    else:
        result["y"] = (t * r).to(TYPES[out])
    return result


def _plain_gradient(s):
    # y = h r w with r = (mean h^2 + eps)^-1/2:
    # dx = r (w dy - h r^2 mean(h w dy)), dw = sum over rows of dy h r
    h, dy, w = s["x"].float(), s["dy"].float(), s["w"].float()
    r = _plain_inverse(h)
    g = dy * w
    dx = r * (g - h * (r * r * (h * g).mean(dim=1, keepdim=True)))
    if s["residual"]:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * h * r).sum(dim=0)}


def _plain_weights(packed, scales, group, K):
    """fp32 values (..., N, K) of INT4 weights."""
    nibbles = torch.stack((packed & 15, packed >> 4), dim=-1).flatten(-2)[..., :K]
    codes = (nibbles ^ 8).float() - 8.0
    return codes * scales.float().transpose(-1, -2).repeat_interleave(group, dim=-1)[..., :K]


def _plain_product(s):
    return (s["x"].float() @ _plain_weights(s["b"], s["sb"], s["group"], s["K"]).t()).to(TYPES[s["out"]])


def _plain_route(logits, top):
    """The `top` largest logits of each row, ties to the lower index, and their softmax among
    themselves; an expert at -infinity is not taken."""
    value, index = torch.sort(logits.float(), dim=1, descending=True, stable=True)
    value, index = value[:, :top], index[:, :top]
    taken = value > -math.inf
    e = torch.where(taken, torch.exp(value - value[:, :1]), 0.0)
    weights = torch.where(taken, e / e.sum(dim=1, keepdim=True), 0.0)
    return torch.where(taken, index, -1).to(torch.int32), weights


def _plain_experts(s):
    H, I, E = s["H"], s["I"], s["E"]
    ids, weights = _plain_route(s["logits"], s["top"])
    x = s["x"].float()
    chosen = ids.unsqueeze(2) == torch.arange(E, device=ids.device)
    share = (chosen * weights.unsqueeze(2)).sum(dim=1)                         # (T, E)
    up = torch.matmul(x, _plain_weights(s["w13"], s["s13"], s["group"], H).transpose(1, 2))
    gate, up = up[..., :I], up[..., I:]
    act = gate / (1.0 + torch.exp(-gate)) * up                                 # (E, T, I)
    down = torch.matmul(act, _plain_weights(s["w2"], s["s2"], s["group"], I).transpose(1, 2))
    y = (down * share.t().unsqueeze(2)).sum(dim=0)
    return {"ids": ids, "weights": weights, "y": y.to(s["x"].dtype)}


# ---- inputs ----

def _up(x, m):
    return (x + m - 1) // m * m


def _activations(g, rows, cols):
    """Activations: normal values, channels of unequal spread, a few of them far out."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    spread = torch.exp(0.7 * torch.randn((cols,), generator=g, device="cuda"))
    return x * torch.where(torch.rand((cols,), generator=g, device="cuda") < 0.004, spread * 20, spread)


def _rows16(x):
    """x in a buffer whose rows span a multiple of 16 bytes, as the products take them."""
    rows, cols = x.shape
    buf = torch.zeros((rows, _up(cols, 16 // x.element_size())), dtype=x.dtype, device=x.device)
    buf[:, :cols] = x
    return buf[:, :cols]


def _weights(g, shape, K, group, scale_type):
    """INT4 codes (*shape, ceil(K/2)), spread as a normal weight's are, in rows of a multiple of
    16 bytes, and scales (..., groups, N)."""
    N, width = shape[-1], (K + 1) // 2
    codes = torch.randn(shape + (2 * width,), generator=g, device="cuda").mul_(2.6).round_().clamp_(-8, 7)
    codes = codes.to(torch.int8).view(torch.uint8) & 15
    packed = torch.zeros(shape + (_up(width, 16),), dtype=torch.uint8, device="cuda")
    packed[..., :width] = codes[..., 0::2] | (codes[..., 1::2] << 4)
    scales = torch.randn(shape[:-1] + ((K + group - 1) // group, N), generator=g, device="cuda")
    scales = 0.3 / math.sqrt(K) * torch.exp(0.3 * scales)
    return packed[..., :width], scales.to(TYPES[scale_type])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind, s = case["kind"], dict(case)
    dtype = TYPES[case["type"]]
    if kind in ("norm", "gradient"):
        rows, cols = case["rows"], case["cols"]
        s["x"] = _activations(g, rows, cols).to(dtype)
        s["w"] = (1.0 + 0.2 * torch.randn((cols,), generator=g, device="cuda")).to(dtype)
        if kind == "norm" and case["residual"]:
            s["res"] = _activations(g, rows, cols).to(dtype)
        if kind == "gradient":
            s["dy"] = (0.01 * torch.randn((rows, cols), generator=g, device="cuda")).to(dtype)
            if case["residual"]:
                s["dh"] = (0.01 * torch.randn((rows, cols), generator=g, device="cuda")).to(dtype)
        return s
    if kind == "product":
        s["x"] = _rows16(_activations(g, case["M"], case["K"]).to(dtype))
        s["b"], s["sb"] = _weights(g, (case["N"],), case["K"], case["group"], case["scales"])
        return s
    T, H, I, E = case["T"], case["H"], case["I"], case["E"]
    s["x"] = _rows16(torch.randn((T, H), generator=g, device="cuda").to(dtype))
    logits = 2.0 * torch.randn((T, E), generator=g, device="cuda")
    if case["pad"]:
        logits[T - case["pad"]:] = -math.inf
    s["logits"] = logits
    s["w13"], s["s13"] = _weights(g, (E, 2 * I), H, case["group"], case["scales"])
    s["w2"], s["s2"] = _weights(g, (E, H), I, case["group"], case["scales"])
    return s


# ---- one pass ----

def run(state):
    if own:
        return _run_own(state)
    plain = {"norm": _plain_norm, "gradient": _plain_gradient, "product": _plain_product, "experts": _plain_experts}
    return plain[state["kind"]](state)


def _run_own(s):
    import precision_dense_gemm_amd as pd

    kind = s["kind"]
    if kind == "norm":
        if s["out"] == "i8":
            got = pd.rms_norm_i8(s["x"], s["w"], EPS, residual=s.get("res"))
            names = ("q", "scale", "h")
        else:
            got = pd.rms_norm(s["x"], s["w"], EPS, residual=s.get("res"), out_dtype=TYPES[s["out"]])
            names = ("y", "h")
            got = got if s["residual"] else (got,)
        return dict(zip(names, got))
    if kind == "gradient":
        dx, dw = pd.rms_norm_backward(s["dy"], s["x"], s["w"], EPS, dh=s.get("dh"))
        return {"dx": dx, "dw": dw}
    if kind == "product":
        return pd.gemm_a16_i4(s["x"], s["b"], s["sb"], s["group"], out_dtype=TYPES[s["out"]])
    ids, weights = pd.moe_route(s["logits"], s["top"])
    y = pd.moe_a16_i4(s["x"], ids, weights, s["w13"], s["s13"], s["w2"], s["s2"], s["group"])
    return {"ids": ids, "weights": weights, "y": y}


# ---- what a pass cannot do without ----

def work(case):
    kind = case["kind"]
    if kind in ("norm", "gradient"):
        n, size = case["rows"] * case["cols"], SIZE[case["type"]]
        moved = case["cols"] * size
        if kind == "norm":   # x, the result; the residual and the sum
            moved += n * (size + SIZE[case["out"]]) + (2 * n * size if case["residual"] else 0)
            moved += 4 * case["rows"] if case["out"] == "i8" else 0
            return {"bytes": moved, "flops": 5 * n}
        moved += n * size * (4 if case["residual"] else 3) + 4 * case["cols"]
        return {"bytes": moved, "flops": 12 * n}

    def stored(N, K):
        return N * ((K + 1) // 2) + N * ((K + case["group"] - 1) // case["group"]) * SIZE[case["scales"]]

    if kind == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * K + stored(N, K) + M * N * SIZE[case["out"]], "flops": 2 * M * N * K}
    H, I, E, top, live = case["H"], case["I"], case["E"], case["top"], case["T"] - case["pad"]
    # experts that some token takes, on average over routers that favour none
    taken = E * (1.0 - (1.0 - top / E) ** live)
    return {"bytes": taken * (stored(2 * I, H) + stored(H, I)) + 4 * case["T"] * H + 4 * case["T"] * E,
            "flops": 6 * live * top * H * I}


# ---- the definition in 64 bits, written apart from the plain forms ----

def _exact_weights(packed, scales, group, K):
    k = torch.arange(K, device=packed.device)
    nibble = (packed[..., k // 2].to(torch.int16) >> (4 * (k % 2)).to(torch.int16)) & 15
    code = torch.where(nibble > 7, nibble - 16, nibble).double()
    return code * scales.double()[..., k // group, :].transpose(-1, -2)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "norm":
        out = {}
        h = s["x"].double()
        if case["residual"]:
            # (a sum of two 16-bit values is exact in 64 bits, and so rounded once)
            out["h"] = (h + s["res"].double()).to(s["x"].dtype).double()
            h = out["h"]
        root = torch.sqrt(h.pow(2).sum(dim=1) / case["cols"] + EPS).unsqueeze(1)
        y = h / root * s["w"].double()
        if case["out"] == "i8":
            return out | {"q": None, "scale": y.abs().amax(dim=1) / 127.0}
        return out | {"y": y}
    if kind == "gradient":
        h, dy, w = s["x"].double(), s["dy"].double(), s["w"].double()
        root = torch.sqrt(h.pow(2).sum(dim=1, keepdim=True) / case["cols"] + EPS)
        n = h / root                                   # d(n)/d(h) = (1 - n n^T / cols) / root
        g = w * dy
        dx = (g - n * (g * n).sum(dim=1, keepdim=True) / case["cols"]) / root
        return {"dx": dx + s["dh"].double() if case["residual"] else dx, "dw": (dy * n).sum(dim=0)}
    group = case["group"]
    if kind == "product":
        return torch.matmul(s["x"].double(), _exact_weights(s["b"], s["sb"], group, case["K"]).t())
    T, H, I, top = case["T"], case["H"], case["I"], case["top"]
    x, logits = s["x"].double(), s["logits"].double()
    y, weights = torch.zeros_like(x), torch.zeros((T, top), dtype=torch.float64, device=x.device)
    order = logits.argsort(dim=1, descending=True, stable=True)[:, :top]
    live = T - case["pad"]
    if live:
        weights[:live] = torch.softmax(logits[:live].gather(1, order[:live]), dim=1)
    for e in range(case["E"]):
        t, slot = torch.nonzero(order[:live] == e, as_tuple=True)
        if t.numel() == 0:
            continue
        both = torch.matmul(x[t], _exact_weights(s["w13"][e], s["s13"][e], group, H).t())
        act = both[:, :I] * torch.sigmoid(both[:, :I]) * both[:, I:]
        y[t] += weights[t, slot].unsqueeze(1) * torch.matmul(act, _exact_weights(s["w2"][e], s["s2"][e], group, I).t())
    return {"ids": None, "weights": weights, "y": y}
