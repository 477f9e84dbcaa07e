"""The operators on 4-bit microscaled (MX) values and the mixture-of-experts layer, as cases to be measured.

An MX row holds K values in blocks of 32 along K: 4-bit codes (sign, two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3,
4, 6 and their negatives; two to a byte, the lower nibble first) and one scale byte per block that stands for 2^(byte - 127).

  "roundtrip"  a matrix is quantised, its blocks along its rows or down its columns, and the values are read back
  "product"    C = A B^T, both operands MX rows, blocks along the shared dimension
  "a16"        C = A B^T, A rows of bf16 or fp16, B MX rows: weights in 4 bits, few rows of activations
  "moe"        router, top-k, gated experts and their weighted sum for a few tokens; weights in 16 bits or MX

`own` false: the plain forms, in elementary torch operations and 32 bits.  `own` true: the package's operators.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = 32


def listed():
    return [
        # A decode step's activations, quantised on their way into a product: what counts is the latency.
        {"name": "roundtrip 16 rows", "op": "roundtrip", "rows": 16, "k": 4096, "type": "bf16", "along": "rows"},
        # A layer's fp32 weights (K x N, as the products take them), quantised once when a model is loaded; no size a multiple of 32.
        {"name": "roundtrip weight columns", "op": "roundtrip", "rows": 16383, "k": 8191, "type": "f32", "along": "columns"},
        # A small batch through a long contraction: the weights are read once.
        {"name": "product 32 rows", "op": "product", "m": 32, "n": 4096, "k": 16384, "c": "bf16"},
        # The benchmark's square product.
        {"name": "product 4096 cube", "op": "product", "m": 4096, "n": 4096, "k": 4096, "c": "f32"},
        # The benchmark's ragged product: no dimension a multiple of any tile or block.
        {"name": "product ragged", "op": "product", "m": 4097, "n": 4095, "k": 2049, "c": "bf16"},
        # A prompt or training batch through a wide layer.
        {"name": "product 8192 cube", "op": "product", "m": 8192, "n": 8192, "k": 8192, "c": "bf16"},
        # One token.
        {"name": "a16 one row", "op": "a16", "m": 1, "n": 4096, "k": 4096, "type": "bf16", "c": "bf16"},
        # An odd batch and odd sizes.
        {"name": "a16 17 rows ragged", "op": "a16", "m": 17, "n": 4095, "k": 2049, "type": "f16", "c": "f16"},
        # The widest batch of single tokens, through a wide layer.
        {"name": "a16 64 rows", "op": "a16", "m": 64, "n": 16384, "k": 8192, "type": "bf16", "c": "f32"},
        # One token through a layer of many small experts.
        {"name": "moe one token mx", "op": "moe", "t": 1, "e": 64, "top": 8, "h": 2048, "i": 1024, "type": "bf16", "w": "mx", "renorm": True},
        # A few tokens, few experts in 16 bits, odd sizes.
        {"name": "moe 16 tokens ragged", "op": "moe", "t": 16, "e": 8, "top": 2, "h": 2049, "i": 4095, "type": "f16", "w": "f16", "renorm": False},
        # A full batch of single tokens: every expert is asked.
        {"name": "moe 64 tokens mx", "op": "moe", "t": 64, "e": 64, "top": 4, "h": 4096, "i": 1024, "type": "bf16", "w": "mx", "renorm": True},
    ]


def _size(rng, low, high):
    """A size between low and high, even over the logarithm; half of them as drawn, half rounded to a multiple of 32."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if rng.random() < 0.5 and n >= 48:
        n = min(high, 32 * ((n + 16) // 32))
    return max(low, min(high, n))


def draw(rng):
    op = rng.choice(("roundtrip", "product", "a16", "moe"))
    while True:
        if op == "roundtrip":
            c = {"op": op, "rows": _size(rng, 1, 16384), "k": _size(rng, 32, 16384), "type": rng.choice(("bf16", "f16", "f32")),
                 "along": rng.choice(("rows", "columns"))}
            if c["rows"] * c["k"] <= 16383 * 8191:
                return c
        elif op == "product":
            c = {"op": op, "m": _size(rng, 1, 8192), "n": _size(rng, 16, 8192), "k": _size(rng, 32, 16384), "c": rng.choice(("bf16", "f16", "f32"))}
            if c["m"] * c["n"] * c["k"] <= 8192 ** 3:
                return c
        elif op == "a16":
            t = rng.choice(("bf16", "f16"))
            return {"op": op, "m": rng.randint(1, 64), "n": _size(rng, 16, 16384), "k": _size(rng, 32, 8192), "type": t, "c": rng.choice((t, "f32"))}
        else:
            t, e = rng.choice(("bf16", "f16")), _size(rng, 4, 128)
            c = {"op": op, "t": rng.choice((1, rng.randint(2, 8), rng.randint(9, 64))), "e": e, "top": rng.randint(1, min(8, e)), "h": _size(rng, 64, 4096),
                 "i": _size(rng, 32, 4096), "type": t, "w": rng.choice((t, "mx")), "renorm": rng.random() < 0.5}
            if c["e"] * c["h"] * c["i"] <= 64 * 4096 * 1024:
                return c


# ---- inputs ---------------------------------------------------------------


def _blocks(k):
    return (k + BLOCK - 1) // BLOCK


def _weights(g, lead, k):
    """MX weights: rows of `lead`, K values each.  Codes as quantised normal values have them, scales spread over some octaves, the last
    block's codes zero past K, one block in 64 all zero.  Scale rows are padded to whole 16 bytes."""
    nb = _blocks(k)
    nib = (torch.randn(lead + (nb * BLOCK,), generator=g, device="cuda") * 2.4).round_().abs_().clamp_(max=7).to(torch.uint8)
    nib += torch.randint(0, 2, nib.shape, generator=g, device="cuda", dtype=torch.uint8) * 8
    nib[..., k:] = 0
    rare = torch.rand(lead + (nb, 1), generator=g, device="cuda") < 1 / 64
    nib = nib.reshape(lead + (nb, BLOCK)).masked_fill_(rare, 0).reshape(lead + (nb * BLOCK,))
    codes = nib[..., 0::2] | (nib[..., 1::2] << 4)
    scales = torch.zeros(lead + (16 * ((nb + 15) // 16),), dtype=torch.uint8, device="cuda")
    mid = 126 - int(round(math.log2(max(k, 4)) / 2))
    scales[..., :nb] = torch.randint(mid - 2, mid + 2, lead + (nb,), generator=g, device="cuda", dtype=torch.uint8)
    return codes.contiguous(), scales


def _activations(g, shape, dtype):
    """Normal values with a few large channels."""
    x = torch.randn(shape, generator=g, device="cuda")
    loud = torch.rand(shape[-1], generator=g, device="cuda") < 1 / 128
    return (x * (1 + 15 * loud)).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "roundtrip":
        shape = (case["rows"], case["k"]) if case["along"] == "rows" else (case["k"], case["rows"])
        s["x"] = _activations(g, shape, TYPES[case["type"]])
    elif case["op"] == "product":
        s["a"] = _weights(g, (case["m"],), case["k"])
        s["b"] = _weights(g, (case["n"],), case["k"])
    elif case["op"] == "a16":
        s["a"] = _activations(g, (case["m"], case["k"]), TYPES[case["type"]])
        s["b"] = _weights(g, (case["n"],), case["k"])
    else:
        e, h, i, dtype = case["e"], case["h"], case["i"], TYPES[case["type"]]
        s["x"] = torch.randn((case["t"], h), generator=g, device="cuda").to(dtype)
        s["router"] = (torch.randn((e, h), generator=g, device="cuda") / math.sqrt(h)).to(dtype)
        if case["w"] == "mx":
            s["w1"] = _weights(g, (e, 2 * i), h)
            s["w2"] = _weights(g, (e, h), i)
        else:
            s["w1"] = (torch.randn((e, 2 * i, h), generator=g, device="cuda") / math.sqrt(h)).to(dtype)
            s["w2"] = (torch.randn((e, h, i), generator=g, device="cuda") / math.sqrt(i)).to(dtype)
    return s


# ---- the plain forms --------------------------------------------------------

VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
VALUES += [-v for v in VALUES]
_tables = {}


def _table():
    """The two values of each byte, on the current device."""
    d = torch.cuda.current_device()
    if d not in _tables:
        _tables[d] = torch.tensor([[VALUES[b & 15], VALUES[b >> 4]] for b in range(256)], device="cuda")
    return _tables[d]


def _decode(q, k):
    """The fp32 values of MX rows."""
    codes, scales = q
    nb = _blocks(k)
    v = _table()[codes[..., : 16 * nb].int()].reshape(codes.shape[:-1] + (nb, BLOCK))
    v = v * torch.exp2(scales[..., :nb].float() - 127).unsqueeze(-1)
    return v.reshape(codes.shape[:-1] + (nb * BLOCK,))[..., :k]


def _plain_roundtrip(s):
    x = s["x"].float()
    if s["along"] == "columns":
        x = x.t()
    rows, k = x.shape
    nb = _blocks(k)
    x = torch.nn.functional.pad(x, (0, nb * BLOCK - k)).reshape(rows, nb, BLOCK)
    # 2^(floor(log2 of the block's largest) - 2): the largest lands in [4, 8), at or past the largest code's octave
    amax = x.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 3, -127).clamp(-127, 127)
    a = torch.ldexp(x, -e)
    m = a.abs()
    # nearest, ties to the even code
    m = 0.5 * ((m > 0.25).float() + (m >= 0.75) + (m > 1.25) + (m >= 1.75)) + (m > 2.5).float() + (m >= 3.5) + 2.0 * (m > 5)
    v = torch.ldexp(torch.copysign(m, a), e).reshape(rows, nb * BLOCK)[:, :k]
    v = v.to(TYPES["bf16" if s["type"] == "bf16" else "f32"])
    return v if s["along"] == "rows" else v.t().contiguous()


def _plain_moe(s):
    x, top, h, i = s["x"].float(), s["top"], s["h"], s["i"]
    # the choice of experts: values next to a border, so in 64 bits; ties go to the lowest index
    p = torch.softmax(s["x"].double() @ s["router"].double().t(), -1)
    order = torch.sort(p, dim=-1, descending=True, stable=True)
    ids, gates = order.indices[:, :top], order.values[:, :top]
    if s["renorm"]:
        gates = gates / gates.sum(-1, keepdim=True)
    gates = gates.float()
    mx = s["w"] == "mx"
    t, e = x.shape[0], s["e"]
    if t * top <= e:  # fewer choices than experts: their weights alone
        pick = ids.reshape(-1)
        w1 = _decode((s["w1"][0][pick], s["w1"][1][pick]), h) if mx else s["w1"][pick].float()
        u = torch.matmul(w1, x.repeat_interleave(top, 0).unsqueeze(-1)).squeeze(-1)
        u = u[:, :i] * torch.sigmoid(u[:, :i]) * u[:, i:]
        w2 = _decode((s["w2"][0][pick], s["w2"][1][pick]), i) if mx else s["w2"][pick].float()
        y = torch.matmul(w2, u.unsqueeze(-1)).squeeze(-1)
        y = (y.reshape(t, top, h) * gates.unsqueeze(-1)).sum(1)
    else:  # every expert on every token, the unasked ones with weight 0
        share = torch.zeros((t, e), device=x.device).scatter_(1, ids, gates)
        w1 = _decode(s["w1"], h) if mx else s["w1"].float()
        u = torch.matmul(x.unsqueeze(0), w1.transpose(1, 2))
        u = u[..., :i] * torch.sigmoid(u[..., :i]) * u[..., i:]
        w2 = _decode(s["w2"], i) if mx else s["w2"].float()
        y = torch.matmul(u * share.t().unsqueeze(-1), w2.transpose(1, 2)).sum(0)
    return y.to(s["x"].dtype), ids.int(), gates


def run(state):
    s = state
    if own:
        import tiled_fp32_gemm_03_amd as g

        if s["op"] == "roundtrip":
            q = g.mx_quantize(s["x"], along=s["along"])
            return g.mx_dequantize(q, dtype=TYPES["bf16" if s["type"] == "bf16" else "f32"], along=s["along"])
        if s["op"] == "product":
            return g.matmul_mx(g.MxTensor(*s["a"], s["k"]), g.MxTensor(*s["b"], s["k"]), dtype=TYPES[s["c"]])
        if s["op"] == "a16":
            return g.matmul_mx(s["a"], g.MxTensor(*s["b"], s["k"]), dtype=TYPES[s["c"]])
        mx = s["w"] == "mx"
        w1 = g.MxTensor(*s["w1"], s["h"]) if mx else s["w1"]
        w2 = g.MxTensor(*s["w2"], s["i"]) if mx else s["w2"]
        return g.moe_layer(s["x"], s["router"], w1, w2, s["top"], renormalize=s["renorm"])
    if s["op"] == "roundtrip":
        return _plain_roundtrip(s)
    if s["op"] == "product":
        return torch.matmul(_decode(s["a"], s["k"]), _decode(s["b"], s["k"]).t()).to(TYPES[s["c"]])
    if s["op"] == "a16":
        return torch.matmul(s["a"].float(), _decode(s["b"], s["k"]).t()).to(TYPES[s["c"]])
    return _plain_moe(s)


# ---- what cannot be done without --------------------------------------------


def work(case):
    width = {"bf16": 2, "f16": 2, "f32": 4}
    mx = lambda rows, k: rows * _blocks(k) * 17  # noqa: E731  16 bytes of codes and one of scale per block
    if case["op"] == "roundtrip":
        n = case["rows"] * case["k"]
        return {"bytes": n * (width[case["type"]] + (2 if case["type"] == "bf16" else 4)), "flops": 4 * n}
    if case["op"] in ("product", "a16"):
        m, n, k = case["m"], case["n"], case["k"]
        a = mx(m, k) if case["op"] == "product" else m * k * 2
        return {"bytes": a + mx(n, k) + m * n * width[case["c"]], "flops": 2 * m * n * k}
    t, e, top, h, i = (case[x] for x in ("t", "e", "top", "h", "i"))
    asked = e * (1 - (1 - top / e) ** t)  # experts that at least one token asks, for even routing
    each = mx(2 * i, h) + mx(h, i) if case["w"] == "mx" else 3 * i * h * 2
    return {"bytes": asked * each + e * h * 2 + 2 * t * h * 2 + t * top * 8, "flops": 6 * t * top * h * i + 2 * t * e * h}


# ---- the definitions in 64 bits -----------------------------------------------


def _exact_values(q, k):
    codes, scales = q
    low, high = codes & 15, codes >> 4
    nib = torch.stack((low, high), -1).flatten(-2).long()
    ex, man = (nib >> 1) & 3, (nib & 1).double()
    mag = torch.where(ex > 0, (1 + man / 2) * torch.pow(2.0, ex.double() - 1), man / 2)
    v = torch.where(nib >= 8, -mag, mag)
    octave = torch.pow(2.0, scales.double() - 127).repeat_interleave(BLOCK, -1)
    return v[..., :k] * octave[..., :k]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "roundtrip":
        x = s["x"].double()
        x = x if case["along"] == "rows" else x.t()
        out = torch.empty_like(x)
        for b in range(_blocks(x.shape[1])):
            w = x[:, b * BLOCK:(b + 1) * BLOCK]
            top = w.abs().max(1, keepdim=True).values
            unit = torch.pow(2.0, torch.where(top > 0, torch.floor(torch.log2(top)) - 2, -127).clamp(-127, 127))
            z = w / unit
            # spacing of the codes around z: 0.5 below 2, then 1, then 2; half-way values to the even multiple
            gap = torch.where(z.abs() < 2, 0.5, torch.where(z.abs() < 4, 1.0, 2.0)).double()
            out[:, b * BLOCK:(b + 1) * BLOCK] = (torch.round(z / gap) * gap).clamp(-6, 6) * unit
        return out if case["along"] == "rows" else out.t().contiguous()
    if case["op"] == "product":
        return _exact_values(s["a"], case["k"]) @ _exact_values(s["b"], case["k"]).t().contiguous()
    if case["op"] == "a16":
        return s["a"].double() @ _exact_values(s["b"], case["k"]).t().contiguous()
    x, i, mx = s["x"].double(), case["i"], case["w"] == "mx"
    z = x @ s["router"].double().t().contiguous()
    z = torch.exp(z - z.max(1, keepdim=True).values)
    z = z / z.sum(1, keepdim=True)
    left, ids, gates = z.clone(), [], []
    for _ in range(case["top"]):
        best = left.max(1, keepdim=True).values
        at = (left == best).int().argmax(1, keepdim=True)  # the first of equals
        ids.append(at)
        gates.append(best)
        left.scatter_(1, at, -1.0)
    ids, gates = torch.cat(ids, 1), torch.cat(gates, 1)
    if case["renorm"]:
        gates = gates / gates.sum(1, keepdim=True)
    y = torch.zeros_like(x)
    for e in range(case["e"]):
        tok, slot = torch.nonzero(ids == e, as_tuple=True)
        if tok.numel() == 0:
            continue
        w1 = _exact_values((s["w1"][0][e], s["w1"][1][e]), case["h"]) if mx else s["w1"][e].double()
        w2 = _exact_values((s["w2"][0][e], s["w2"][1][e]), i) if mx else s["w2"][e].double()
        u = x[tok] @ w1.t().contiguous()
        u = u[:, :i] / (1 + torch.exp(-u[:, :i])) * u[:, i:]
        y.index_add_(0, tok, gates[tok, slot].unsqueeze(1) * (u @ w2.t().contiguous()))
    return y, ids.int(), gates
