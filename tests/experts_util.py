"""The experts' products and their gradients in 64 bits, with bounds of what fp32
sums and the roundings between the products may be off (no code of the library).

A product of K terms in fp32 is off by at most (K + 8) 2^-23 of the sum of its
terms' magnitudes.  With hs half a step of the 16-bit format, s = 1 / (1 + exp(-p)):
  p, q (first product)      ep, eq: that bound
  u = p s q                 |silu'| <= 1.1: (|silu| + 1.1 ep)(|q| + eq) - |silu q|, and 2^-20 |u|
                            for exp, division and products in fp32; kept in 16 bits: hs more
  a choice's term of y      gate |W2| (error of u), its own fp32 sum, kept in fp32: 2^-24
  v = W2^T dy               ev: the bound of its sum
  dp = gate v q f(p)        f = s (1 + p (1 - s)), |f| <= 1.1, |f'| <= 0.5, and f itself is off by
                            2^-20 at most: gate ((|v| + ev)(|q| + eq)(|f| + 0.5 ep + 2^-20) - |v q f|), hs
  dq = gate v silu(p)       likewise with |silu'| <= 1.1
  gate u                    as u
and the last products by their operands' errors and their own sums.
"""
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def _mm(a, b):
    return a.contiguous() @ b.contiguous()


def reference(x, ids, gates, w1, w2, dy=None):
    """{"y": (value, bound), and with dy "dx", "dgates", "dw1", "dw2"}, in 64 bits."""
    dtype, dev = x.dtype, x.device
    hs, tiny = HALF_STEP[dtype], TINY[dtype]
    E, H, I = w2.shape
    T, top = ids.shape
    x, gates = x.double(), gates.double()
    zero = lambda *s: torch.zeros(s, dtype=torch.float64, device=dev)  # noqa: E731
    eps = 2.0 ** -23
    y, by = zero(T, H), zero(T, H)
    mag = zero(T, H)  # sum of the terms' magnitudes
    if dy is not None:
        dy = dy.double()
        dx, bdx, mdx = zero(T, H), zero(T, H), zero(T, H)
        dg, bdg = zero(T, top), zero(T, top)
        dw1, bw1, dw2, bw2 = (zero(*s) for s in ((E, 2 * I, H), (E, 2 * I, H), (E, H, I), (E, H, I)))
    for e in range(E):
        tok, slot = torch.nonzero(ids == e, as_tuple=True)
        n = tok.numel()
        if n == 0:
            continue
        a1, a2 = w1[e].double(), w2[e].double()
        xt, g = x[tok], gates[tok, slot].unsqueeze(1)
        h, bh = _mm(xt, a1.t()), (H + 8) * eps * _mm(xt.abs(), a1.abs().t())
        p, q, ep, eq = h[:, :I], h[:, I:], bh[:, :I], bh[:, I:]
        s = torch.sigmoid(p)
        silu = p * s
        u = silu * q
        eu = (silu.abs() + 1.1 * ep) * (q.abs() + eq) - u.abs() + 2.0 ** -20 * u.abs()
        ru = eu + hs * (u.abs() + eu) + tiny
        t, at = _mm(u, a2.t()), a2.abs().t()
        bt = _mm(ru, at) + (I + 8) * eps * _mm(u.abs() + ru, at)
        gt, gb = g * t, g.abs() * bt * (1 + eps)
        gb = gb + 2.0 ** -24 * (gt.abs() + gb)
        y.index_add_(0, tok, gt)
        by.index_add_(0, tok, gb)
        mag.index_add_(0, tok, gt.abs() + gb)
        if dy is None:
            continue
        dt = dy[tok]
        v, ev = _mm(dt, a2), (H + 8) * eps * _mm(dt.abs(), a2.abs())
        dg[tok, slot] = (v * u).sum(1)
        bdg[tok, slot] = ((v.abs() + ev) * (u.abs() + eu) - (v * u).abs()
                          + (I + 16) * eps * (v.abs() + ev) * (u.abs() + eu)).sum(1)
        f = s * (1 + p * (1 - s))
        dp, dq = g * v * q * f, g * v * silu
        bp = g.abs() * ((v.abs() + ev) * (q.abs() + eq) * (f.abs() + 0.5 * ep + 2.0 ** -20) - (v * q * f).abs())
        bq = g.abs() * ((v.abs() + ev) * (silu.abs() * (1 + 2.0 ** -20) + 1.1 * ep) - (v * silu).abs())
        bp, bq = (b + (hs + 2.0 ** -20) * (d.abs() + b) + tiny for b, d in ((bp, dp), (bq, dq)))
        dh, bdh = torch.cat((dp, dq), 1), torch.cat((bp, bq), 1)
        r, br = _mm(dh, a1), _mm(bdh, a1.abs()) + (2 * I + 8) * eps * _mm(dh.abs() + bdh, a1.abs())
        br = br + 2.0 ** -24 * (r.abs() + br)
        dx.index_add_(0, tok, r)
        bdx.index_add_(0, tok, br)
        mdx.index_add_(0, tok, r.abs() + br)
        dw1[e] = _mm(dh.t(), xt)
        bw1[e] = _mm(bdh.t(), xt.abs()) + (n + 8) * eps * _mm((dh.abs() + bdh).t(), xt.abs())
        gu = g * u
        bu = g.abs() * eu * (1 + eps) + eps * gu.abs()
        bu = bu + hs * (gu.abs() + bu) + tiny
        dw2[e] = _mm(dt.t(), gu)
        bw2[e] = _mm(dt.abs().t(), bu) + (n + 8) * eps * _mm(dt.abs().t(), gu.abs() + bu)
    out = {"y": (y, by + top * eps * mag)}
    if dy is not None:
        out |= {"dx": (dx, bdx + top * eps * mdx), "dgates": (dg, bdg), "dw1": (dw1, bw1), "dw2": (dw2, bw2)}
    return out


def check(got, ref, what):
    """`got` against (value, bound): every element within the bound and the half step of its
    type, and the whole within three such half steps of the norm (the operands', the
    terms' and its own roundings, each at most one)."""
    value, bound = ref
    hs, tiny = HALF_STEP.get(got.dtype, 2.0 ** -24), TINY.get(got.dtype, 2.0 ** -150)
    d = (got.double() - value).abs()
    assert torch.isfinite(d).all(), what
    over = d - (bound * (1 + hs) + hs * value.abs() + tiny)
    if over.numel():
        assert float(over.max()) <= 0, (what, float(over.max()), float(d.max()))
    norm = float(value.norm())
    assert float(d.norm()) <= (2e-5 + (3 * hs if got.dtype in HALF_STEP else 0)) * norm + 1e-30, (what, float(d.norm()) / norm)
