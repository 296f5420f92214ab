"""Dense float64 reference of the windowed attention with, for every output, a bound on the error that the library's
arithmetic may make (derived here, before any run).

u = 2^-24 is half a step of fp32, w the half step the softmax weights (and dS) are rounded to before their product
(2^-8 for a plain bf16 weight, 2^-16 for a bf16 hi + lo pair, 0 on the fp32 path), r the half step of the output's type.

* A score is a sum of d_k products and one scaling: |ds| <= (d_k + 4) u sum|q||k| scale.  lse and exp take it over and
  add a few u of their own (the exponent's argument, up to max|s - m| ~ A = 2 max|s|, is rounded too: A u; the fast
  base-2 exponential has 2 u): a weight is off by the factor e_p = 2 |ds| + (2 A + n + 16) u, n the number of its terms.
* o = sum p v: (e_p + w) sum p|v| + r |o|.
* dP = dO . v: (d_v + 4) u sum|dO||v|.  delta = dO . o from o as given (rounded to its type, half step r_o):
  r_o sum|dO||o| + (d_v + 4) u sum|dO||o|.
* dS = P (dP - delta): P [ (e_p + w + 4 u) |dP - delta| + the two errors above ];  dq and dk sum it against |k| and |q|,
  dv sums (e_p + w) P against |dO|; each adds n u of its absolute sum and r of its value.
* Half steps are relative only for normal numbers.  A weight below 2^-126 is subnormal: rounding or flushing it may cost
  its whole value, so every weight is off by 2^-126 more (dS: that times |dP - delta| + 1), and a result below 2^-126 by
  2^-126 once more.  Weights that small occur with scores of several hundred.
"""

import torch

U = 2.0 ** -24
TINY = 2.0 ** -126
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def mask(L, window, n_sink, device="cpu"):
    t = torch.arange(L, device=device)
    back = t[:, None] - t[None, :]
    far = torch.zeros_like(back, dtype=torch.bool) if window <= 0 else back >= window
    return (back >= 0) & (~far | (t[None, :] < n_sink))


def dense(q, k, v, window, n_sink, lens=None, scale=None, dO=None, w=0.0, out=None, o_half=None):
    """{"o", "lse", "dq", "dk", "dv"} -> (value, bound), float64.  Rows behind lens are zero.  ``out``: half step of the
    outputs' type (q's by default); ``o_half``: half step of the o that the backward is given."""
    out = HALF[q.dtype] if out is None else out
    o_half = out if o_half is None else o_half
    B, H, L, dk = q.shape
    Hkv, dv = k.shape[1], v.shape[-1]
    G = H // Hkv
    scale = dk ** -0.5 if scale is None else scale
    live = torch.ones(B, L, dtype=torch.bool, device=q.device)
    if lens is not None:
        live = torch.arange(L, device=q.device)[None, :] < lens.to(q.device)[:, None].clamp(0, L)
    zap = lambda x: torch.where(live[:, None, :, None], x.double(), 0.0)  # noqa: E731
    qd = zap(q).view(B, Hkv, G, L, dk)
    kd, vd = zap(k)[:, :, None], zap(v)[:, :, None]
    see = mask(L, window, n_sink, q.device) & live[:, None, None, None, :]
    s = scale * qd @ kd.transpose(-1, -2)
    sabs = (scale * qd.abs() @ kd.abs().transpose(-1, -2)).masked_fill(~see, 0.0)
    s = s.masked_fill(~see, -torch.inf)
    lse = torch.logsumexp(s, -1)
    lse = torch.where(live[:, None, None], lse, 0.0)
    p = torch.exp(s - lse[..., None])
    p = torch.where(see & live[:, None, None, :, None], p, 0.0)
    n = see.sum(-1, keepdim=True).double()
    A = 2 * sabs.amax(-1, keepdim=True)
    e_s = (dk + 4) * U * sabs.amax(-1, keepdim=True)
    e_p = 2 * e_s + (2 * A + n + 16) * U
    o = p @ vd
    res = {"o": (o, (e_p + w) * (p @ vd.abs()) + out * o.abs() + TINY * (1 + see.double() @ vd.abs())),
           "lse": (lse, (e_s + (A + n + 16) * U).squeeze(-1) + 2 * U * lse.abs())}
    if dO is not None:
        g = zap(dO).view(B, Hkv, G, L, dv)
        dp = g @ vd.transpose(-1, -2)
        delta = (g * o).sum(-1, keepdim=True)
        oabs = (g.abs() * o.abs()).sum(-1, keepdim=True)
        e_o = ((e_p + w) * (p @ vd.abs()) * g.abs()).sum(-1, keepdim=True)  # the given o's own error
        e = (dv + 4) * U * (g.abs() @ vd.abs().transpose(-1, -2)) + (o_half + (dv + 4) * U) * oabs + e_o
        ds = p * (dp - delta)
        e_ds = p * ((e_p + w + 4 * U) * (dp - delta).abs() + e)
        m = live.sum(-1).double().view(B, 1, 1, 1, 1) * G * U  # the terms of a key's sums
        tr = lambda x: x.transpose(-1, -2)  # noqa: E731
        tiny = TINY * see * ((dp - delta).abs() + 1)
        dq = scale * ds @ kd
        dkk = (scale * tr(ds) @ qd).sum(2)
        dvv = (tr(p) @ g).sum(2)
        res["dq"] = dq, scale * (e_ds + n * U * ds.abs() + tiny) @ kd.abs() + out * dq.abs() + TINY
        res["dk"] = dkk, (scale * tr(e_ds + m * ds.abs() + tiny) @ qd.abs()).sum(2) + out * dkk.abs() + TINY
        res["dv"] = dvv, (tr((e_p + w + m) * p + TINY * see) @ g.abs()).sum(2) + out * dvv.abs() + TINY
    shape = lambda x: x.flatten(1, 2) if x.dim() == 5 or (x.dim() == 4 and x.shape[2] == G and x.shape[3] == L) else x  # noqa: E731
    res["lse"] = tuple(x.reshape(B, H, L) for x in res["lse"])
    return {name: pair if name == "lse" else tuple(shape(x) for x in pair) for name, pair in res.items()}


def worst(got, pair):
    """Largest error in units of its bound (a value past the end must be exactly what it was: zero here)."""
    ref, bound = pair
    err = (got.double() - ref).abs()
    assert torch.isfinite(err).all(), "not finite"
    return float((err / (bound + 1e-300)).where(err > 0, torch.zeros_like(err)).max()) if err.numel() else 0.0
