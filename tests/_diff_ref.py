"""Plain 64-bit forms of differential attention and of the append, for the tests, and the
error bounds that the kernels' roundings allow.

Bounds.  The kernels round each map's unnormalised probabilities to bf16 (relative error at
most u = 2^-8, half a step) before the product with V, sum them unrounded, and round O once;
the exponentials (polynomial: 1.01e-4 relative) and fp32 sums stay within e = 2^-12 of the
probability.  So |O - O_ref| <= (u + e) (P_1 |V| + |lam| P_2 |V|) + u |O_ref| element by
element, and the log-sum-exp is off by at most e plus its own fp32 rounding."""

import math

import numpy as np
import torch

U_BF16 = 2.0 ** -8   # half a step of bf16, relative
E_PROB = 2.0 ** -12  # exponential and fp32 sums, relative


def visible(Lq, Lk, causal, kl):
    i = torch.arange(Lq)[:, None]
    j = torch.arange(Lk)[None, :]
    vis = (j < kl).expand(Lq, Lk)
    return vis & (j <= i + (Lk - Lq)) if causal else vis


def _clean(x, kl):
    """Rows at and past kl are not part of the problem, whatever they hold."""
    x = x.clone()
    x[..., kl:, :] = 0
    return x


def _maps(q, k, vis, scale):
    h = q.shape[-1] // 2
    P, lse = [], []
    for m in (slice(0, h), slice(h, 2 * h)):
        s = (q[:, m] @ k[:, m].T * scale).masked_fill(~vis, -math.inf)
        l = torch.logsumexp(s, -1)
        P.append(torch.exp(s - torch.where(torch.isfinite(l), l, torch.zeros_like(l))[:, None]))
        lse.append(l)
    return P, torch.stack(lse)


def fwd(Q, K, V, lam, scale=None, causal=False, k_lens=None):
    """Tensors of any type on the CPU -> O, O2, lse [B,Hq,2,Lq], and the bounds of O and O2."""
    Q, K, V, lam = (t.double() for t in (Q, K, V, lam))
    B, Hq, Lq, d = Q.shape
    Hkv, Lk = K.shape[1], K.shape[2]
    scale = 1.0 / math.sqrt(d / 2) if scale is None else scale
    lam = lam.expand(Hq)
    O, O2, tol, tol2 = (torch.zeros_like(Q) for _ in range(4))
    lse = torch.zeros(B, Hq, 2, Lq, dtype=torch.float64)
    for b in range(B):
        kl = Lk if k_lens is None else int(k_lens[b])
        vis = visible(Lq, Lk, causal, kl)
        for hq in range(Hq):
            g = hq // (Hq // Hkv)
            k, v = _clean(K[b, g], kl), _clean(V[b, g], kl)
            (p1, p2), lse[b, hq] = _maps(Q[b, hq], k, vis, scale)
            O2[b, hq] = p2 @ v
            O[b, hq] = p1 @ v - lam[hq] * O2[b, hq]
            a2 = p2 @ v.abs()
            tol[b, hq] = (U_BF16 + E_PROB) * (p1 @ v.abs() + lam[hq].abs() * a2)
            tol2[b, hq] = (U_BF16 + E_PROB) * a2
    return O, O2, lse, tol + U_BF16 * O.abs(), tol2 + U_BF16 * O2.abs()


def bwd(Q, K, V, lam, dO, scale=None, causal=False, k_lens=None):
    """dQ, dK, dV, dlam [Hq] in 64 bits, from the formulas."""
    Q, K, V, lam, dO = (t.double() for t in (Q, K, V, lam, dO))
    B, Hq, Lq, d = Q.shape
    Hkv, Lk, h = K.shape[1], K.shape[2], d // 2
    scale = 1.0 / math.sqrt(h) if scale is None else scale
    lam = lam.expand(Hq)
    dQ, dK, dV = (torch.zeros_like(t) for t in (Q, K, V))
    dlam = torch.zeros(Hq, dtype=torch.float64)
    for b in range(B):
        kl = Lk if k_lens is None else int(k_lens[b])
        vis = visible(Lq, Lk, causal, kl)
        for hq in range(Hq):
            g = hq // (Hq // Hkv)
            k, v = _clean(K[b, g], kl), _clean(V[b, g], kl)
            P, _ = _maps(Q[b, hq], k, vis, scale)
            dP = dO[b, hq] @ v.T
            for m, c in ((0, 1.0), (1, -lam[hq])):
                part = slice(m * h, (m + 1) * h)
                D = (P[m] * dP).sum(-1, keepdim=True)
                dS = c * P[m] * (dP - D) * scale
                dQ[b, hq, :, part] = dS @ k[:, part]
                dK[b, g, :, part] += dS.T @ Q[b, hq, :, part]
                dV[b, g] += c * P[m].T @ dO[b, hq]
                if m:
                    dlam[hq] -= D.sum()
    return dQ, dK, dV, dlam


def rotate(x, cos, sin, maps, interleaved):
    """x [T, H, d], cos and sin [T, rope_dim / 2], in 64 bits."""
    T, H, d = x.shape
    half, part = cos.shape[1], d // maps
    y = x.double().clone()
    c, s = cos.double()[:, None], sin.double()[:, None]
    for m in range(maps):
        i = torch.arange(half)
        a = m * part + (2 * i if interleaved else i)
        b = a + (1 if interleaved else half)
        xa, xb = x[..., a].double(), x[..., b].double()
        y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
    return y


def rotation_bound(x, ref, maps, half, interleaved):
    """|y - ref| for two fp32 products, one sum and one rounding to bf16."""
    mag = x.double().abs()
    part = x.shape[-1] // maps
    amp = torch.zeros_like(mag)
    for m in range(maps):
        i = torch.arange(half)
        a = m * part + (2 * i if interleaved else i)
        b = a + (1 if interleaved else half)
        amp[..., a] = amp[..., b] = mag[..., a] + mag[..., b]
    return U_BF16 * ref.abs() + 2.0 ** -22 * amp


def assert_within(got, ref, bound, what):
    got, ref, bound = (np.asarray(t.detach().double().cpu()) for t in (got, ref, bound))
    assert np.all(np.isfinite(got)), f"{what}: values that are not finite"
    over = np.abs(got - ref) - bound
    assert over.size == 0 or over.max() <= 0, \
        f"{what}: {over.max():.3e} past a bound of {bound.flat[over.argmax()]:.3e}"


def assert_lse(got, ref, what="LSE"):
    got, ref = got.detach().double().cpu(), ref.cpu()
    fin = torch.isfinite(ref)
    assert torch.equal(got[~fin], ref[~fin]), f"{what}: rows without a key"
    err = (got[fin] - ref[fin]).abs()
    assert err.numel() == 0 or bool((err <= E_PROB + 2.0 ** -22 * ref[fin].abs()).all()), \
        f"{what}: off by {err.max():.3e}"
