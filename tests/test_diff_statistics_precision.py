"""Statistics that the differential calls keep in 32 bits, against bounds that 16-bit
probabilities or a coarser exponential would exceed (shown on the CPU for each).

Log-sum-exp.  The score products are exact and summed in fp32 in a handful of steps, so a score s
is off by a few 2^-23 of its size; the exponential's argument takes three more roundings of its
size; a sum of positive terms stays within 2^-18 for these lengths (at most 64 additions in a row).
The forward's polynomial adds 2.9e-6 at most for the whole of a row.  So the forward's LSE is held
to 2^-17 + 2^-21 (|LSE| + max |s|) and the decode's, without polynomials, to 2^-18 and the same.

dlam = -sum P_2 dP.  P_2's errors are of two kinds: the row's LSE and its roundings, one relative
error (2^-17) for a whole row of terms, whose sum is D_2; and the score's, the argument's and the
exponential's, a few 1e-6 of each term, independent, so that they grow as the root of the terms'
squares: 2^-15 of that root is over five times their standard deviation.  The result is rounded
once (2^-8).  With dO made orthogonal to O_2 the sum is small beside its terms, and what is left
shows their rounding."""

import math
import os
import sys

import numpy as np
import pytest
import torch

from tests import _diff_ref as ref
from tests.test_diff_decode import _problem
from tests.test_diff_fwd import problem

BF, I32 = torch.bfloat16, torch.int32


def _lib():
    import exact_io_aware_46_b200 as attn

    return attn


# ------------------------------------------------------------------ log-sum-exp


def _largest_scores(Q, K, causal, k_lens, scale):
    """max |s| of each row and map over its visible keys, [B, Hq, 2, Lq]."""
    B, Hq, Lq, d = Q.shape
    Hkv, Lk, h = K.shape[1], K.shape[2], d // 2
    out = torch.zeros(B, Hq, 2, Lq, dtype=torch.float64)
    for b in range(B):
        kl = Lk if k_lens is None else k_lens[b]
        vis = ref.visible(Lq, Lk, causal, kl)
        for hq in range(Hq):
            k = ref._clean(K[b, hq // (Hq // Hkv)].double(), kl)
            for m in (0, 1):
                s = Q[b, hq, :, m * h:(m + 1) * h].double() @ k[:, m * h:(m + 1) * h].T * scale
                out[b, hq, m] = s.abs().masked_fill(~vis, 0).amax(-1)
    return out


def _assert_lse(got, lse, top, base):
    got, fin = got.double().cpu(), torch.isfinite(lse)
    assert torch.equal(got[~fin], lse[~fin])
    over = (got[fin] - lse[fin]).abs() - (base + 2.0 ** -21 * (lse[fin].abs() + top[fin]))
    assert over.numel() == 0 or over.max() <= 0, f"LSE {over.max():.2e} past its bound"


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,Lq,Lk,d,causal,k_lens,scale", [
    (2, 3, 3, 421, 421, 128, True, None, None),
    (1, 4, 2, 300, 300, 64, True, None, None),
    (2, 2, 1, 333, 390, 64, False, [383, 129], None),
    (1, 2, 2, 700, 1500, 128, True, None, None),
    (2, 2, 2, 390, 390, 128, True, [390, 250], 1.0),
    (2, 2, 2, 390, 390, 64, False, [390, 250], 1.0),
])
def test_forward_lse(B, Hq, Hkv, Lq, Lk, d, causal, k_lens, scale):
    Q, K, V, _, lam = problem(B, Hq, Hkv, Lq, Lk, d, 500 + Lq + Lk, k_lens)
    kl = None if k_lens is None else torch.tensor(k_lens, dtype=I32, device="cuda")
    lse = ref.fwd(Q, K, V, lam, scale=scale, causal=causal, k_lens=k_lens)[2]
    top = _largest_scores(Q, K, causal, k_lens, scale or 1 / math.sqrt(d / 2))
    l = _lib().attn_fwd_diff(Q.cuda(), K.cuda(), V.cuda(), lam.cuda(), scale=scale, causal=causal,
                             k_lens=kl)[2]
    _assert_lse(l, lse, top, 2.0 ** -17)


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,Lmax,d,lens,scale", [
    (3, 4, 2, 700, 128, [0, 1, 700], None),
    (2, 16, 2, 2049, 64, [2049, 640], None),
    (40, 8, 4, 2500, 128, [(61 * b) % 2501 for b in range(40)], None),
    (2, 4, 2, 900, 64, [777, 130], 1.0),
])
def test_decode_lse(B, Hq, Hkv, Lmax, d, lens, scale):
    Q, K, V, lam = _problem(B, Hq, Hkv, Lmax, d, lens, 600 + Lmax)
    lse = ref.fwd(Q, K, V, lam, scale=scale, k_lens=lens)[2]
    top = _largest_scores(Q, K, False, lens, scale or 1 / math.sqrt(d / 2))
    l = _lib().attn_fwd_splitkv_decode_diff(Q.cuda(), K.cuda(), V.cuda(), lam.cuda(),
                                            torch.tensor(lens, dtype=I32, device="cuda"),
                                            scale=scale)[1]
    _assert_lse(l, lse[..., 0], top[..., 0], 2.0 ** -18)


# keys 6 and 7 of eight, whose exponentials are the polynomial's, hold a row's mass: key 7 is the
# maximum, key 6 lies x (log2) below it.  Each score is one exact product.
POLY_BOUND = 0.5 * 2.9e-6 + 2.0 ** -21  # half the mass at most, and fp32


def _two_keys():
    x = -(torch.arange(1, 128) / 128).to(torch.float64)  # log2 distance of key 6, exact in bf16
    return x


def _poly_lse(degree):
    """ln(1 + 2^x) with 2^x by the fitted polynomial, in fp32."""
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                        "exact_io_aware_46_b200", "csrc")
    sys.path.insert(0, csrc)
    from exp2_poly_fit import eval_f32, fit

    coef, _ = fit(degree)
    return np.log1p(eval_f32(coef, _two_keys().numpy().astype(np.float32)).astype(np.float64))


def test_a_coarser_polynomial_is_past_the_bound():
    exact = np.log1p(np.exp2(_two_keys().numpy()))
    assert np.abs(_poly_lse(4) - exact).max() <= POLY_BOUND
    assert np.abs(_poly_lse(3) - exact).max() > 5 * POLY_BOUND


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m", [0, 1])
def test_forward_lse_of_the_polynomial_columns(d, m):
    x = _two_keys()
    n, scale = len(x), math.log(2.0)
    Q, K = torch.zeros(1, 1, n, d), torch.zeros(1, 1, 8, d)
    at = m * d // 2
    Q[0, 0, :, at], K[0, 0, 6, at] = x.float(), 1.0  # score x
    Q[0, 0, :, at + 1], K[0, 0, :6, at + 1] = 1.0, -200.0  # no weight
    V = torch.ones(1, 1, 8, d)
    l = _lib().attn_fwd_diff(Q.to(BF).cuda(), K.to(BF).cuda(), V.to(BF).cuda(),
                             torch.ones(1, device="cuda"), scale=scale)[2]
    want = torch.log1p(torch.exp2(x))
    assert (l[0, 0, m].double().cpu() - want).abs().max() <= POLY_BOUND


# ------------------------------------------------------------------ dlam


def _orthogonal(dO, O2):
    """dO without its component along O2, row by row, in bf16."""
    o = O2.double()
    s = (dO.double() * o).sum(-1, keepdim=True) / (o * o).sum(-1, keepdim=True).clamp_min(1e-30)
    return (dO.double() - s * o).to(BF)


def _dlam(q2, k2, v, dO, vis, scale, lse=None):
    """One head of one sequence, in 64 bits: -sum P_2 dP, its bound before the result's rounding,
    and the same sum with P_2 rounded to bf16."""
    s = (q2 @ k2.T * scale).masked_fill(~vis, -math.inf)
    l = torch.logsumexp(s, -1, keepdim=True)
    P = torch.exp(s - torch.where(torch.isfinite(l), l, torch.zeros_like(l)))
    t = P * (dO @ v.T)
    rows = t.sum(-1)
    bound = 2.0 ** -17 * rows.abs().sum() + 2.0 ** -15 * t.square().sum().sqrt()
    coarse = -(P.to(BF).double() * (dO @ v.T)).sum()
    return torch.stack([-rows.sum(), bound, coarse])


CASES = [
    # B, Hq, Hkv, Lq, Lk, d, causal, k_lens
    (1, 2, 2, 200, 200, 128, True, None),
    (1, 2, 2, 256, 256, 64, False, None),
    (2, 4, 1, 300, 300, 64, True, None),
    (2, 2, 2, 190, 190, 128, False, [120, 50]),
    (1, 2, 2, 100, 260, 128, True, None),
    (8, 16, 16, 300, 300, 64, True, [300, 1, 128, 129, 255, 256, 257, 290]),
    (1, 16, 1, 700, 700, 128, True, None),
]


def _head_sums(B, Hq, Hkv, Lq, Lk, d, causal, k_lens, lam_count):
    """Inputs with dO orthogonal to O_2, and [dlam, bound, coarse] of every head in 64 bits."""
    Q, K, V, dO, lam = problem(B, Hq, Hkv, Lq, Lk, d, 700 + Lq + Lk, k_lens, fill=0.0)
    dO = _orthogonal(dO, ref.fwd(Q, K, V, lam, causal=causal, k_lens=k_lens)[1])
    out = torch.zeros(Hq, 3, dtype=torch.float64)
    h = d // 2
    for b in range(B):
        vis = ref.visible(Lq, Lk, causal, Lk if k_lens is None else k_lens[b])
        for hq in range(Hq):
            g = hq // (Hq // Hkv)
            out[hq] += _dlam(Q[b, hq, :, h:].double(), K[b, g, :, h:].double(), V[b, g].double(),
                             dO[b, hq].double(), vis, 1 / math.sqrt(h))
    if lam_count == 1:
        lam, out = lam[:1], out.sum(0, keepdim=True)
    return (Q, K, V, dO, lam), out


@pytest.mark.parametrize("case", CASES)
def test_probabilities_of_16_bits_are_past_the_bound(case):
    _, out = _head_sums(*case, lam_count=0)
    want, bound, coarse = out.unbind(-1)
    over = (coarse.to(BF).double() - want).abs() / (bound + ref.U_BF16 * want.abs())
    assert over.max() > 2, over


@pytest.mark.gpu
@pytest.mark.parametrize("lam_count", [0, 1])
@pytest.mark.parametrize("case", CASES)
def test_dlam(case, lam_count):
    attn = _lib()
    B, Hq, Hkv, Lq, Lk, d, causal, k_lens = case
    inputs, out = _head_sums(*case, lam_count)
    want, bound, _ = out.unbind(-1)
    kl = None if k_lens is None else torch.tensor(k_lens, dtype=I32, device="cuda")
    q, k, v, do, w = (t.cuda() for t in inputs)
    O, O2, L = attn.attn_fwd_diff(q, k, v, w, causal=causal, k_lens=kl)
    dlam = attn.attn_bwd_diff(q, k, v, w, O, O2, do, L, causal=causal, k_lens=kl)[3]
    ref.assert_within(dlam, want, bound + ref.U_BF16 * want.abs(), "dlam")


@pytest.mark.gpu
def test_dlam_at_a_training_size():
    """B=2, H=16, L=8192, d=128, causal: two heads' sums over both sequences in 64 bits."""
    attn = _lib()
    B, H, L, d = 2, 16, 8192, 128
    g = torch.Generator(device="cuda").manual_seed(22)
    rn = lambda: torch.randn(B, H, L, d, generator=g, device="cuda").to(BF)
    Q, K, V, dO = rn(), rn(), rn(), rn()
    lam = torch.rand(H, generator=g, device="cuda")
    O, O2, lse = attn.attn_fwd_diff(Q, K, V, lam, causal=True)
    for b in range(B):
        dO[b] = _orthogonal(dO[b], O2[b])
    dlam = attn.attn_bwd_diff(Q, K, V, lam, O, O2, dO, lse, causal=True)[3]
    vis = torch.ones(L, L, dtype=torch.bool, device="cuda").tril()
    for h in (0, 11):
        out = sum(_dlam(Q[b, h, :, d // 2:].double(), K[b, h, :, d // 2:].double(),
                        V[b, h].double(), dO[b, h].double(), vis, 1 / math.sqrt(d / 2))
                  for b in range(B))
        want, bound, coarse = out.cpu().unbind(0)
        tol = bound + ref.U_BF16 * want.abs()
        assert (coarse - want).abs() > tol
        ref.assert_within(dlam[h], want, tol, f"dlam of head {h}")
