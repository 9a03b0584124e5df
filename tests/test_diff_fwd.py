"""attn_fwd_diff against the definition in 64 bits."""

import math

import pytest
import torch

from tests import _diff_ref as ref
from tests.test_binding_validation import FakeCuda, rejects

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _lib():
    import exact_io_aware_46_b200 as attn

    return attn


def problem(B, Hq, Hkv, Lq, Lk, d, seed, k_lens=None, fill=math.nan):
    """Inputs; K and V rows past each sequence's length hold `fill`."""
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g).to(BF)
    Q, K, V, dO = rn(B, Hq, Lq, d), rn(B, Hkv, Lk, d), rn(B, Hkv, Lk, d), rn(B, Hq, Lq, d)
    for b, n in enumerate(k_lens or []):
        K[b, :, n:], V[b, :, n:] = fill, fill
    return Q, K, V, dO, torch.rand(Hq, generator=g) * 1.6 - 0.3


CASES = [
    # B, Hq, Hkv, Lq, Lk, d, causal, k_lens
    (1, 1, 1, 1, 1, 128, False, None),
    (1, 2, 2, 256, 256, 64, False, None),
    (2, 3, 3, 421, 421, 128, True, None),          # several tiles, ragged tail
    (1, 4, 2, 300, 300, 64, True, None),           # grouped heads
    (2, 2, 2, 333, 333, 128, False, [200, 77]),    # padding that ends inside a tile
    (2, 2, 1, 333, 390, 64, True, [383, 129]),
    (1, 6, 2, 100, 300, 128, True, None),          # Lq < Lk
    (1, 2, 2, 300, 100, 128, True, None),          # Lq > Lk: leading rows see no key
    (1, 2, 1, 129, 513, 64, False, None),
    (2, 2, 2, 260, 260, 128, True, [0, 128]),      # a sequence without a key; a whole tile
    (1, 8, 1, 1, 700, 128, True, [699]),           # one new token
    (2, 2, 2, 5, 0, 128, False, None),             # no keys at all
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,Lq,Lk,d,causal,k_lens", CASES)
def test_fwd_matches_definition(B, Hq, Hkv, Lq, Lk, d, causal, k_lens):
    attn = _lib()
    Q, K, V, _, lam = problem(B, Hq, Hkv, Lq, Lk, d, 17 + Lq + Lk + d, k_lens)
    O, O2, lse, tol, tol2 = ref.fwd(Q, K, V, lam, causal=causal, k_lens=k_lens)
    kl = None if k_lens is None else torch.tensor(k_lens, dtype=I32, device="cuda")
    o, o2, l = attn.attn_fwd_diff(Q.cuda(), K.cuda(), V.cuda(), lam.cuda(), causal=causal,
                                  k_lens=kl)
    ref.assert_within(o, O, tol, "O")
    ref.assert_within(o2, O2, tol2, "O2")
    ref.assert_lse(l, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_fwd_large_scores_and_one_weight(d, causal):
    """Scale 1: most probabilities underflow and the running maxima move at each map's own
    pace; infinities past the lengths; one weight for all heads."""
    attn = _lib()
    k_lens = [390, 250]
    Q, K, V, _, lam = problem(2, 2, 2, 390, 390, d, 50 + d, k_lens, fill=math.inf)
    O, O2, lse, tol, tol2 = ref.fwd(Q, K, V, lam[:1], scale=1.0, causal=causal, k_lens=k_lens)
    o, o2, l = attn.attn_fwd_diff(Q.cuda(), K.cuda(), V.cuda(), lam[:1].cuda(), scale=1.0,
                                  causal=causal,
                                  k_lens=torch.tensor(k_lens, dtype=I32, device="cuda"))
    ref.assert_within(o, O, tol, "O")
    ref.assert_within(o2, O2, tol2, "O2")
    ref.assert_lse(l, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_fwd_equal_maps_and_zero_weight(d):
    """q1 = q2 and k1 = k2: O = (1 - lam) O_1, O2 = O_1; lam = 0: O = O_1."""
    attn = _lib()
    Q, K, V, _, _ = problem(1, 2, 1, 200, 200, d, 8)
    Q[..., d // 2:], K[..., d // 2:] = Q[..., :d // 2], K[..., :d // 2]
    lam = torch.tensor([1.0, 0.0])
    O, O2, _, tol, _ = ref.fwd(Q, K, V, lam, causal=True)
    o, o2, l = attn.attn_fwd_diff(Q.cuda(), K.cuda(), V.cuda(), lam.cuda(), causal=True)
    assert torch.equal(l[:, :, 0], l[:, :, 1])
    assert torch.equal(o[:, 1], o2[:, 1])
    ref.assert_within(o, O, tol, "O")


@pytest.mark.gpu
def test_fwd_outputs_aligned_to_16_bytes_a_side_stream_and_no_aux():
    attn = _lib()
    B, H, L, d = 1, 2, 300, 128
    Q, K, V, _, lam = (t.cuda() for t in problem(B, H, H, L, L, d, 3))
    o, o2, l = attn.attn_fwd_diff(Q, K, V, lam, causal=True)
    n = B * H * L * d
    buf = torch.empty(2, n + 8, dtype=BF, device="cuda")
    odd = [b[8:].view(B, H, L, d) for b in buf]
    assert all(t.data_ptr() % 32 == 16 for t in odd[:1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, a2, la = attn.attn_fwd_diff(Q, K, V, lam, causal=True, O=odd[0], O2=odd[1], stream=side)
    c, c2, lc = attn.attn_fwd_diff(Q, K, V, lam, causal=True, want_aux=False)
    torch.cuda.synchronize()
    assert torch.equal(a, o) and torch.equal(a2, o2) and torch.equal(la, l)
    assert torch.equal(c, o) and c2 is None and lc is None


@pytest.mark.gpu
def test_fwd_reports_a_bad_length_and_two_graphs_share_a_workspace():
    attn = _lib()
    Q, K, V, _, lam = problem(2, 2, 2, 200, 200, 128, 4)
    O, _, _, tol, _ = ref.fwd(Q, K, V, lam, k_lens=[200, 0])
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    args = [t.cuda() for t in (Q, K, V, lam)]
    o, o2, l = attn.attn_fwd_diff(*args, workspace=ws,
                                  k_lens=torch.tensor([200, 201], dtype=I32, device="cuda"))
    assert attn.attn_read_device_status(ws) == (attn.ATTN_ERR_INVALID, attn.ATTN_DEV_BAD_KLEN)
    ref.assert_within(o, O, tol, "O")
    assert (o2[1] == 0).all() and (l[1] == -math.inf).all()
    attn.attn_clear_device_status(ws)
    graphs, outs = [], []
    for causal in (False, True):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(attn.attn_fwd_diff(*args, causal=causal, workspace=ws)[0])
        graphs.append(graph)
    for _ in range(2):
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    for causal, got in zip((False, True), outs):
        O, _, _, tol, _ = ref.fwd(Q, K, V, lam, causal=causal)
        ref.assert_within(got, O, tol, f"O causal={causal}")


@pytest.mark.gpu
def test_fwd_prefill_size_sampled():
    """B=4, H=16, L=4096, d=128, causal: heads at both ends, rows of every kind."""
    attn = _lib()
    B, H, L, d = 4, 16, 4096, 128
    g = torch.Generator(device="cuda").manual_seed(12)
    rn = lambda: torch.randn(B, H, L, d, generator=g, device="cuda").to(BF)
    Q, K, V = rn(), rn(), rn()
    lam = torch.rand(H, generator=g, device="cuda")
    o, o2, l = attn.attn_fwd_diff(Q, K, V, lam, causal=True)
    rows = torch.tensor([0, 1, 127, 128, 2047, 2048, 4000, 4095])
    for b, h in ((0, 0), (1, 9), (3, 15)):
        one = [t[b:b + 1, h:h + 1].cpu() for t in (Q, K, V)]
        O, O2, lse, tol, tol2 = ref.fwd(*one, lam[h:h + 1].cpu(), causal=True)
        pick = lambda t: t[0, 0, rows]
        ref.assert_within(o[b, h].cpu()[rows], pick(O), pick(tol), "O")
        ref.assert_within(o2[b, h].cpu()[rows], pick(O2), pick(tol2), "O2")
        ref.assert_lse(l[b, h].cpu()[:, rows], lse[0, 0][:, rows])


def test_fwd_rejections():
    attn = _lib()
    B, Hq, Hkv, L, d = 2, 4, 2, 16, 128
    Q, KV, lam = FakeCuda((B, Hq, L, d), BF), FakeCuda((B, Hkv, L, d), BF), FakeCuda((Hq,), F32)
    f = attn.attn_fwd_diff
    rejects(lambda: f(Q, KV, FakeCuda((B, Hkv, L, 64), BF), lam), "V", "shape")
    rejects(lambda: f(Q, KV, KV, FakeCuda((Hq, 1), F32)), "lam")
    rejects(lambda: f(Q, KV, KV, FakeCuda((Hkv,), F32)), "lam")
    rejects(lambda: f(Q, KV, KV, FakeCuda((Hq,), F32, "cuda:1")), "lam", "cuda:1")
    rejects(lambda: f(Q, KV, KV, lam, O2=KV), "O2")
    rejects(lambda: f(Q, KV, KV, lam, lse=FakeCuda((B, Hq, L, 2), F32)), "lse")
    rejects(lambda: f(Q, KV, KV, lam, k_lens=FakeCuda((B,), torch.int64)), "k_lens")
    rejects(lambda: f(Q, KV, KV, lam, workspace=FakeCuda((16,), torch.uint8)), "workspace")
    rejects(lambda: f(torch.zeros(B, Hq, L, d, dtype=BF), KV, KV, lam), "Q", "CUDA")


def test_fwd_rejects_on_host():
    import ctypes

    attn = _lib()
    P = ctypes.c_void_p(256 * 1024)

    def call(Q=P, K=P, lam=P, n_lam=2, O=P, O2=None, B=1, Hq=2, Hkv=1, Lq=8, Lk=8, d=128,
             scale=0.1, mask=0, nb=256):
        return attn.lib().attn_fwd_diff(Q, K, P, lam, n_lam, O, O2, None, B, Hq, Hkv, Lq, Lk, d,
                                        scale, mask, None, P, nb, None)

    for bad in (dict(Q=None), dict(K=None), dict(lam=None), dict(n_lam=3), dict(n_lam=0),
                dict(O=None), dict(O2=ctypes.c_void_p(256 * 1024 + 8)), dict(Hq=3, Hkv=2, n_lam=3),
                dict(scale=0.0), dict(scale=float("inf")), dict(mask=2), dict(nb=16), dict(Lk=-1),
                dict(lam=ctypes.c_void_p(256 * 1024 + 2))):
        assert call(**bad) == attn.ATTN_ERR_INVALID, bad
    assert call(d=96) == attn.ATTN_ERR_UNSUPPORTED
    assert call(B=1 << 20, Lq=1 << 20) == attn.ATTN_ERR_UNSUPPORTED
    assert call(Lq=0) == 0 and call(Lq=0, Q=None, O=None) == 0


def test_polynomial_exponential():
    """The differential forward's software 2^x: degree 4, within 2.9e-6 of the exact value, read
    from the CUDA source; the fit reproduces its constants."""
    import os
    import re
    import sys

    import numpy as np

    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                        "exact_io_aware_46_b200", "csrc")
    src = open(os.path.join(csrc, "sm100.cuh")).read()
    body = src[src.index("ex2_poly4_nz(float2 x)"):]
    body = body[:body.index("\n}\n")]
    pairs = re.findall(r"make_float2\(([0-9.e-]+)f, \1f\)", body)
    coef = [float(v) for v in pairs if abs(float(v)) < 100][::-1]  # c0 ... c4
    assert len(coef) == 5 and coef[0] == 1.0
    sys.path.insert(0, csrc)
    from exp2_poly_fit import eval_f32, fit

    x = np.linspace(-125.0, 8.0, 2_000_001, dtype=np.float32)
    y = eval_f32(coef, x).astype(np.float64)
    assert np.abs(y / np.exp2(x.astype(np.float64)) - 1.0).max() <= 2.9e-6
    want, err = fit(4)
    assert err <= 2.8e-6 and np.allclose(np.float32(coef), np.float32(want), rtol=1e-5)
