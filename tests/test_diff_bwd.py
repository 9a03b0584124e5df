"""attn_bwd_diff (fed with attn_fwd_diff's O, O2 and LSE) against the formulas in 64 bits and
against differences of the definition.

Tolerances.  Each gradient passes through at most four bf16 roundings of relative size u = 2^-8
at most, about u / sqrt(6) in the mean square: the probabilities, W or dS, the saved O and O2 (in
D), and the result.  Their root mean square sum is 2 u / sqrt(6) = 3.2e-3; the library's bar for
gradients, 1e-2 in relative L2, leaves a factor of three for sums that cancel.  Where a row sees
one key, dS = P (dP - D) is zero and only the rounding of D is left, so dQ and dK are also
allowed an absolute u |dP| of it: those cases are measured against |scale| u times the size of
the products.  dlam sums P_2 dP of both signs, each to 2^-13 (the exponentials' 1e-4), and is
rounded once: u |dlam| + 2^-13 sum |P_2 dP|."""

import math

import pytest
import torch

from tests import _diff_ref as ref
from tests.test_binding_validation import FakeCuda, rejects
from tests.test_diff_fwd import problem

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
BAR = 1e-2


def _lib():
    import exact_io_aware_46_b200 as attn

    return attn


def _dlam_bound(Q, K, V, lam, dO, causal, k_lens, scale=None):
    Q, K, V, dO = (t.double() for t in (Q, K, V, dO))
    B, Hq, Lq, d = Q.shape
    G, Lk = Hq // K.shape[1], K.shape[2]
    scale = 1.0 / math.sqrt(d / 2) if scale is None else scale
    out = torch.zeros(Hq, dtype=torch.float64)
    for b in range(B):
        kl = Lk if k_lens is None else k_lens[b]
        vis = ref.visible(Lq, Lk, causal, kl)
        for h in range(Hq):
            k, v = ref._clean(K[b, h // G], kl), ref._clean(V[b, h // G], kl)
            P, _ = ref._maps(Q[b, h], k, vis, scale)
            out[h] += (P[1] * (dO[b, h] @ v.T)).abs().sum()
    return 2.0 ** -13 * out


def _rel(a, b):
    n = b.norm().item()
    return (a.detach().double().cpu() - b).norm().item() / (n if n > 0 else 1.0)


def _grads(Q, K, V, lam, dO, causal, k_lens, scale=None, **kw):
    attn = _lib()
    kl = None if k_lens is None else torch.tensor(k_lens, dtype=I32, device="cuda")
    q, k, v, do, w = (t.cuda() for t in (Q, K, V, dO, lam))
    O, O2, L = attn.attn_fwd_diff(q, k, v, w, scale=scale, causal=causal, k_lens=kl)
    return attn.attn_bwd_diff(q, k, v, w, O, O2, do, L, scale=scale, causal=causal, k_lens=kl, **kw)


CASES = [
    # B, Hq, Hkv, Lq, Lk, d, causal, k_lens
    (1, 2, 2, 200, 200, 128, True, None),
    (1, 2, 2, 256, 256, 64, False, None),
    (1, 6, 2, 150, 150, 128, True, None),          # three heads a group
    (2, 4, 1, 300, 300, 64, True, None),           # four heads a group, several tiles
    (2, 2, 2, 190, 190, 128, False, [120, 50]),    # padding that ends inside a tile
    (2, 2, 1, 190, 257, 64, True, [257, 130]),
    (1, 2, 2, 100, 260, 128, True, None),          # Lq < Lk
    (1, 2, 2, 260, 100, 128, True, None),          # Lq > Lk: leading rows see no key
    (1, 1, 1, 64, 128, 64, False, None),
    (2, 2, 1, 300, 300, 128, True, [0, 300]),      # a sequence without a key
    (1, 3, 3, 17, 600, 128, False, [513]),
    (3, 2, 2, 520, 520, 128, True, [384, 128, 520]),
    # (those above have few enough items to be split; these are not)
    (8, 16, 16, 300, 300, 64, True, [300, 1, 128, 129, 255, 256, 257, 290]),
    (5, 20, 10, 260, 390, 128, False, None),
    (1, 16, 1, 700, 700, 128, True, None),         # one key/value head: parts of several heads
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,Lq,Lk,d,causal,k_lens", CASES)
def test_bwd_matches_formulas(B, Hq, Hkv, Lq, Lk, d, causal, k_lens):
    Q, K, V, dO, lam = problem(B, Hq, Hkv, Lq, Lk, d, 23 + Lq + Lk + d, k_lens)
    got = _grads(Q, K, V, lam, dO, causal, k_lens)
    want = ref.bwd(Q, K, V, lam, dO, causal=causal, k_lens=k_lens)
    for g, w, name in zip(got[:3], want[:3], ("dQ", "dK", "dV")):
        assert torch.isfinite(g).all(), name
        assert _rel(g, w) <= BAR, f"{name}: rel-L2 {_rel(g, w):.3e}"
    bound = _dlam_bound(Q, K, V, lam, dO, causal, k_lens)
    ref.assert_within(got[3], want[3], bound + ref.U_BF16 * want[3].abs(), "dlam")
    for b, n in enumerate(k_lens or []):  # rows that no query sees
        assert (got[1][b, :, n:] == 0).all() and (got[2][b, :, n:] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_bwd_large_scores_and_one_weight(d, causal):
    """Scale 1: P sits on few keys a row; the shared weight's gradient is the heads' sum."""
    k_lens = [330, 201]
    Q, K, V, dO, lam = problem(2, 4, 2, 330, 330, d, 90 + d, k_lens, fill=math.inf)
    got = _grads(Q, K, V, lam[:1], dO, causal, k_lens, scale=1.0)
    want = ref.bwd(Q, K, V, lam[:1], dO, scale=1.0, causal=causal, k_lens=k_lens)
    for g, w, name in zip(got[:3], want[:3], ("dQ", "dK", "dV")):
        assert _rel(g, w) <= BAR, f"{name}: rel-L2 {_rel(g, w):.3e}"
    total = want[3].sum()[None]
    bound = _dlam_bound(Q, K, V, lam[:1], dO, causal, k_lens, 1.0).sum()
    ref.assert_within(got[3], total, bound + ref.U_BF16 * total.abs(), "dlam")


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_bwd_against_differences(d):
    """<gradient, direction> against central differences of sum(O dO) in 64 bits."""
    Q, K, V, dO, lam = problem(1, 4, 2, 70, 140, d, 12)
    got = _grads(Q, K, V, lam, dO, True, None)
    g = torch.Generator().manual_seed(1)
    f = lambda *x: (ref.fwd(*x, causal=True)[0] * dO.double()).sum()
    at = [t.double() for t in (Q, K, V, lam)]
    for n, (x, grad) in enumerate(zip(at, got)):
        # along the gradient itself the sum does not cancel; plus a random direction
        grad = grad.double().cpu()
        for u in (grad / grad.norm(), torch.randn(x.shape, generator=g).double()):
            u = u / u.norm()
            eps = 1e-5
            move = lambda s: f(*[y + s * eps * u if i == n else y for i, y in enumerate(at)])
            diff = (move(1) - move(-1)) / (2 * eps)
            assert abs((grad * u).sum() - diff) <= BAR * grad.norm(), n


@pytest.mark.gpu
def test_bwd_single_key_rows_and_lengths_of_one():
    """One key: P is 1 and the scores have no gradient.  dS is what the roundings of O and O2
    leave of dP - D: at most u (|dO| . |O| + 2 |lam| |dO| . |O2|) + fp32 sums."""
    attn = _lib()
    for Lq, Lk, causal in ((1, 1, False), (3, 1, False), (1, 1, True)):
        Q, K, V, dO, lam = problem(2, 2, 1, Lq, Lk, 128, 40 + Lq)
        got = _grads(Q, K, V, lam, dO, causal, None)
        want = ref.bwd(Q, K, V, lam, dO, causal=causal)
        O, O2, _, _, _ = ref.fwd(Q, K, V, lam, causal=causal)
        a = dO.double().abs()
        slack = ref.U_BF16 * ((a * O.abs()).sum(-1) + 2 * (lam[:, None].abs() * (a * O2.abs()).sum(-1)))
        slack = (slack + 1e-4 * (a.sum(-1))) / 8 * (1 + lam[:, None].abs())
        big = K.double().abs().max()
        assert bool((got[0].double().cpu().abs().amax(-1) <= slack * big).all()), "dQ"
        assert bool((got[1].double().cpu().abs() <= slack.sum() * Q.double().abs().max()).all()), "dK"
        assert _rel(got[2], want[2]) <= BAR
        bound = _dlam_bound(Q, K, V, lam, dO, causal, None)
        ref.assert_within(got[3], want[3], bound + ref.U_BF16 * want[3].abs(), "dlam")


@pytest.mark.gpu
def test_bwd_empty_axes():
    attn = _lib()
    for Lq, Lk in ((0, 130), (130, 0), (0, 0)):
        Q, K, V, dO, lam = problem(2, 2, 1, Lq, Lk, 64, 9)
        dQ, dK, dV, dlam = _grads(Q, K, V, lam, dO, False, None)
        assert all(bool((t == 0).all()) for t in (dQ, dK, dV, dlam))


@pytest.mark.gpu
def test_bwd_repeats_and_reuses_its_workspace_in_a_graph():
    """dK, dV and dlam bit for bit, dQ within its last bit, over replays that share a workspace
    with a call of another shape; outputs at 16-byte boundaries."""
    attn = _lib()
    Q, K, V, dO, lam = (t.cuda() for t in problem(1, 4, 2, 300, 300, 128, 5))
    O, O2, L = attn.attn_fwd_diff(Q, K, V, lam, causal=True)
    base = attn.attn_bwd_diff(Q, K, V, lam, O, O2, dO, L, causal=True)
    n = attn.attn_bwd_diff_workspace_size(1, 4, 2, 300, 300, 128)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    odd = [torch.empty(t.numel() + 8, dtype=BF, device="cuda")[8:].view(t.shape) for t in base[:3]]
    assert odd[1].data_ptr() % 32 == 16
    call = lambda: attn.attn_bwd_diff(Q, K, V, lam, O, O2, dO, L, causal=True, workspace=ws,
                                      dQ=odd[0], dK=odd[1], dV=odd[2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    half = [t[:, :, :150].contiguous() for t in (Q, K, V, dO)]
    h = attn.attn_fwd_diff(*half[:3], lam)
    for _ in range(2):
        attn.attn_bwd_diff(*half[:3], lam, h[0], h[1], half[3], h[2], workspace=ws)
        for t in odd:
            t.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[1], base[1]) and torch.equal(got[2], base[2])
        assert torch.equal(got[3], base[3])
        assert (got[0].float() - base[0].float()).norm() <= 2e-3 * base[0].float().norm()
    assert attn.attn_read_device_status(ws) == (0, 0)


@pytest.mark.gpu
def test_bwd_reports_a_bad_length():
    attn = _lib()
    Q, K, V, dO, lam = (t.cuda() for t in problem(2, 2, 2, 140, 140, 64, 6))
    kl = torch.tensor([140, -3], dtype=I32, device="cuda")
    O, O2, L = attn.attn_fwd_diff(Q, K, V, lam, k_lens=kl)
    ws = torch.zeros(attn.attn_bwd_diff_workspace_size(2, 2, 2, 140, 140, 64), dtype=torch.uint8,
                     device="cuda")
    dQ, dK, dV, dlam = attn.attn_bwd_diff(Q, K, V, lam, O, O2, dO, L, k_lens=kl, workspace=ws)
    assert attn.attn_read_device_status(ws) == (attn.ATTN_ERR_INVALID, attn.ATTN_DEV_BAD_KLEN)
    assert all(bool((t[1] == 0).all()) for t in (dQ, dK, dV))
    want = ref.bwd(*(t[:1].cpu() for t in (Q, K, V)), lam.cpu(), dO[:1].cpu())
    for g, w in zip((dQ, dK, dV), want):
        assert _rel(g[:1], w) <= BAR


@pytest.mark.gpu
def test_bwd_training_size_sampled():
    """B=2, H=16, L=8192, d=128, causal: sampled rows of dQ of two heads, dK and dV of the last
    keys (few rows see them), against the formulas on slices that hold all they depend on."""
    attn = _lib()
    B, H, L, d = 2, 16, 8192, 128
    g = torch.Generator(device="cuda").manual_seed(21)
    rn = lambda: torch.randn(B, H, L, d, generator=g, device="cuda").to(BF)
    Q, K, V, dO = rn(), rn(), rn(), rn()
    lam = torch.rand(H, generator=g, device="cuda")
    O, O2, lse = attn.attn_fwd_diff(Q, K, V, lam, causal=True)
    dQ, dK, dV, _ = attn.attn_bwd_diff(Q, K, V, lam, O, O2, dO, lse, causal=True)
    for b, h in ((0, 0), (1, 15)):
        w = lam[h:h + 1].cpu()
        for r0, r1 in ((0, 40), (4000, 4040), (L - 40, L)):
            # rows r0..r1 against their keys 0..r1: the causal mask aligned to the corner
            s = [Q[b, h, r0:r1], K[b, h, :r1], V[b, h, :r1], dO[b, h, r0:r1]]
            q, k, v, do = (t.cpu()[None, None] for t in s)
            rq, rk, rv, _ = ref.bwd(q, k, v, w, do, causal=True)
            assert _rel(dQ[b, h, r0:r1], rq[0, 0]) <= BAR, (b, h, r0)
        # the last 40 keys are seen by the last 40 rows alone
        assert _rel(dK[b, h, L - 40:], rk[0, 0, L - 40:]) <= BAR
        assert _rel(dV[b, h, L - 40:], rv[0, 0, L - 40:]) <= BAR


def test_bwd_rejections():
    attn = _lib()
    B, Hq, Hkv, L, d = 2, 4, 2, 16, 128
    Q, KV, lam = FakeCuda((B, Hq, L, d), BF), FakeCuda((B, Hkv, L, d), BF), FakeCuda((Hq,), F32)
    lse = FakeCuda((B, Hq, 2, L), F32)

    def call(O=Q, O2=Q, dO=Q, L_=lse, w=lam, **kw):
        return lambda: attn.attn_bwd_diff(Q, KV, KV, w, O, O2, dO, L_, **kw)

    rejects(call(O2=None), "O2", "required")
    rejects(call(O=KV), "O")
    rejects(call(dO=FakeCuda((B, Hq, L, d), F32)), "dO", "bfloat16")
    rejects(call(dO=FakeCuda((B, Hq, L, d), BF, contiguous=False)), "dO", "contiguous")
    rejects(call(L_=FakeCuda((B, Hq, L), F32)), "lse")
    rejects(call(w=FakeCuda((Hkv,), F32)), "lam")
    rejects(call(dlam=FakeCuda((Hq,), F32)), "dlam", "bfloat16")
    rejects(call(w=FakeCuda((1,), F32), dlam=FakeCuda((Hq,), BF)), "dlam")
    rejects(call(dK=Q), "dK")
    rejects(call(workspace=FakeCuda((256,), torch.uint8)), "workspace", "needs")


def test_bwd_rejects_on_host():
    import ctypes

    attn = _lib()
    P = ctypes.c_void_p(256 * 1024)

    def call(Q=P, K=P, lam=P, n_lam=2, O2=P, dO=P, lse=P, dV=P, dlam=P, B=1, Hq=2, Hkv=1, Lq=8,
             Lk=8, d=128, scale=0.1, mask=0, nb=1 << 24):
        return attn.lib().attn_bwd_diff(Q, K, P, lam, n_lam, P, O2, dO, lse, P, P, dV, dlam, B, Hq,
                                        Hkv, Lq, Lk, d, scale, mask, None, P, nb, None)

    for bad in (dict(Q=None), dict(K=None), dict(lam=None), dict(n_lam=3), dict(O2=None),
                dict(dO=None), dict(lse=None), dict(dV=None), dict(dlam=None),
                dict(Hq=3, Hkv=2, n_lam=3), dict(scale=-1.0), dict(mask=2), dict(nb=256),
                dict(dlam=ctypes.c_void_p(256 * 1024 + 1)),
                dict(dO=ctypes.c_void_p(256 * 1024 + 8))):
        assert call(**bad) == attn.ATTN_ERR_INVALID, bad
    assert call(d=96) == attn.ATTN_ERR_UNSUPPORTED
    assert call(B=1 << 20, Lq=1 << 20, nb=1 << 62) == attn.ATTN_ERR_UNSUPPORTED


def test_bwd_workspace_is_a_closed_form():
    """fp32 dQ accumulator and four statistics per query row (padded to 128 per head), 16 partial
    sums of dlam per (sequence, head, 128-key tile, part), and with several parts each
    one's fp32 dV and dK."""
    attn = _lib()

    def want(B, Hq, Hkv, Lq, Lk, d, parts):
        rows = B * Hq * ((max(Lq, 1) + 127) // 128 * 128)
        n = rows * d * 4 + rows * 16 + B * Hq * ((Lk + 127) // 128) * parts * 64
        n += parts * B * Hkv * Lk * d * 8 if parts > 1 else 0
        return 256 + (n + 255) // 256 * 256

    for a, parts in (((2, 16, 16, 8192, 8192, 128), 1), ((1, 6, 2, 100, 300, 64), 3)):
        assert attn.attn_bwd_diff_workspace_size(*a) == want(*a, parts)
