"""attn_fwd_splitkv_decode_diff and its paged form against the definition in 64 bits, and a
decode loop that appends to the cache it reads."""

import math

import pytest
import torch

from tests import _diff_ref as ref
from tests.test_append_paged import _tables
from tests.test_binding_validation import FakeCuda, rejects

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _lib():
    import exact_io_aware_46_b200 as attn

    return attn


def _pages(K, V, page, seed, fill):
    """[B,Hkv,Lmax,d] caches -> pages in random order (rows without a token hold `fill`) and
    the block table."""
    B, Hkv, L, d = K.shape
    nb = (L + page - 1) // page
    order = torch.randperm(B * nb + 2, generator=torch.Generator().manual_seed(seed))
    table = order[:B * nb].view(B, nb)
    out = []
    for x in (K, V):
        p = torch.full((B * nb + 2, Hkv, page, d), fill, dtype=BF)
        for b in range(B):
            for j in range(nb):
                rows = x[b, :, j * page:(j + 1) * page]
                p[table[b, j], :, :rows.shape[1]] = rows
        out.append(p)
    return out[0], out[1], table.to(I32)


def _problem(B, Hq, Hkv, Lmax, d, lens, seed, fill=math.nan):
    """Caches whose rows past each sequence's length hold `fill`."""
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g).to(BF)
    Q, K, V = rn(B, Hq, 1, d), rn(B, Hkv, Lmax, d), rn(B, Hkv, Lmax, d)
    for b, n in enumerate(lens):
        K[b, :, n:], V[b, :, n:] = fill, fill
    return Q, K, V, torch.rand(Hq, generator=g) * 1.6 - 0.3


CASES = [
    # B, Hq, Hkv, Lmax, d, lengths, page
    (1, 1, 1, 1, 128, [1], 16),                              # one token of all
    (2, 2, 2, 300, 128, [300, 129], 16),
    (3, 4, 2, 700, 128, [0, 1, 700], 64),                    # an empty sequence
    (2, 6, 2, 520, 128, [513, 257], 32),                     # groups of three; one past a split
    (1, 8, 1, 1000, 128, [999], 128),                        # groups of eight
    (2, 16, 2, 2049, 64, [2049, 640], 16),
    (3, 5, 1, 200, 64, [200, 64, 65], 64),                   # groups of five, pages end in a tile
    (1, 4, 4, 4200, 64, [4111], 1024),                       # many splits, large pages
    (40, 8, 4, 2500, 128, [(61 * b) % 2501 for b in range(40)], 64),   # longer splits
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,Lmax,d,lens,page", CASES)
def test_decode_matches_definition(B, Hq, Hkv, Lmax, d, lens, page):
    attn = _lib()
    Q, K, V, lam = _problem(B, Hq, Hkv, Lmax, d, lens, 31 + Lmax + d + Hq)
    O, _, lse, tol, _ = ref.fwd(Q, K, V, lam, k_lens=lens)
    kl = torch.tensor(lens, dtype=I32, device="cuda")
    o, l = attn.attn_fwd_splitkv_decode_diff(Q.cuda(), K.cuda(), V.cuda(), lam.cuda(), kl)
    ref.assert_within(o, O, tol, "O")
    ref.assert_lse(l, lse[..., 0])
    kp, vp, table = _pages(K, V, page, 3, math.nan)
    op, lp = attn.attn_fwd_splitkv_decode_diff_paged(Q.cuda(), kp.cuda(), vp.cuda(), table.cuda(),
                                                     lam.cuda(), kl)
    ref.assert_within(op, O, tol, "paged O")
    ref.assert_lse(lp, lse[..., 0], "paged LSE")


@pytest.mark.gpu
@pytest.mark.parametrize("d,Hq,Hkv", [(64, 8, 4), (128, 4, 4), (128, 32, 4)])
def test_decode_large_scores_in_long_splits(d, Hq, Hkv):
    """Scale 1 and enough sequences for splits of many 128-key blocks: the maxima move from block
    to block, after the next block's scores were formed."""
    attn = _lib()
    B, Lmax = 40, 1500
    lens = [(37 * b * b + 1) % (Lmax + 1) for b in range(B)]
    Q, K, V, lam = _problem(B, Hq, Hkv, Lmax, d, lens, 13)
    K *= torch.linspace(0.2, 1.5, Lmax)[:, None].to(BF)  # later keys score higher
    for b, n in enumerate(lens):
        K[b, :, n:] = math.nan
    O, _, lse, tol, _ = ref.fwd(Q, K, V, lam, scale=1.0, k_lens=lens)
    kl = torch.tensor(lens, dtype=I32, device="cuda")
    o, l = attn.attn_fwd_splitkv_decode_diff(Q.cuda(), K.cuda(), V.cuda(), lam.cuda(), kl, scale=1.0)
    ref.assert_within(o, O, tol, "O")
    ref.assert_lse(l, lse[..., 0])
    kp, vp, table = _pages(K, V, 64, 3, math.nan)
    op, lp = attn.attn_fwd_splitkv_decode_diff_paged(Q.cuda(), kp.cuda(), vp.cuda(), table.cuda(),
                                                     lam.cuda(), kl, scale=1.0)
    assert torch.equal(op, o) and torch.equal(lp, l)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_decode_large_scores_one_weight_and_infinities_past_the_end(d):
    """Scale 1: the running maxima jump from split to split; garbage is infinite."""
    attn = _lib()
    lens = [777, 130]
    Q, K, V, lam = _problem(2, 4, 2, 900, d, lens, 6, fill=-math.inf)
    O, _, lse, tol, _ = ref.fwd(Q, K, V, lam[:1], scale=1.0, k_lens=lens)
    o, l = attn.attn_fwd_splitkv_decode_diff(Q.cuda(), K.cuda(), V.cuda(), lam[:1].cuda(),
                                             torch.tensor(lens, dtype=I32, device="cuda"),
                                             scale=1.0)
    ref.assert_within(o, O, tol, "O")
    ref.assert_lse(l, lse[..., 0])


@pytest.mark.gpu
def test_decode_reports_bad_lengths_and_pages():
    attn = _lib()
    lens = [600, 600, 600]
    Q, K, V, lam = _problem(3, 4, 2, 600, 128, lens, 9)
    kp, vp, table = _pages(K, V, 16, 8, 0.0)
    O, _, _, tol, _ = ref.fwd(Q, K, V, lam, k_lens=lens)
    table[1, 3] = kp.shape[0]                       # in the first split of sequence 1
    kl = torch.tensor([600, 600, 609], dtype=I32)   # sequence 2: past its 608 rows
    n = attn.attn_decode_diff_workspace_size(3, 4, 2, table.shape[1] * 16, 128)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    o, l = attn.attn_fwd_splitkv_decode_diff_paged(Q.cuda(), kp.cuda(), vp.cuda(), table.cuda(),
                                                   lam.cuda(), kl.cuda(), workspace=ws)
    code, bits = attn.attn_read_device_status(ws)
    assert code == attn.ATTN_ERR_INVALID
    assert bits == attn.ATTN_DEV_BAD_KLEN | attn.ATTN_DEV_BAD_PAGE
    ref.assert_within(o[0], O[0], tol[0], "the sound sequence")
    assert torch.isfinite(o).all() and (o[2] == 0).all() and (l[2] == -math.inf).all()


@pytest.mark.gpu
def test_append_then_decode_steps_in_a_graph():
    """Serving steps: k_lens grows, the append rotates and stores, the decode reads the cache;
    captured once and replayed, against the whole history in 64 bits."""
    attn = _lib()
    B, Hq, Hkv, d, page, cap = 3, 4, 2, 128, 16, 96
    g = torch.Generator().manual_seed(4)
    cos, sin = _tables(cap, 32)
    kp = torch.full((B * cap // page, Hkv, page, d), math.nan, dtype=BF, device="cuda")
    vp = kp.clone()
    table = torch.randperm(B * cap // page, generator=g).view(B, -1).to(I32).cuda()
    lam = torch.rand(Hq, generator=g)
    lens = torch.zeros(B, dtype=I32, device="cuda")
    prompt = [17, 1, 30]
    T = sum(prompt)
    new = lambda n, h: torch.randn(n, h, d, generator=g).to(BF)
    K, V = new(T, Hkv), new(T, Hkv)
    cu = torch.tensor([0, 17, 18, 48], dtype=I32)
    lens += torch.tensor(prompt, dtype=I32, device="cuda")
    rope = dict(cos=cos.cuda(), sin=sin.cuda(), maps=2)
    attn.attn_kv_append_paged(K.cuda(), V.cuda(), kp, vp, table, lens, cu_seqlens=cu.cuda(), **rope)
    hist = [[(K[a:b], V[a:b])] for a, b in zip(cu[:-1], cu[1:])]
    q, k, v = (torch.zeros(B, h, d, dtype=BF, device="cuda") for h in (Hq, Hkv, Hkv))
    lam_d = lam.cuda()
    qr = torch.zeros_like(q)
    ws = torch.zeros(attn.attn_decode_diff_workspace_size(B, Hq, Hkv, cap, d), dtype=torch.uint8,
                     device="cuda")
    O = torch.zeros(B, Hq, 1, d, dtype=BF, device="cuda")
    lse = torch.zeros(B, Hq, 2, device="cuda")

    def step():
        lens.add_(1)
        attn.attn_kv_append_paged(k, v, kp, vp, table, lens, Q=q, Q_out=qr, workspace=ws, **rope)
        attn.attn_fwd_splitkv_decode_diff_paged(qr.view(B, Hq, 1, d), kp, vp, table, lam_d, lens,
                                                O=O, lse=lse, workspace=ws)

    step()  # warm-up outside the graph; its row is appended again below
    lens.sub_(1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        nq, nk, nv = new(B, Hq), new(B, Hkv), new(B, Hkv)
        for dst, src in ((q, nq), (k, nk), (v, nv)):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        for b in range(B):
            hist[b].append((nk[b:b + 1], nv[b:b + 1]))
            kb, vb = (torch.cat([h[i] for h in hist[b]]) for i in (0, 1))
            n = kb.shape[0]
            # the cache holds the rotated rows rounded to bf16: the same within a rounding
            # there are no ties in the way, so the 64-bit rotation rounds to the same values
            # except where fp32 falls on the other side; the decode's own bound is checked
            # against the rows as stored
            stored = kp[table[b].long()].transpose(0, 1).reshape(Hkv, cap, d)[:, :n].cpu()
            y = ref.rotate(kb, cos[:n], sin[:n], 2, False).transpose(0, 1)
            bound = ref.rotation_bound(kb, y.transpose(0, 1), 2, 32, False).transpose(0, 1)
            ref.assert_within(stored, y, bound, "rotated keys")
            assert torch.equal(vp[table[b].long()].transpose(0, 1).reshape(Hkv, cap, d)[:, :n].cpu(),
                               vb.transpose(0, 1))
            o, _, l, tol, _ = ref.fwd(qr[b:b + 1].view(1, Hq, 1, d).cpu(), stored[None],
                                      vb.transpose(0, 1)[None], lam)
            ref.assert_within(O[b:b + 1], o, tol, "O")
            ref.assert_lse(lse[b:b + 1], l[..., 0])
    assert attn.attn_read_device_status(ws) == (0, 0)


def test_decode_rejections():
    attn = _lib()
    B, Hq, Hkv, d = 2, 4, 2, 128
    Q, cache, kl = FakeCuda((B, Hq, 1, d), BF), FakeCuda((B, Hkv, 256, d), BF), FakeCuda((B,), I32)
    lam = FakeCuda((Hq,), F32)
    f = attn.attn_fwd_splitkv_decode_diff
    rejects(lambda: f(Q, cache, cache, FakeCuda((3,), F32), kl), "lam")
    rejects(lambda: f(Q, cache, cache, FakeCuda((Hq,), BF), kl), "lam", "float32")
    rejects(lambda: f(Q, cache, cache, torch.zeros(Hq), kl), "lam", "CUDA")
    rejects(lambda: f(FakeCuda((B, Hq, 2, d), BF), cache, cache, lam, kl), "Q", "1")
    rejects(lambda: f(Q, cache, cache, lam, None), "k_lens")
    rejects(lambda: f(Q, FakeCuda((3, Hkv, 256, d), BF), FakeCuda((3, Hkv, 256, d), BF), lam, kl),
            "Kcache")
    rejects(lambda: f(Q, cache, cache, lam, kl, lse=FakeCuda((B, Hq), F32)), "lse")
    g = attn.attn_fwd_splitkv_decode_diff_paged
    pages, tab = FakeCuda((40, Hkv, 16, d), BF), FakeCuda((B, 16), I32)
    rejects(lambda: g(Q, pages, pages, None, lam, kl), "block_table")
    rejects(lambda: g(Q, pages, pages, FakeCuda((3, 16), I32), lam, kl), "block_table")
    rejects(lambda: g(Q, pages, FakeCuda((40, Hkv, 32, d), BF), tab, lam, kl), "Vpages")
    rejects(lambda: g(Q, pages, pages, tab, lam, kl, workspace=FakeCuda((256,), torch.uint8)),
            "workspace", "needs")


def test_decode_rejects_on_host():
    import ctypes

    attn = _lib()
    P = ctypes.c_void_p(256 * 1024)

    def call(lam=P, n_lam=4, Hq=4, Hkv=2, L=256, d=128, kl=P, nb=1 << 24, K=P):
        return attn.lib().attn_fwd_splitkv_decode_diff(P, K, P, lam, n_lam, P, None, 2, Hq, Hkv, L,
                                                       d, 0.1, kl, P, nb, None)

    for bad in (dict(lam=None), dict(n_lam=3), dict(n_lam=0), dict(kl=None), dict(nb=256),
                dict(Hq=3), dict(K=None), dict(L=-1)):
        assert call(**bad) == attn.ATTN_ERR_INVALID, bad
    assert call(d=96) == attn.ATTN_ERR_UNSUPPORTED
    assert call(Hq=18, Hkv=2, n_lam=18) == attn.ATTN_ERR_UNSUPPORTED  # nine heads a group

    def paged(bt=P, mb=16, page=16, n_pages=40):
        return attn.lib().attn_fwd_splitkv_decode_diff_paged(P, P, P, bt, mb, page, n_pages, P, 1, P,
                                                             None, 2, 4, 2, 128, 0.1, P, P,
                                                             1 << 24, None)

    assert paged(bt=None) == 1 and paged(mb=0) == 1 and paged(n_pages=0) == 1
    assert paged(page=24) == 2 and paged(page=8) == 2


def test_decode_workspace_is_a_closed_form():
    """fp32 partial output and log-sum-exp per (sequence, head, map, split); a split is the
    longest of 2048, 1024, 512, 256 and 128 rows that gives 148 of them, 128 at least."""
    attn = _lib()

    def want(B, Hq, Hkv, L, d, ch):
        n = B * Hq * 2 * ((L + ch - 1) // ch)
        return 256 + (n * d * 4 + n * 4 + 255) // 256 * 256

    for a, ch in (((64, 32, 8, 32768, 128), 2048), ((1, 32, 8, 4096, 128), 128),
                  ((1, 32, 8, 131072, 128), 2048), ((2, 16, 2, 40000, 64), 1024)):
        assert attn.attn_decode_diff_workspace_size(*a) == want(*a, ch)
