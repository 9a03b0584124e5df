"""The differential calls and the append together: overlapping streams, sizes past 2^31 elements,
and a training step beside a serving step."""

import math

import pytest
import torch

from tests import _diff_ref as ref
from tests.test_append_paged import _tables
from tests.test_diff_fwd import problem

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


def _lib():
    import exact_io_aware_46_b200 as attn

    return attn


def _like(got, want, what):
    """The same call twice: dQ's additions come in no fixed order, everything else is equal."""
    for name, a, b in zip(what, got, want):
        if name == "dQ":
            assert (a.float() - b.float()).norm() <= 2e-3 * b.float().norm()
        else:
            assert torch.equal(a, b), name


def test_training_and_decode_steps_on_two_streams_at_once():
    """A forward and backward on one stream, append and decode on another, each with its own
    workspaces, overlapping for many rounds: what each gives alone."""
    attn = _lib()
    Q, K, V, dO, lam = (t.cuda() for t in problem(2, 8, 2, 500, 500, 128, 61))
    B, Hq, Hkv, d, page, cap = 8, 8, 2, 128, 16, 2048
    g = torch.Generator(device="cuda").manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)
    kp, vp = rn(B * cap // page, Hkv, page, d), rn(B * cap // page, Hkv, page, d)
    table = torch.randperm(B * cap // page, generator=g, device="cuda").view(B, -1).to(I32)
    lens = torch.tensor([1 + 250 * b for b in range(B)], dtype=I32, device="cuda")
    q, k, v = rn(B, Hq, d), rn(B, Hkv, d), rn(B, Hkv, d)
    cos, sin = (t.cuda() for t in _tables(cap, 32))

    def train():
        O, O2, L = attn.attn_fwd_diff(Q, K, V, lam, causal=True)
        return (O, O2, L) + attn.attn_bwd_diff(Q, K, V, lam, O, O2, dO, L, causal=True)

    def serve():
        qr = attn.attn_kv_append_paged(k, v, kp, vp, table, lens, Q=q, cos=cos, sin=sin, maps=2)
        return (qr,) + attn.attn_fwd_splitkv_decode_diff_paged(qr.view(B, Hq, 1, d), kp, vp, table,
                                                               lam, lens)

    want = train(), serve()
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        with torch.cuda.stream(one):
            a = train()
        with torch.cuda.stream(two):
            b = serve()
        got.append((a, b))
    torch.cuda.synchronize()
    for a, b in got:
        _like(a, want[0], ("O", "O2", "LSE", "dQ", "dK", "dV", "dlam"))
        _like(b, want[1], ("Q", "O", "LSE"))


def test_append_past_2_31_elements():
    """A cache of 2^31 + 2^27 elements: the last page is written and nothing else of its table."""
    attn = _lib()
    Hkv, page, d = 8, 64, 128
    n_pages = (2 ** 31 + 2 ** 27) // (Hkv * page * d)
    kp = torch.zeros(n_pages, Hkv, page, d, dtype=BF, device="cuda")
    vp = torch.zeros_like(kp)
    g = torch.Generator().manual_seed(8)
    K, V = (torch.randn(3, Hkv, d, generator=g).to(BF).cuda() for _ in "KV")
    pages = [n_pages - 1, n_pages // 2, 2 ** 31 // (Hkv * page * d)]
    table = torch.tensor([[p] for p in pages], dtype=I32, device="cuda")
    lens = torch.tensor([64, 1, 30], dtype=I32, device="cuda")
    attn.attn_kv_append_paged(K, V, kp, vp, table, lens)
    for b, p in enumerate(pages):
        row = int(lens[b]) - 1
        assert torch.equal(kp[p, :, row], K[b]) and torch.equal(vp[p, :, row], V[b])
        assert int((kp[p] != 0).any(-1).sum()) == Hkv
    assert int((vp != 0).any(-1).any(-1).any(-1).sum()) == 3


def test_fwd_and_bwd_past_2_31_elements():
    """[1040, 16, 1040, 128]: the first head, the one whose rows cross element 2^31, the last."""
    attn = _lib()
    B, H, L, d = 1040, 16, 1040, 128
    assert B * H * L * d > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(2)

    def rn():
        x = torch.empty(B, H, L, d, dtype=BF, device="cuda")
        for b in range(0, B, 65):  # in slices: the random numbers are drawn in 32 bits
            x[b:b + 65] = torch.randn(65, H, L, d, generator=g, device="cuda").to(BF)
        return x

    Q, K, V, dO = rn(), rn(), rn(), rn()
    lam = torch.rand(H, generator=g, device="cuda")
    O, O2, lse = attn.attn_fwd_diff(Q, K, V, lam, causal=True)
    dQ, dK, dV, _ = attn.attn_bwd_diff(Q, K, V, lam, O, O2, dO, lse, causal=True)
    cross = 2 ** 31 // (L * d)
    for bh in (0, cross, B * H - 1):
        b, h = divmod(bh, H)
        one = [t[b:b + 1, h:h + 1].cpu() for t in (Q, K, V, dO)]
        w = lam[h:h + 1].cpu()
        o, o2, l, tol, tol2 = ref.fwd(*one[:3], w, causal=True)
        ref.assert_within(O[b, h], o[0, 0], tol[0, 0], f"O of head {bh}")
        ref.assert_within(O2[b, h], o2[0, 0], tol2[0, 0], f"O2 of head {bh}")
        ref.assert_lse(lse[b, h], l[0, 0])
        want = ref.bwd(*one[:3], w, one[3], causal=True)
        for got, r, name in zip((dQ, dK, dV), want, ("dQ", "dK", "dV")):
            e = (got[b, h].double().cpu() - r[0, 0]).norm() / r.norm()
            assert e <= 1e-2, f"{name} of head {bh}: {e:.3e}"


def test_a_shared_weight_trains_like_copies_of_it():
    """One weight for all heads: the same outputs as H equal weights, and their gradients' sum."""
    attn = _lib()
    Q, K, V, dO, lam = (t.cuda() for t in problem(1, 8, 4, 300, 300, 64, 19))
    one, many = lam[:1].contiguous(), lam[:1].expand(8).contiguous()
    out = []
    for w in (one, many):
        O, O2, L = attn.attn_fwd_diff(Q, K, V, w, causal=True)
        out.append((O, O2, L) + attn.attn_bwd_diff(Q, K, V, w, O, O2, dO, L, causal=True))
    _like(out[0][:6], out[1][:6], ("O", "O2", "LSE", "dQ", "dK", "dV"))
    a, b = out[0][6].double().sum().item(), out[1][6].double()
    # each of the eight is rounded once to bf16, the shared one too
    assert math.isclose(a, b.sum().item(), rel_tol=0, abs_tol=2 ** -8 * (b.abs().sum().item() + abs(a)))


@pytest.mark.parametrize("d", [64, 128])
def test_a_row_that_is_not_a_number_stays_one(d):
    """A NaN in a query row is a NaN in that row's results, and in no other row's; a row that sees
    no key still gets zeros."""
    attn = _lib()
    Q, K, V, _, lam = (t.cuda() for t in problem(2, 4, 2, 150, 140, d, 71))
    want = attn.attn_fwd_diff(Q, K, V, lam, causal=True)
    bad = Q.clone()
    bad[1, 2, [3, 40, 149]] = math.nan  # row 3 sees no key (150 queries, 140 keys)
    O, O2, L = attn.attn_fwd_diff(bad, K, V, lam, causal=True)
    hit = torch.zeros(2, 4, 150, dtype=torch.bool, device="cuda")
    hit[1, 2, [40, 149]] = True
    for got, ref_ in ((O, want[0]), (O2, want[1])):
        assert got[hit].isnan().all() and torch.equal(got[~hit], ref_[~hit])
    lh = hit[:, :, None].expand(2, 4, 2, 150)
    assert L[lh].isnan().all() and torch.equal(L[~lh], want[2][~lh])
    assert (O[:, :, :10] == 0).all() and (L[..., :10] == -math.inf).all()

    lens = torch.tensor([140, 77], dtype=I32, device="cuda")
    q = Q[:, :, -1:].contiguous()
    want = attn.attn_fwd_splitkv_decode_diff(q, K, V, lam, lens)
    q[1, 3] = math.nan
    O, L = attn.attn_fwd_splitkv_decode_diff(q, K, V, lam, lens)
    hit = torch.zeros(2, 4, dtype=torch.bool, device="cuda")
    hit[1, 3] = True
    assert O[hit].isnan().all() and torch.equal(O[~hit], want[0][~hit])
    assert L[hit].isnan().all() and torch.equal(L[~hit], want[1][~hit])


@pytest.mark.parametrize("fill", [0x7F, 0x80, 0xFF])
@pytest.mark.parametrize("extra", [0, 1])
def test_calls_need_no_cleared_workspace_but_for_its_status(fill, extra):
    """As many query tiles as SMs, and one more: on memory that holds anything, the calls that may
    go without clearing give what they give on cleared workspaces."""
    attn = _lib()
    B, Hq, L, d = 1, attn.attn_num_sms() + extra, 128, 64
    Q, K, V, dO, lam = (t.cuda() for t in problem(B, Hq, Hq, L, L, d, 81))
    lens = torch.tensor([L], dtype=I32, device="cuda")
    kp, vp, table = K.clone(), V.clone(), torch.zeros(1, 1, dtype=I32, device="cuda")
    tok = Q[0, :, :1].transpose(0, 1).contiguous()

    def run(ws):
        O, O2, lse = attn.attn_fwd_diff(Q, K, V, lam, workspace=ws(attn.attn_fwd_diff_workspace_size(
            B, Hq, Hq, L, L, d), extra == 0))
        out = (O, O2, lse) + attn.attn_bwd_diff(Q, K, V, lam, O, O2, dO, lse, workspace=ws(
            attn.attn_bwd_diff_workspace_size(B, Hq, Hq, L, L, d), True))
        qr = attn.attn_kv_append_paged(tok, tok, kp, vp, table, lens, Q=tok, workspace=ws(
            attn.attn_kv_append_paged_workspace_size(), True))
        return out + (qr, kp) + attn.attn_fwd_splitkv_decode_diff(
            qr.view(B, Hq, 1, d), kp, vp, lam, lens, workspace=ws(
                attn.attn_decode_diff_workspace_size(B, Hq, Hq, L, d), True))

    what = ("O", "O2", "lse", "dQ", "dK", "dV", "dlam", "q", "pages", "dO", "dlse")

    def any_memory(n, may):
        return torch.full((n,), fill if may else 0, dtype=torch.uint8, device="cuda")

    want = run(lambda n, may: torch.zeros(n, dtype=torch.uint8, device="cuda"))
    for _ in range(3):
        _like(run(any_memory), want, what)
    # the binding's own workspaces, handed out where a filled block was
    for _ in range(3):
        for n in (256, 1 << 16, 1 << 20, 1 << 23):
            torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        _like(run(lambda n, may: None), want, what)
