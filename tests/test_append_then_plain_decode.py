"""The append and the plain paged decode together: pages allocated zeroed, and pages handed on from
another sequence with its rows still in them (the plain decode reads whole 128-row blocks, so it
wants finite values behind a sequence's end)."""

import math

import pytest
import torch

from tests import _diff_ref as ref
from tests.test_append_paged import _tables

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


def _decode(q, k, v):
    """Plain attention of one row a head in 64 bits: (O, LSE, bound of O); q [Hq, d], k and v
    [Hkv, n, d].  The kernel rounds the probabilities and O to bf16."""
    G = q.shape[0] // k.shape[0]
    k, v = (x.double().repeat_interleave(G, 0) for x in (k, v))
    s = torch.einsum("hd,hnd->hn", q.double(), k) / math.sqrt(q.shape[-1])
    p = s.softmax(-1)
    O = torch.einsum("hn,hnd->hd", p, v)
    bound = (ref.U_BF16 + ref.E_PROB) * torch.einsum("hn,hnd->hd", p, v.abs())
    return O, torch.logsumexp(s, -1), bound + ref.U_BF16 * O.abs()


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("d", [64, 128])
def test_prompts_and_steps_on_zeroed_and_on_recycled_pages(d, page):
    import exact_io_aware_46_b200 as attn

    B, Hq, Hkv, cap = 3, 4, 2, 512
    g = torch.Generator().manual_seed(5 + d + page)
    new = lambda n, h: torch.randn(n, h, d, generator=g).to(BF)
    nb = cap // page
    cos, sin = _tables(cap, d // 2)
    rope = dict(cos=cos.cuda(), sin=sin.cuda())
    kp = torch.zeros(B * nb, Hkv, page, d, dtype=BF, device="cuda")
    vp = torch.zeros_like(kp)
    for prompt in ([130, 1, 300], [17, 200, 3]):  # the second on the first's pages
        table = torch.randperm(B * nb, generator=g).view(B, nb).to(I32).cuda()
        cu = torch.tensor([0] + torch.tensor(prompt).cumsum(0).tolist(), dtype=I32)
        lens = torch.tensor(prompt, dtype=I32, device="cuda")
        K, V = new(sum(prompt), Hkv), new(sum(prompt), Hkv)
        attn.attn_kv_append_paged(K.cuda(), V.cuda(), kp, vp, table, lens, cu_seqlens=cu.cuda(),
                                  **rope)
        hist = [[(K[a:b], V[a:b])] for a, b in zip(cu[:-1], cu[1:])]
        for _ in range(2):
            q, k, v = new(B, Hq), new(B, Hkv), new(B, Hkv)
            lens += 1
            qr = attn.attn_kv_append_paged(k.cuda(), v.cuda(), kp, vp, table, lens, Q=q.cuda(),
                                           **rope)
            o, l = attn.attn_fwd_splitkv_decode_paged(qr.view(B, Hq, 1, d), kp, vp, table, lens)
            for b in range(B):
                hist[b].append((k[b:b + 1], v[b:b + 1]))
                kb, vb = (torch.cat([x[i] for x in hist[b]]) for i in (0, 1))
                n = kb.shape[0]
                rows = lambda pages: pages[table[b].long()].transpose(0, 1).reshape(
                    Hkv, cap, d)[:, :n].cpu()
                y = ref.rotate(kb, cos[:n], sin[:n], 1, False).transpose(0, 1)
                bound = ref.rotation_bound(kb, y.transpose(0, 1), 1, d // 2, False)
                ref.assert_within(rows(kp), y, bound.transpose(0, 1), "rotated keys")
                assert torch.equal(rows(vp), vb.transpose(0, 1))
                O, lse, tol = _decode(qr[b].cpu(), rows(kp), rows(vp))
                ref.assert_within(o[b, :, 0], O, tol, "O")
                ref.assert_lse(l[b], lse)
