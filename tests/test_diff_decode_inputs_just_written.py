"""Lengths and weights written by the kernel right before a differential decode, many times without
a pause: each decode sees its own (its kernels are set up while the one before still runs)."""

import pytest
import torch

from tests.test_diff_decode import _problem

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.mark.parametrize("B,Lmax", [(1, 300), (4, 2000)])
def test_decodes_between_writes_of_their_lengths_and_weights(B, Lmax):
    import exact_io_aware_46_b200 as attn

    d, Hq, Hkv, n = 64, 8, 2, 16
    Q, K, V, lam = (t.cuda() for t in _problem(B, Hq, Hkv, Lmax, d, [Lmax] * B, 21))
    g = torch.Generator().manual_seed(2)
    lens = torch.randint(0, Lmax + 1, (n, B), generator=g).to(I32).cuda()
    lams = torch.rand(n, Hq, generator=g).cuda()
    want = [attn.attn_fwd_splitkv_decode_diff(Q, K, V, lams[i].clone(), lens[i].clone())
            for i in range(n)]
    torch.cuda.synchronize()
    ws = torch.zeros(attn.attn_decode_diff_workspace_size(B, Hq, Hkv, Lmax, d), dtype=torch.uint8,
                     device="cuda")
    kl, w = torch.zeros(B, dtype=I32, device="cuda"), torch.zeros(Hq, device="cuda")
    got = [(torch.empty_like(o), torch.empty_like(l)) for o, l in want]
    for _ in range(20):
        for i in range(n):
            kl.copy_(lens[i])
            w.copy_(lams[i])
            attn.attn_fwd_splitkv_decode_diff(Q, K, V, w, kl, O=got[i][0], lse=got[i][1],
                                              workspace=ws)
    torch.cuda.synchronize()
    for (a, la), (o, l) in zip(got, want):
        assert torch.equal(a, o) and torch.equal(la, l)
