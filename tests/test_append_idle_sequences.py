"""attn_kv_append_paged: the length of a sequence that gets no token is checked like the others'."""

import pytest
import torch

BF, I32 = torch.bfloat16, torch.int32


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 3, 200])
def test_a_bad_length_of_a_sequence_without_tokens_is_reported(B):
    """One token for sequence 0, none for the others (more of them than a block has threads): a
    length below zero or past the cache sets the status, and the token is still appended."""
    import exact_io_aware_46_b200 as attn

    g = torch.Generator().manual_seed(7)
    Hkv, d, page, nb = 2, 64, 16, 2
    K, V = (torch.randn(1, Hkv, d, generator=g).to(BF).cuda() for _ in "KV")
    table = torch.arange((B + 1) * nb, dtype=I32, device="cuda").view(B + 1, nb)
    cu = torch.ones(B + 2, dtype=I32)
    cu[0] = 0
    for bad in (-1, nb * page + 1, -2 ** 31, 2 ** 31 - 1, None, 0, nb * page):
        lens = torch.zeros(B + 1, dtype=I32)
        lens[0] = 5
        if bad is not None:
            lens[B] = bad
        kp = torch.zeros((B + 1) * nb, Hkv, page, d, dtype=BF, device="cuda")
        vp = torch.zeros_like(kp)
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        attn.attn_kv_append_paged(K, V, kp, vp, table, lens.cuda(), cu_seqlens=cu.cuda(),
                                  workspace=ws)
        want = (0, 0) if bad in (None, 0, nb * page) else (attn.ATTN_ERR_INVALID,
                                                            attn.ATTN_DEV_BAD_KLEN)
        assert attn.attn_read_device_status(ws) == want, bad
        assert torch.equal(kp[0, :, 4], K[0]) and torch.equal(vp[0, :, 4], V[0])
        assert int((kp != 0).any(-1).sum()) == Hkv and int((vp != 0).any(-1).sum()) == Hkv
