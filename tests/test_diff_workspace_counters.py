"""A forward of few query tiles on a workspace that was never cleared leaves its counters sound: a
later forward of many tiles on the same workspace does all of its tiles."""

import pytest
import torch

from tests.test_diff_fwd import problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fill", [0x01, 0x7F, 0xFF])
def test_a_small_forward_leaves_the_counters_at_zero(fill):
    import exact_io_aware_46_b200 as attn

    small = [t.cuda() for t in problem(1, 2, 2, 130, 130, 64, 3)]
    large = [t.cuda() for t in problem(3, 100, 100, 40, 40, 64, 4)]
    Q, K, V, _, lam = large
    assert Q.shape[0] * Q.shape[1] > attn.attn_num_sms()
    want = attn.attn_fwd_diff(Q, K, V, lam, causal=True)
    ws = torch.full((256,), fill, dtype=torch.uint8, device="cuda")
    status = ws.view(torch.int32)[0].item()
    for _ in range(2):
        attn.attn_fwd_diff(*small[:3], small[4], workspace=ws)
        assert ws.view(torch.int32)[0].item() == status  # the status word is the caller's
        assert (ws.view(torch.int32)[1:3] == 0).all()
    for _ in range(2):
        outs = [torch.zeros_like(Q), torch.zeros_like(Q), torch.zeros_like(want[2])]
        got = attn.attn_fwd_diff(Q, K, V, lam, causal=True, O=outs[0], O2=outs[1], lse=outs[2],
                                 workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
