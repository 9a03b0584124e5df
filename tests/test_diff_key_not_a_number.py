"""attn_fwd_diff, and its decode, with one element of K that is not a number, or infinite, at every
key index modulo eight: the exponentials of some columns are polynomials, and a score that is not
a number must not become a small weight there.

What the definition gives: a NaN score makes its row's softmax NaN, and so does a score of +inf
(inf - inf); a score of -inf is a key without weight.  Rows that do not see the key keep their
bounds."""

import math

import pytest
import torch

from tests import _diff_ref as ref
from tests.test_diff_fwd import problem

pytestmark = pytest.mark.gpu
I32 = torch.int32


def _lib():
    import exact_io_aware_46_b200 as attn

    return attn


def _check(o, o2, l, hit, m, refs):
    O, O2, lse, tol, tol2 = refs
    assert o[hit].isnan().all(), "O"
    assert l[hit][..., m].isnan().all(), "LSE"
    ref.assert_within(o[~hit], O[~hit], tol[~hit], "O elsewhere")
    ref.assert_lse(l[~hit], lse[~hit], "LSE elsewhere")
    ref.assert_lse(l[hit][..., 1 - m], lse[hit][..., 1 - m], "LSE of the other map")
    if m:
        assert o2[hit].isnan().all(), "O2"
    keep = ~hit if m else torch.ones_like(hit)
    ref.assert_within(o2[keep], O2[keep], tol2[keep], "O2 elsewhere")


@pytest.mark.parametrize("m", [0, 1])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_a_key_that_is_not_a_number_reaches_the_rows_that_see_it(value, d, m):
    attn = _lib()
    L, causal, at = 200, True, m * d // 2 + 5
    for j in [*range(8, 16), 70, 191]:
        Q, K, V, _, lam = problem(1, 2, 1, L, L, d, 300 + j)
        K[0, 0, j, at] = value
        hit = (torch.arange(L) >= j).expand(1, 2, L)
        if value == math.inf:
            hit = hit & (Q[..., at] > 0)
        lse_rows = lambda x: x.cpu().transpose(2, 3)  # [B, H, L, 2]
        O, O2, lse, tol, tol2 = ref.fwd(Q, K, V, lam, causal=causal)
        o, o2, l = attn.attn_fwd_diff(Q.cuda(), K.cuda(), V.cuda(), lam.cuda(), causal=causal)
        _check(o.cpu(), o2.cpu(), lse_rows(l), hit, m, (O, O2, lse_rows(lse), tol, tol2))


@pytest.mark.parametrize("m", [0, 1])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_the_decode_gives_not_a_number_too(value, d, m):
    """A map's scores are products with whole rows of K, zeros standing for the other half: an
    element that is not finite is NaN in O, and in the other map, of the heads that read its row."""
    attn = _lib()
    L, at = 700, m * d // 2 + 3
    for j in [*range(128, 136), 699]:
        Q, K, V, _, lam = problem(2, 4, 2, 1, L, d, 400 + j)
        O, _, lse, tol, _ = ref.fwd(Q, K, V, lam)
        K[1, 1, j, at] = value
        hit = torch.zeros(2, 4, dtype=torch.bool)
        hit[1, 2:] = True  # the group's heads
        o, l = attn.attn_fwd_splitkv_decode_diff(Q.cuda(), K.cuda(), V.cuda(), lam.cuda(),
                                                 torch.tensor([L, L], dtype=I32, device="cuda"))
        o, l = o.cpu(), l.cpu()
        assert o[hit].isnan().all() and l[hit][:, 1 - m].isnan().all()
        own = l[hit][:, m]  # an infinite key against its own map: by the sign of the score
        plus = torch.ones(2, dtype=torch.bool) if value != math.inf else Q[1, 2:, 0, at] > 0
        assert own[plus].isnan().all() and own[~plus].isfinite().all()
        ref.assert_within(o[~hit], O[~hit], tol[~hit], "O elsewhere")
        ref.assert_lse(l[~hit], lse[..., 0][~hit], "LSE elsewhere")
