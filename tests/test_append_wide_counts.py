"""attn_kv_append_paged refuses counts that the library's 32-bit arguments would cut short (a block
table of 2^32 + 4 columns would be read as one of 4, and other sequences' pages written)."""

import pytest
import torch

import exact_io_aware_46_b200 as attn
from tests.test_append_paged import FakeTokens
from tests.test_binding_validation import FakeCuda, rejects

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.mark.parametrize("extra", [-2 ** 31, 0, 4])
def test_counts_past_32_bits_are_refused(extra):
    n, B, Hkv, d = 2 ** 32 + extra, 2, 2, 128
    kv, pages = FakeTokens((6, Hkv, d)), FakeCuda((9, Hkv, 16, d), BF)
    table, lens, cu = FakeCuda((B, 4), I32), FakeCuda((B,), I32), FakeCuda((B + 1,), I32)
    c = FakeCuda((n, 64), F32)
    call = attn.attn_kv_append_paged
    rejects(lambda: call(kv, kv, pages, pages, FakeCuda((B, n), I32), lens, cu_seqlens=cu),
            "blocks", "limit")
    rejects(lambda: call(kv, kv, pages, pages, FakeCuda((n, 4), I32), FakeCuda((n,), I32),
                         cu_seqlens=FakeCuda((n + 1,), I32)), "sequences", "limit")
    rejects(lambda: call(kv, kv, pages, pages, table, lens, cu_seqlens=cu, cos=c, sin=c),
            "positions", "limit")
