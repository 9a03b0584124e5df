"""attn_kv_append_paged against the rotation in 64 bits: which rows are written, what they
hold, and that everything else in the cache and in Q_out stays as it was."""

import pytest
import torch

from tests._diff_ref import assert_within, rotate, rotation_bound
from tests.test_binding_validation import FakeCuda, rejects

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _lib():
    import exact_io_aware_46_b200 as attn

    return attn


def _tables(n_pos, half, seed=5):
    """Angles of ordinary frequencies; the kernel takes any table."""
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))
    ang = torch.arange(n_pos, dtype=torch.float64)[:, None] * freq + 0.1 * seed
    return ang.cos().float(), ang.sin().float()


def _problem(n_new, past, Hq, Hkv, d, page, seed, pad=0, spare=2):
    """Packed tokens, a cache full of numbers, and a block table over pages in random order."""
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g).to(BF)
    B, T = len(n_new), sum(n_new) + pad
    nb = max(1, max((a + b + page - 1) // page for a, b in zip(n_new, past)))
    table = torch.randperm(B * nb + spare, generator=g)[:B * nb].view(B, nb).to(I32)
    cu = torch.tensor([0] + torch.tensor(n_new).cumsum(0).tolist(), dtype=I32)
    lens = torch.tensor([a + b for a, b in zip(n_new, past)], dtype=I32)
    return dict(Q=rn(T, Hq, d), K=rn(T, Hkv, d), V=rn(T, Hkv, d),
                Kp=rn(B * nb + spare, Hkv, page, d), Vp=rn(B * nb + spare, Hkv, page, d),
                table=table, cu=cu, lens=lens)


def _expect(x, n_new, past, cos, sin, maps, inter, page, skip=()):
    """References (64 bits), bounds, and the mask of what may change, for Q_out, Kp and Vp."""
    half = cos.shape[1]
    kref, vref = x["Kp"].double(), x["Vp"].double()
    kb, vb = torch.zeros_like(kref), torch.zeros_like(vref)
    qref, qb = torch.full_like(x["Q"].double(), 7.0), torch.zeros_like(x["Q"].double())
    t = 0
    for b, n in enumerate(n_new):
        for i in range(n):
            row = past[b] + i
            if b not in skip:
                pg, at = int(x["table"][b, row // page]), row % page
                c, s = cos[row:row + 1], sin[row:row + 1]
                for src, ref, bnd, idx in ((x["Q"], qref, qb, t), (x["K"], kref, kb, (pg, slice(None), at))):
                    y = rotate(src[t:t + 1], c, s, maps, inter)
                    ref[idx] = y[0]
                    bnd[idx] = rotation_bound(src[t:t + 1], y, maps, half, inter)[0]
                vref[pg, :, at] = x["V"][t].double()
            t += 1
    return (qref, qb), (kref, kb), (vref, vb)


def _run(x, cos, sin, maps, inter, cu=True, q=True, **kw):
    attn = _lib()
    c = {k: v.cuda() for k, v in x.items()}
    q_out = torch.full_like(c["Q"], 7.0) if q else None
    out = attn.attn_kv_append_paged(
        kw.pop("K", c["K"]), kw.pop("V", c["V"]), c["Kp"], c["Vp"], c["table"], c["lens"],
        cu_seqlens=c["cu"] if cu else None, Q=kw.pop("Q", c["Q"]) if q else None, Q_out=q_out,
        cos=cos.cuda() if cos.shape[1] else None, sin=sin.cuda() if cos.shape[1] else None,
        maps=maps, interleaved=inter, **kw)
    torch.cuda.synchronize()
    assert out is q_out
    return out, c["Kp"], c["Vp"]


CASES = [
    # new tokens, earlier rows, Hq, Hkv, d, page, rope_dim, maps, interleaved, pad
    ([1], [0], 1, 1, 128, 16, 128, 1, False, 0),            # the first token of all
    ([1], [130], 32, 8, 128, 64, 128, 1, False, 0),
    ([1, 1, 1], [15, 16, 17], 4, 2, 64, 16, 64, 1, True, 0),  # around a page's end
    ([3, 0, 33, 1], [0, 9, 30, 63], 8, 2, 128, 32, 64, 2, False, 4),  # an idle sequence, padding
    ([40, 7], [5, 250], 6, 2, 128, 256, 32, 2, True, 0),     # partly rotated halves, odd group
    ([129, 1, 64], [0, 0, 64], 4, 4, 64, 64, 32, 2, False, 1),
    ([70], [3], 2, 2, 64, 16, 16, 1, True, 0),
    ([12, 5], [60, 1], 4, 1, 128, 64, 0, 1, False, 0),       # no rotation
    ([2] * 70, [1] * 70, 2, 1, 64, 16, 48, 1, False, 3),     # more than 32 and 64 sequences
]


@pytest.mark.gpu
@pytest.mark.parametrize("n_new,past,Hq,Hkv,d,page,rope,maps,inter,pad", CASES)
def test_append_matches_rotation(n_new, past, Hq, Hkv, d, page, rope, maps, inter, pad):
    x = _problem(n_new, past, Hq, Hkv, d, page, 11 + sum(n_new) + page, pad)
    cos, sin = _tables(max(a + b for a, b in zip(n_new, past)), rope // 2)
    got = _run(x, cos, sin, maps, inter)
    for g, (ref, bound), what in zip(got, _expect(x, n_new, past, cos, sin, maps, inter, page),
                                     ("Q_out", "Kpages", "Vpages")):
        assert_within(g, ref, bound, what)
    # one token per sequence: the same without offsets
    if set(n_new) == {1} and not pad:
        for a, b in zip(got, _run(x, cos, sin, maps, inter, cu=False)):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_append_views_of_a_fused_projection_in_place_and_without_q():
    Hq, Hkv, d = 4, 2, 128
    n_new, past = [9, 30], [4, 40]
    x = _problem(n_new, past, Hq, Hkv, d, 32, 77)
    cos, sin = _tables(80, 64)
    want = _run(x, cos, sin, 1, False)
    qkv = torch.cat([x[n].flatten(1) for n in "QKV"], 1).cuda()
    views = {n: qkv[:, a * d:(a + h) * d].unflatten(1, (h, d))
             for n, a, h in (("Q", 0, Hq), ("K", Hq, Hkv), ("V", Hq + Hkv, Hkv))}
    for a, b in zip(_run(x, cos, sin, 1, False, **views), want):
        assert torch.equal(a, b)
    _, kp, vp = _run(x, cos, sin, 1, False, q=False)
    assert torch.equal(kp, want[1]) and torch.equal(vp, want[2])
    # Q rotated in place
    attn = _lib()
    c = {k: v.cuda() for k, v in x.items()}
    attn.attn_kv_append_paged(c["K"], c["V"], c["Kp"], c["Vp"], c["table"], c["lens"],
                              cu_seqlens=c["cu"], Q=c["Q"], Q_out=c["Q"], cos=cos.cuda(),
                              sin=sin.cuda())
    assert torch.equal(c["Q"], want[0]) and torch.equal(c["Kp"], want[1])


@pytest.mark.gpu
def test_append_device_errors_write_nothing():
    attn = _lib()
    n_new, past, page = [3, 4, 2], [10, 0, 20], 16
    cos, sin = _tables(64, 64)

    def check(change, bit, skip, n_pos=64, tokens=None):
        x = _problem(n_new, past, 2, 1, 128, page, 91)
        x["table"] = torch.cat([x["table"], x["table"]], 1).contiguous()  # room of 4 pages
        change(x)
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        got = _run(x, cos[:n_pos], sin[:n_pos], 1, False, workspace=ws)
        code, bits = attn.attn_read_device_status(ws)
        assert code == attn.ATTN_ERR_INVALID and bits == bit
        for g, (ref, bound), what in zip(got, _expect(x, n_new, past, cos, sin, 1, False, page,
                                                      skip), ("Q_out", "Kpages", "Vpages")):
            assert_within(g, ref, bound, what)

    bad_len, bad_page = attn.ATTN_DEV_BAD_KLEN, attn.ATTN_DEV_BAD_PAGE
    check(lambda x: x["lens"].__setitem__(1, 3), bad_len, (1,))      # fewer rows than new tokens
    check(lambda x: x["lens"].__setitem__(1, -1), bad_len, (1,))
    check(lambda x: x["lens"].__setitem__(1, 65), bad_len, (1,))     # past the block table
    check(lambda x: x["table"].__setitem__((0, 0), -1), bad_page, (0,))
    check(lambda x: x["table"].__setitem__((2, 1), 10 ** 6), bad_page, (2,))
    check(lambda x: None, bad_len, (2,), n_pos=20)                   # past the rotation's table
    check(lambda x: x["cu"].__setitem__(3, 10), bad_len, (2,))       # past the tokens


@pytest.mark.gpu
def test_append_replayed_from_a_graph_and_on_another_stream():
    attn = _lib()
    n_new, past = [1, 1, 1, 1], [30, 2, 15, 46]  # three pages: room for one more step
    x = _problem(n_new, past, 8, 2, 128, 16, 5)
    cos, sin = _tables(128, 32)
    c = {k: v.cuda() for k, v in x.items()}
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    q_out = torch.zeros_like(c["Q"])
    args = dict(Q=c["Q"], Q_out=q_out, cos=cos.cuda(), sin=sin.cuda(), maps=2, workspace=ws)
    call = lambda **kw: attn.attn_kv_append_paged(c["K"], c["V"], c["Kp"], c["Vp"], c["table"],
                                                  c["lens"], **args, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    # two replays: the second on other tokens and one row further
    for step in range(2):
        if step:
            for n in "QKV":
                c[n].copy_(torch.randn_like(c[n].float()).to(BF))
            c["lens"] += 1
            past = [p + 1 for p in past]
        kp, vp = c["Kp"].cpu(), c["Vp"].cpu()
        graph.replay()
        torch.cuda.synchronize()
        y = {n: c[n].cpu() for n in "QKV"} | {"Kp": kp, "Vp": vp, "table": x["table"]}
        for g, (ref, bound), what in zip((q_out, c["Kp"], c["Vp"]),
                                         _expect(y, n_new, past, cos, sin, 2, False, 16),
                                         ("Q_out", "Kpages", "Vpages")):
            assert_within(g, ref, bound, what)


def test_append_rejections():
    attn = _lib()
    T, Hq, Hkv, d, B = 6, 4, 2, 128, 2
    kv, q = FakeTokens((T, Hkv, d)), FakeTokens((T, Hq, d))
    pages, tab = FakeCuda((9, Hkv, 16, d), BF), FakeCuda((B, 4), I32)
    lens, cu = FakeCuda((B,), I32), FakeCuda((B + 1,), I32)
    c = FakeCuda((64, 64), F32)

    def call(K=kv, V=kv, Kp=pages, Vp=pages, t=tab, l=lens, cu_=cu, **kw):
        return lambda: attn.attn_kv_append_paged(K, V, Kp, Vp, t, l, cu_seqlens=cu_, **kw)

    rejects(call(K=FakeTokens((T, 3, d))), "K", "shape")
    rejects(call(V=FakeTokens((T - 1, Hkv, d))), "V", "shape")
    rejects(call(K=FakeTokens((T, Hkv, d), stride=(Hkv * d + 4, d, 1))), "K", "strides")
    rejects(call(K=FakeTokens((T, Hkv, d), stride=(Hkv * d, 1, Hkv))), "K", "strides")
    rejects(call(K=FakeTokens((T, Hkv, d), stride=(0, d, 1))), "K", "strides")
    rejects(call(K=FakeTokens((T, Hkv, d), dtype=F32)), "K", "bfloat16")
    rejects(call(K=torch.zeros(T, Hkv, d, dtype=BF)), "K", "CUDA")
    rejects(call(V=FakeTokens((T, Hkv, d), device="cuda:1")), "V", "cuda:1")
    rejects(call(Vp=FakeCuda((9, Hkv, 32, d), BF)), "Vpages")
    rejects(call(t=FakeCuda((B + 1, 4), I32)), "block_table")
    rejects(call(l=FakeCuda((B,), torch.int64)), "k_lens")
    rejects(call(cu_=FakeCuda((B,), I32)), "cu_seqlens")
    rejects(call(cu_=None), "cu_seqlens")
    rejects(call(Q=FakeTokens((T, 3, d))), "multiple")
    rejects(call(Q=FakeTokens((T + 1, Hq, d))), "Q", "shape")
    rejects(call(Q_out=q), "Q_out")
    rejects(call(Q=q, Q_out=FakeCuda((T, Hq, 64), BF)), "Q_out")
    rejects(call(cos=c), "together")
    rejects(call(cos=c, sin=FakeCuda((64, 32), F32)), "sin")
    rejects(call(cos=FakeCuda((64, 64), torch.float64), sin=c), "cos")
    rejects(call(workspace=FakeCuda((128,), torch.uint8)), "workspace", "needs")


class FakeTokens(FakeCuda):
    """FakeCuda with strides."""

    def __init__(self, shape, dtype=BF, device="cuda:0", stride=None):
        super().__init__(shape, dtype, device, contiguous=stride is None)
        self._stride = stride

    def stride(self):
        return self._stride


def test_append_rejects_on_host():
    import ctypes

    attn = _lib()
    P = 256 * 1024

    def call(Q=P, Qo=P, K=P, ks=256, Kp=P, bt=P, mb=4, page=16, n_pages=9, cu=P, kl=P, B=2, T=6,
             Hq=4, Hkv=2, d=128, cos=P, n_pos=64, rope=128, maps=1, inter=0, ws=P, nb=256):
        p = lambda a: None if a is None else ctypes.c_void_p(a)
        return attn.lib().attn_kv_append_paged(p(Q), 512, p(K), ks, p(P), 256, p(Qo), p(Kp), p(P),
                                               p(bt), mb, page, n_pages, p(cu), p(kl), B, T, Hq,
                                               Hkv, d, p(cos), p(P), n_pos, rope, maps, inter,
                                               p(ws), nb, None)

    assert call(T=0) == 0 and call(T=0, K=None) == 0
    for bad in (dict(K=None), dict(Kp=None), dict(bt=None), dict(kl=None), dict(ws=None),
                dict(Qo=None), dict(Q=None), dict(cu=None), dict(B=0), dict(T=-1), dict(Hq=3),
                dict(ks=252), dict(ks=-256), dict(maps=3), dict(inter=2), dict(rope=-16),
                dict(cos=None), dict(n_pos=0), dict(n_pos=-1), dict(ws=P + 16), dict(nb=64),
                dict(K=P + 8), dict(cos=P + 4), dict(mb=0), dict(n_pages=0), dict(page=0)):
        assert call(**bad) == attn.ATTN_ERR_INVALID, bad
    for no in (dict(d=96), dict(page=24), dict(page=8), dict(rope=8), dict(rope=144),
               dict(rope=128, maps=2), dict(d=64, rope=128)):
        assert call(**no) == attn.ATTN_ERR_UNSUPPORTED, no
