"""The compiled part of the Python binding: it takes sound calls, gives what the Python code gives
for them, and leaves everything else to that code and its messages."""

import pytest
import torch

import exact_io_aware_46_b200 as attn

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def test_it_is_built_and_leaves_host_tensors_to_python():
    b = attn._binding
    assert b is not None
    t, f = torch.zeros((1, 2, 8, 64), dtype=BF), torch.zeros(2)
    attn.lib()
    assert b.fwd_diff(t, t, t, f, None, False, None, None, None, None, None, True) is None
    assert b.fwd_diff(*[None] * 12) is None and b.fwd_diff() is None
    assert b.bwd_diff(*[None] * 16) is None and b.bwd_diff(t) is None
    assert b.decode_diff(*[None] * 11) is None and b.append(*[None] * 14) is None
    for call in (lambda: attn.attn_fwd_diff(t, t, t, f),
                 lambda: attn.attn_bwd_diff(t, t, t, f, t, t, t, f),
                 lambda: attn.attn_fwd_splitkv_decode_diff(t, t, t, f, f),
                 lambda: attn.attn_kv_append_paged(t, t, t, t, f, f)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    with pytest.raises(TypeError):
        b.bind(1, 2)
    with pytest.raises(ValueError):
        b.bind(*[0] * len(attn._BOUND))
    attn._binding.bind(*(attn.ctypes.cast(getattr(attn.lib(), n), attn.ctypes.c_void_p).value
                         for n in attn._BOUND))


class Taken:
    """_binding, noting for each call whether it took it."""

    def __init__(self, real):
        self.real, self.took = real, []

    def __getattr__(self, name):
        fn = getattr(self.real, name)

        def call(*a):
            r = fn(*a)
            self.took.append(r is not None)
            return r

        return call


def _calls(dev):
    """(name, call, is it the common form): every entry point with tensors of all sorts."""
    g = torch.Generator(device=dev).manual_seed(5)
    rn = lambda *s: torch.randn(*s, generator=g, device=dev).to(BF)
    B, Hq, Hkv, L, d = 2, 4, 2, 70, 64
    q, k, v, go, lam = rn(B, Hq, L, d), rn(B, Hkv, L, d), rn(B, Hkv, L, d), rn(B, Hq, L, d), \
        torch.rand(Hq, generator=g, device=dev)
    kl = torch.tensor([L, 33], dtype=I32, device=dev)
    O, O2, lse = attn.attn_fwd_diff(q, k, v, lam, causal=True)
    new = lambda n: torch.zeros(n, dtype=torch.uint8, device=dev)
    fw = attn.attn_fwd_diff_workspace_size(B, Hq, Hkv, L, L, d)
    bw = attn.attn_bwd_diff_workspace_size(B, Hq, Hkv, L, L, d)
    one = rn(B, Hq, 1, d)
    pages = lambda: (k.view(B * Hkv, 1, L, d)[:, :, :64].reshape(B * 2, Hkv, 32, d).clone(),
                     v.view(B * Hkv, 1, L, d)[:, :, :64].reshape(B * 2, Hkv, 32, d).clone())
    kp, vp = pages()
    table = torch.tensor([[2, 0], [1, 3]], dtype=I32, device=dev)
    lens = torch.tensor([50, 17], dtype=I32, device=dev)
    cos, sin = torch.rand(64, 16, generator=g, device=dev), torch.rand(64, 16, generator=g, device=dev)
    fused = rn(B, Hq + 2 * Hkv, d)
    tq, tk, tv = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    cu = torch.tensor([0, 1, 2], dtype=I32, device=dev)
    class Sub(torch.Tensor):
        pass

    def app(**kw):
        a, b = pages()
        r = attn.attn_kv_append_paged(tk, tv, a, b, table, lens, **kw)
        return (r, a, b)

    par = torch.nn.Parameter(q.clone())
    yield "plain", lambda: attn.attn_fwd_diff(q, k, v, lam), True
    yield "masks", lambda: attn.attn_fwd_diff(q, k, v, lam[:1], 0.3, True, kl), True
    yield "no aux", lambda: attn.attn_fwd_diff(q, k, v, lam, want_aux=False), True
    yield "lse alone", lambda: attn.attn_fwd_diff(q, k, v, lam, lse=torch.empty_like(lse),
                                                  want_aux=False), True
    yield "outputs", lambda: attn.attn_fwd_diff(q, k, v, lam, O=torch.empty_like(q),
                                                O2=torch.empty_like(q), workspace=new(fw)), True
    yield "parameter", lambda: attn.attn_fwd_diff(par, k, v, lam), True
    yield "whole-number scale", lambda: attn.attn_fwd_diff(q, k, v, lam, scale=1), False
    yield "subclass", lambda: attn.attn_fwd_diff(q.as_subclass(Sub), k, v, lam), False
    yield "stream", lambda: attn.attn_fwd_diff(q, k, v, lam,
                                               stream=torch.cuda.current_stream()), False
    yield "empty", lambda: attn.attn_fwd_diff(q[:, :, :0], k, v, lam), True
    yield "bwd", lambda: attn.attn_bwd_diff(q, k, v, lam, O, O2, go, lse, causal=True), True
    yield "bwd outputs", lambda: attn.attn_bwd_diff(
        q, k, v, lam, O, O2, go, lse, causal=True, k_lens=None, dQ=torch.empty_like(q),
        dK=torch.empty_like(k), dV=torch.empty_like(k), dlam=lam.to(BF), workspace=new(bw)), True
    yield "decode", lambda: attn.attn_fwd_splitkv_decode_diff(one, k, v, lam, kl), True
    yield "decode, O alone", lambda: attn.attn_fwd_splitkv_decode_diff(
        one, k, v, lam, kl, O=torch.empty_like(one), want_lse=False), True
    yield "pages", lambda: attn.attn_fwd_splitkv_decode_diff_paged(one, kp, vp, table, lam, lens), True
    yield "append", lambda: app(), True
    yield "append all", lambda: app(cu_seqlens=cu, Q=tq, cos=cos, sin=sin, maps=2,
                                    interleaved=True, workspace=new(256)), True
    yield "append in place", lambda: app(Q=tq.contiguous(), Q_out=torch.empty(B, Hq, d, dtype=BF,
                                                                              device=dev)), True


@pytest.mark.gpu
def test_both_forms_give_the_same(monkeypatch):
    real = attn._binding
    attn.lib()
    for name, call, common in _calls("cuda"):
        seen = Taken(real)
        monkeypatch.setattr(attn, "_binding", seen)
        got = call()
        assert any(seen.took) == common, name
        monkeypatch.setattr(attn, "_binding", None)
        want = call()
        monkeypatch.setattr(attn, "_binding", real)
        assert type(got) is type(want) and len(got) == len(want), name
        for i, (a, b) in enumerate(zip(got, want)):
            if a is None or b is None:
                assert a is b, name
                continue
            assert a.shape == b.shape and a.dtype is b.dtype, name
            assert a.is_contiguous() and b.is_contiguous(), name
            assert not a.requires_grad, name
            if name.startswith("bwd") and i == 0:  # dQ's additions come in no fixed order
                assert (a.float() - b.float()).norm() <= 2e-3 * b.float().norm(), name
            else:
                assert torch.equal(a, b), (name, i)


@pytest.mark.gpu
def test_outputs_that_were_passed_in_are_returned():
    g = torch.Generator(device="cuda").manual_seed(6)
    q = torch.randn(1, 2, 40, 128, generator=g, device="cuda").to(BF)
    lam = torch.rand(2, generator=g, device="cuda")
    O, O2, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(1, 2, 2, 40, device="cuda")
    r = attn.attn_fwd_diff(q, q, q, lam, O=O, O2=O2, lse=lse)
    assert r[0] is O and r[1] is O2 and r[2] is lse
    outs = [torch.empty_like(q) for _ in range(3)] + [torch.empty(2, device="cuda", dtype=BF)]
    r = attn.attn_bwd_diff(q, q, q, lam, O, O2, q, lse, dQ=outs[0], dK=outs[1], dV=outs[2],
                           dlam=outs[3])
    assert all(a is b for a, b in zip(r, outs))
    kl = torch.tensor([40], dtype=I32, device="cuda")
    one, l1 = q[:, :, :1].contiguous(), torch.empty(1, 2, 2, device="cuda")
    o1 = torch.empty_like(one)
    r = attn.attn_fwd_splitkv_decode_diff(one, q, q, lam, kl, O=o1, lse=l1)
    assert r[0] is o1 and r[1] is l1


@pytest.mark.gpu
def test_unsound_calls_raise_as_before():
    dev = "cuda"
    q = torch.zeros(2, 4, 8, 64, dtype=BF, device=dev)
    k = torch.zeros(2, 2, 8, 64, dtype=BF, device=dev)
    lam, lse = torch.zeros(4, device=dev), torch.zeros(2, 4, 2, 8, device=dev)
    kl = torch.tensor([8, 8], dtype=I32, device=dev)
    for bad in (lambda: attn.attn_fwd_diff(q, k, k[:, :, :4], lam),
                lambda: attn.attn_fwd_diff(q, k, k, lam[:3]),
                lambda: attn.attn_fwd_diff(q, k, k, lam.cpu()),
                lambda: attn.attn_fwd_diff(q, k, k, lam, k_lens=kl.long()),
                lambda: attn.attn_fwd_diff(q.transpose(1, 2), k, k, lam),
                lambda: attn.attn_fwd_diff(q.float(), k, k, lam),
                lambda: attn.attn_fwd_diff(q, k, k, lam, O=q[:1]),
                lambda: attn.attn_fwd_diff(q, k, k, lam, workspace=torch.zeros(8, device=dev)),
                lambda: attn.attn_bwd_diff(q, k, k, lam, q, q, q, lse[:, :, :1]),
                lambda: attn.attn_bwd_diff(q, k, k, lam, q, q, q, lse, dK=q),
                lambda: attn.attn_fwd_splitkv_decode_diff(q, k, k, lam, kl),
                lambda: attn.attn_fwd_splitkv_decode_diff(q[:, :, :1].contiguous(), k, k, lam, kl[:1]),
                lambda: attn.attn_kv_append_paged(k, k, k, k, kl, kl)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(attn.AttnError):  # a status of the library itself: scale
        attn.attn_fwd_diff(q, k, k, lam, scale=-1.0)
    small = torch.zeros(16, dtype=torch.uint8, device=dev)
    with pytest.raises(ValueError, match="workspace"):
        attn.attn_bwd_diff(q, k, k, lam, q, q, q, lse, workspace=small)
    d96 = torch.zeros(1, 1, 8, 96, dtype=BF, device=dev)
    with pytest.raises(attn.AttnError):
        attn.attn_fwd_diff(d96, d96, d96, lam[:1])


@pytest.mark.gpu
def test_threads_call_at_once():
    """Four host threads, each on a stream of its own: what one call alone gives."""
    import threading

    g = torch.Generator(device="cuda").manual_seed(8)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)
    q, k, v = rn(2, 4, 300, 64), rn(2, 2, 300, 64), rn(2, 2, 300, 64)
    lam, kl = torch.rand(4, generator=g, device="cuda"), torch.tensor([300, 9], dtype=I32, device="cuda")
    one = q[:, :, :1].contiguous()

    def work():
        return attn.attn_fwd_diff(q, k, v, lam, causal=True) + \
            attn.attn_fwd_splitkv_decode_diff(one, k, v, lam, kl)

    want, got = work(), [None] * 4
    torch.cuda.synchronize()

    def run(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            got[i] = [work() for _ in range(25)][-1]
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for r in got:
        assert r is not None and all(torch.equal(a, b) for a, b in zip(r, want))
