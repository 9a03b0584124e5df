"""The compiled checks of the differential calls and the append accept no call that the Python
checks refuse: every argument of a sound call is changed in turn, and whatever the extension takes,
the Python code has to take as well.  Both hand their calls to functions that launch nothing, so
a difference shows here and not as an access out of range."""

import ctypes

import pytest
import torch

import exact_io_aware_46_b200 as attn

pytestmark = pytest.mark.gpu
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


class Still:
    """The library with the calls that launch replaced by ones that answer ATTN_OK."""

    QUERIES = [n for n in attn._BOUND if n.endswith("_size") or n == "attn_num_sms"]

    def __init__(self):
        real = attn.lib()
        self.kept = []
        for name in attn._BOUND:
            fn = getattr(real, name)
            if name not in self.QUERIES:
                res, args = attn.SIGNATURES[name]
                # (the workspace's size, its last argument but one, is the library's own check)
                fn = ctypes.CFUNCTYPE(res, *args)(
                    lambda *a: attn.ATTN_ERR_INVALID if len(a) > 2 and a[-2] < 256 else 0)
            self.kept.append(fn)
            setattr(self, name, fn)

    def addresses(self):
        return [ctypes.cast(f, ctypes.c_void_p).value for f in self.kept]


@pytest.fixture
def still(monkeypatch):
    s, real, binding = Still(), attn.lib(), attn._binding
    monkeypatch.setattr(attn, "lib", lambda: s)
    binding.bind(*s.addresses())
    yield s
    binding.bind(*(ctypes.cast(getattr(real, n), ctypes.c_void_p).value
                         for n in attn._BOUND))


def _sound():
    new = lambda shape, t: torch.zeros(shape, dtype=t, device="cuda")
    B, Hq, Hkv, L, d, T, page = 2, 4, 2, 24, 64, 5, 16
    q, kv, one = new((B, Hq, L, d), BF), new((B, Hkv, L, d), BF), new((B, Hq, 1, d), BF)
    lam, kl, lse = new((Hq,), F32), new((B,), I32), new((B, Hq, 2, L), F32)
    pages, table = new((6, Hkv, page, d), BF), new((B, 3), I32)
    ws = new((1 << 22,), U8)
    yield attn.attn_fwd_diff, dict(Q=q, K=kv, V=kv, lam=lam, scale=0.1, causal=True, k_lens=kl, O=q,
                                   O2=q, lse=lse, workspace=ws)
    yield attn.attn_bwd_diff, dict(Q=q, K=kv, V=kv, lam=lam, O=q, O2=q, dO=q, lse=lse, scale=0.1,
                                   causal=False, k_lens=kl, dQ=q, dK=kv, dV=kv, dlam=new((Hq,), BF),
                                   workspace=ws)
    l1 = new((B, Hq, 2), F32)
    yield attn.attn_fwd_splitkv_decode_diff, dict(Q=one, Kc=kv, Vc=kv, lam=lam, k_lens=kl,
                                                  scale=0.1, O=one, lse=l1, workspace=ws)
    yield attn.attn_fwd_splitkv_decode_diff_paged, dict(Q=one, Kp=pages, Vp=pages,
                                                        block_table=table, lam=lam, k_lens=kl,
                                                        scale=0.1, O=one, lse=l1, workspace=ws)
    c = new((40, 8), F32)
    fused = new((T, Hq + 2 * Hkv, d), BF)
    yield attn.attn_kv_append_paged, dict(
        K=fused[:, Hq:Hq + Hkv], V=fused[:, Hq + Hkv:], Kp=pages, Vp=pages, block_table=table,
        k_lens=kl, cu_seqlens=new((B + 1,), I32), Q=fused[:, :Hq], Q_out=new((T, Hq, d), BF), cos=c,
        sin=c, maps=2, interleaved=True, workspace=ws)


def _changed(x):
    """Other things to pass in the place of x."""
    yield None
    if not isinstance(x, torch.Tensor):
        yield from (0, 1, 2, 3, -1, 2 ** 40, 0.5, -0.5, "x", True)
        return
    yield x.cpu()
    yield 1.0
    for t in (BF, F32, torch.float16, I32, torch.int64, U8):
        if t != x.dtype:
            yield torch.zeros(x.shape, dtype=t, device="cuda")
    same = lambda shape: torch.zeros(shape, dtype=x.dtype, device="cuda")
    for i, n in enumerate(x.shape):
        for m in {0, 1, n - 1, n + 1, 2 * n, 3}:
            yield same((*x.shape[:i], m, *x.shape[i + 1:]))
        yield x.narrow(i, 0, max(n - 1, 0))
    yield same((*x.shape, 1))
    yield same((1, *x.shape))
    yield x[0]
    if x.dim() > 1:
        yield x.transpose(0, 1)
        yield x.transpose(-1, -2)
        yield x[:1].expand(x.shape)
        yield same((*x.shape[:-1], 2 * x.shape[-1]))[..., ::2]


def _outcome(call, kw):
    try:
        call(**kw)
        return None
    except Exception as e:  # noqa: BLE001
        return e


def test_what_the_extension_takes_python_takes(still, monkeypatch):
    real, took = attn._binding, 0

    class Seen:
        def __getattr__(self, name):
            def call(*a):
                r = getattr(real, name)(*a)
                self.__dict__["took"] = r is not None
                return r

            return call

    for call, kw in _sound():
        changes = [kw] + [{**kw, n: y} for n, x in kw.items() for y in _changed(x)]
        # two at once, where one shape has to follow another
        for a, b in (("K", "V"), ("Kp", "Vp"), ("Kc", "Vc"), ("cos", "sin"), ("O", "O2")):
            if a in kw and b in kw:
                changes += [{**kw, a: y, b: y} for y in _changed(kw[a])]
        first = True
        for c in changes:
            seen = Seen()
            monkeypatch.setattr(attn, "_binding", seen)
            _outcome(call, c)
            if seen.__dict__.get("took"):
                took += 1
                monkeypatch.setattr(attn, "_binding", None)
                e = _outcome(call, c)
                assert e is None, (call.__name__, e, [n for n in c if c[n] is not kw[n]])
            else:
                assert not first, call.__name__  # the sound call itself is taken
            first = False
    monkeypatch.setattr(attn, "_binding", real)
    assert took > 20
