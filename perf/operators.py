"""Measured cases of differential attention and of the paged cache's append.

Four operators, as a user's program calls them:

* ``append``  rotates the new tokens' Q and K by position and writes K and V into the paged cache;
* ``fwd``     differential attention O = (softmax(s q1 k1^T) - lam softmax(s q2 k2^T)) V, each head
              row holding the two maps' halves [x1 x2];
* ``bwd``     its gradients dQ, dK, dV and dlam;
* ``decode``  its form for one new token per sequence over a (paged) cache.

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits."""

import math
import random

import torch

own = False

BF = torch.bfloat16


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one conversation's next token: a launch and a few dependent loads
        dict(name="append_one_token", op="append", B=1, Hq=32, Hkv=8, d=128, n_lo=1, n_hi=1,
             past=2900, page=64, maps=1, rope=128, interleaved=False, fused=True, pad=0, lens=11),
        # a decode step of a serving batch, two maps a head (each half is rotated by itself)
        dict(name="append_batch_step", op="append", B=64, Hq=32, Hkv=8, d=128, n_lo=1, n_hi=1,
             past=4000, page=64, maps=2, rope=64, interleaved=False, fused=True, pad=0, lens=12),
        # packed prompts of uneven length out of one QKV projection, in a buffer padded for replay
        dict(name="append_prompts", op="append", B=16, Hq=16, Hkv=16, d=128, n_lo=256, n_hi=4096,
             past=0, page=64, maps=1, rope=64, interleaved=True, fused=True, pad=77, lens=13),
        # the smallest forward of the benchmark's workloads
        dict(name="fwd_tiny", op="fwd", B=1, Hq=2, Hkv=2, Lq=256, Lk=256, d=64, causal=False,
             k_lo=0, k_hi=0, lens=0),
        # the benchmark's prefill
        dict(name="fwd_prefill", op="fwd", B=4, Hq=16, Hkv=16, Lq=4096, Lk=4096, d=128,
             causal=True, k_lo=0, k_hi=0, lens=0),
        # a prompt's later part behind an earlier one, padded batch, grouped heads, odd sizes
        dict(name="fwd_chunk_padded", op="fwd", B=3, Hq=32, Hkv=8, Lq=1001, Lk=5003, d=128,
             causal=True, k_lo=4100, k_hi=5003, lens=21),
        dict(name="bwd_tiny", op="bwd", B=1, Hq=2, Hkv=2, Lq=256, Lk=256, d=64, causal=False,
             k_lo=0, k_hi=0, lens=0),
        # the benchmark's backward
        dict(name="bwd_train", op="bwd", B=2, Hq=16, Hkv=16, Lq=8192, Lk=8192, d=128, causal=True,
             k_lo=0, k_hi=0, lens=0),
        # narrow heads shared by groups, padded batch, odd length
        dict(name="bwd_grouped_padded", op="bwd", B=3, Hq=16, Hkv=4, Lq=1999, Lk=1999, d=64,
             causal=True, k_lo=1200, k_hi=1999, lens=31),
        # one conversation's next token over its cache
        dict(name="decode_one_seq", op="decode", B=1, Hq=32, Hkv=8, d=128, paged=True, page=64,
             Lmax=4096, k_lo=2901, k_hi=2901, lens=41),
        # the benchmark's decode: a full serving batch
        dict(name="decode_batch", op="decode", B=64, Hq=32, Hkv=8, d=128, paged=True, page=64,
             Lmax=32768, k_lo=1024, k_hi=32768, lens=42),
        # few sequences, narrow heads in groups of eight, uneven lengths, contiguous cache
        dict(name="decode_few_narrow", op="decode", B=7, Hq=16, Hkv=2, d=64, paged=False, page=0,
             Lmax=9001, k_lo=1, k_hi=9001, lens=43),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], uniform over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "fwd", "bwd", "decode"])
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 8] if op == "decode" else [1, 2, 3, 4])
    lens = rng.randrange(1 << 30)
    if op == "append":
        maps = rng.choice([1, 2])
        B = _log(rng, 1, 128)
        n_hi = 1 if rng.random() < 0.5 else _log(rng, 2, 2048)
        while B * n_hi > 32768:
            B = max(1, B // 2)
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, d=d, n_lo=1, n_hi=n_hi,
                    past=rng.choice([0, _log(rng, 1, 4000)]), page=rng.choice([16, 64, 256]),
                    maps=maps, rope=d // maps // rng.choice([1, 2]),
                    interleaved=rng.random() < 0.5, fused=rng.random() < 0.5,
                    pad=rng.choice([0, 5]), lens=lens)
    if op == "decode":
        B, Lmax = _log(rng, 1, 64), _log(rng, 64, 32768)
        while B * Lmax * Hkv * d > 64 * 8192 * 8 * 128:
            B = max(1, B // 2)
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, d=d, paged=rng.random() < 0.6,
                    page=rng.choice([16, 32, 64, 128, 256]), Lmax=Lmax, k_lo=1, k_hi=Lmax,
                    lens=lens)
    B = rng.choice([1, 1, 2, 3, 4])
    # gradients of a few keys are next to zero (of one key zero), and say nothing of the rest
    least = 16 if op == "bwd" else 1
    Lq = _log(rng, least, 4096)
    Lk = Lq if op == "bwd" or rng.random() < 0.6 else Lq + _log(rng, 1, 4096)
    while B * Hkv * G * Lq * Lk > 2 * 16 * 8192 * 8192 // 4:
        B, Lq, Lk = max(1, B // 2), max(least, Lq // 2), max(least, Lk // 2)
    pad = rng.random() < 0.4
    return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, Lq=Lq, Lk=Lk, d=d, causal=rng.random() < 0.7,
                k_lo=(Lk + 1) // 2 if pad else 0, k_hi=Lk if pad else 0, lens=lens)


def _ints(n, lo, hi, seed):
    r = random.Random(seed)
    return [r.randint(lo, hi) for _ in range(n)]


def _k_lens(c):
    """Visible keys of each sequence of a case."""
    if c["op"] == "decode" or c["k_hi"]:
        return _ints(c["B"], c["k_lo"], c["k_hi"], c["lens"])
    return [c["Lk"]] * c["B"]


def _append_sizes(c):
    """New tokens and earlier rows of each sequence."""
    n = _ints(c["B"], c["n_lo"], c["n_hi"], c["lens"])
    past = _ints(c["B"], c["past"] // 2, c["past"], c["lens"] + 1)
    return n, past


def _pairs(c):
    """Visible (query, key) pairs of one head, summed over the batch."""
    total = 0
    for kl in _k_lens(c):
        if not c["causal"]:
            total += c["Lq"] * kl
            continue
        off = c["Lk"] - c["Lq"]
        full = max(0, min(c["Lq"], c["Lq"] - (kl - off) + 1))  # rows that see all kl keys
        part = c["Lq"] - full
        total += full * kl + part * off + part * (part + 1) // 2
    return total


def work(case):
    c = case
    d, Hq, Hkv, B = c["d"], c["Hq"], c["Hkv"], c["B"]
    if c["op"] == "append":
        n, past = _append_sizes(c)
        T, rows = sum(n), max(a + b for a, b in zip(n, past))
        lo = min(past)
        return dict(bytes=2 * T * (Hq + 2 * Hkv) * d * 2 + min(T, rows - lo) * c["rope"] * 4,
                    flops=3 * T * (Hq + Hkv) * c["maps"] * c["rope"])
    if c["op"] == "decode":
        keys = sum(_k_lens(c))
        # K, V rows; Q in; O out, two LSE a head; scores of both maps and one weighted sum
        return dict(bytes=keys * Hkv * d * 4 + B * Hq * (d * 4 + 8), flops=keys * Hq * 4 * d)
    q, k = B * Hq * c["Lq"], Hkv * sum(_k_lens(c))
    if c["op"] == "fwd":
        # Q in, O and O2 out, two LSE a row; K and V in
        return dict(bytes=q * (6 * d + 8) + k * 4 * d, flops=4 * d * Hq * _pairs(c))
    # Q, O, O2, dO in, dQ out, two LSE a row; K, V in, dK, dV out
    return dict(bytes=q * (10 * d + 8) + k * 8 * d, flops=10 * d * Hq * _pairs(c))


# ------------------------------------------------------------------ inputs


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(BF)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _table(g, B, nb):
    """Block table [B, nb] of distinct pages in random order."""
    return torch.randperm(B * nb, generator=g, device="cuda").to(torch.int32).view(B, nb)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = dict(c)
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    if c["op"] == "append":
        n, past = _append_sizes(c)
        T = sum(n) + c["pad"]
        cols = (Hq + 2 * Hkv) * d
        if c["fused"]:  # views of one projection's output
            qkv = _randn(g, T, cols)
            st["Q"] = qkv[:, :Hq * d].view(T, Hq, d)
            st["K"] = qkv[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d)
            st["V"] = qkv[:, (Hq + Hkv) * d:].view(T, Hkv, d)
        else:
            st["Q"], st["K"], st["V"] = (_randn(g, T, h, d) for h in (Hq, Hkv, Hkv))
        rows = max(a + b for a, b in zip(n, past))
        nb = (rows + c["page"] - 1) // c["page"]
        st["table"] = _table(g, B, nb)
        st["Kp"] = _randn(g, B * nb, Hkv, c["page"], d)
        st["Vp"] = _randn(g, B * nb, Hkv, c["page"], d)
        st["n_tok"] = sum(n)
        cu = [0]
        for x in n:
            cu.append(cu[-1] + x)
        # a step of one token a sequence needs no offsets
        st["cu"] = None if c["n_hi"] == 1 and not c["pad"] else _i32(cu)
        st["k_lens"] = _i32([a + b for a, b in zip(n, past)])
        st["seq"] = torch.tensor([b for b in range(B) for _ in range(n[b])], device="cuda")
        st["row"] = torch.tensor([past[b] + i for b in range(B) for i in range(n[b])],
                                 device="cuda")
        half = c["rope"] // 2
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
        ang = torch.arange(rows, dtype=torch.float64)[:, None] * freq
        st["cos"], st["sin"] = ang.cos().float().cuda(), ang.sin().float().cuda()
        st["Q_out"] = torch.zeros(T, Hq, d, dtype=BF, device="cuda")
    elif c["op"] == "decode":
        kl = _k_lens(c)
        st["lens_host"] = kl
        st["k_lens"] = _i32(kl)
        st["Q"] = _randn(g, B, Hq, 1, d)
        st["lam"] = torch.rand(Hq, generator=g, device="cuda") * 0.8 + 0.1
        if c["paged"]:
            # pages are handed out as the sequences grow: only those that hold rows exist
            nb = (c["Lmax"] + c["page"] - 1) // c["page"]
            need = [(x + c["page"] - 1) // c["page"] for x in kl]
            order = torch.randperm(sum(need), generator=g, device="cuda").to(torch.int32)
            st["table"] = torch.zeros(B, nb, dtype=torch.int32, device="cuda")
            at = 0
            for b, x in enumerate(need):
                st["table"][b, :x] = order[at:at + x]
                at += x
            shape = (sum(need), Hkv, c["page"], d)
        else:
            shape = (B, Hkv, c["Lmax"], d)
        st["K"], st["V"] = _randn(g, *shape), _randn(g, *shape)
        st["O"] = torch.empty_like(st["Q"])
        st["lse"] = torch.empty(B, Hq, 2, device="cuda")
    else:
        Lq, Lk = c["Lq"], c["Lk"]
        st["Q"] = _randn(g, B, Hq, Lq, d)
        st["K"], st["V"] = _randn(g, B, Hkv, Lk, d), _randn(g, B, Hkv, Lk, d)
        st["lam"] = torch.rand(Hq, generator=g, device="cuda") * 0.8 + 0.1
        st["lens_host"] = _k_lens(c)
        st["k_lens"] = _i32(st["lens_host"]) if c["k_hi"] else None
        if c["op"] == "bwd":
            st["dO"] = _randn(g, B, Hq, Lq, d)
            # what the forward of the same step left behind
            st["O"], st["O2"], st["lse"] = _plain_fwd(st)
    return st


# ------------------------------------------------------------------ plain forms (32 bits)


def _mask(st):
    """Visible (query, key) pairs of each sequence, [B, 1, 1, Lq, Lk]."""
    Lq, Lk = st["Lq"], st["Lk"]
    i = torch.arange(Lq, device="cuda")[:, None]
    j = torch.arange(Lk, device="cuda")
    vis = (j <= i + (Lk - Lq) if st["causal"] else j >= 0).expand(1, 1, 1, Lq, Lk)
    if st["k_lens"] is not None:
        vis = vis & (j < st["k_lens"].view(-1, 1, 1, 1, 1))
    return vis


def _grouped(st, name):
    """A tensor [B, H, L, d] in 32 bits as [B, Hkv, heads of the group, L, d]."""
    x = st[name].float()
    return x.view(st["B"], st["Hkv"], -1, x.shape[2], st["d"])


def _half(x, m):
    """Map m's half of the head rows."""
    h = x.shape[-1] // 2
    return x[..., m * h:(m + 1) * h]


def _plain_map(q, k, m, vis):
    """One map's probabilities and the log-sum-exp of its rows."""
    s = _half(q, m) @ _half(k, m).transpose(-1, -2) / math.sqrt(q.shape[-1] // 2)
    s = torch.where(vis, s, -math.inf)
    mx = s.amax(-1, keepdim=True)
    mx = torch.where(mx == -math.inf, 0.0, mx)
    p = torch.exp(s - mx)
    l = p.sum(-1, keepdim=True)
    return p / torch.where(l > 0, l, 1.0), (mx + torch.log(l)).squeeze(-1)


def _plain_fwd(st):
    q, k, v = (_grouped(st, n) for n in "QKV")
    vis = _mask(st)
    lam = st["lam"].view(st["Hkv"], -1, 1, 1)
    p, l1 = _plain_map(q, k, 0, vis)
    o1 = p @ v
    p, l2 = _plain_map(q, k, 1, vis)
    o2 = p @ v
    lse = torch.stack([l1, l2], 3).view(st["B"], st["Hq"], 2, st["Lq"])
    return (o1 - lam * o2).view_as(st["Q"]).to(BF), o2.view_as(st["Q"]).to(BF), lse


def _plain_bwd_map(st, m, c, p, dp, q, k):
    """Gradients of one map's halves and rowsum(p dp); the map's weight in O is c."""
    D = (p * dp).sum(-1, keepdim=True)
    ds = c * p * (dp - D) / math.sqrt(st["d"] // 2)
    dq = ds @ _half(k, m)
    dk = (ds.transpose(-1, -2) @ _half(q, m)).sum(2)
    return dq.view(*st["Q"].shape[:3], -1), dk, D


def _plain_bwd(st):
    q, k, v, do = (_grouped(st, n) for n in ("Q", "K", "V", "dO"))
    vis = _mask(st)
    lam = st["lam"].view(st["Hkv"], -1, 1, 1)
    p1, p2 = _plain_map(q, k, 0, vis)[0], _plain_map(q, k, 1, vis)[0]
    dV = ((p1 - lam * p2).transpose(-1, -2) @ do).sum(2)
    dp = do @ v.transpose(-1, -2)
    dq1, dk1, _ = _plain_bwd_map(st, 0, 1.0, p1, dp, q, k)
    dq2, dk2, D2 = _plain_bwd_map(st, 1, -lam, p2, dp, q, k)
    return (torch.cat([dq1, dq2], -1).to(BF), torch.cat([dk1, dk2], -1).to(BF), dV.to(BF),
            -D2.sum((0, 3, 4)).view(-1).to(BF))


def _plain_decode(st):
    B, Hq, Hkv, d = st["B"], st["Hq"], st["Hkv"], st["d"]
    n = max(st["lens_host"])
    k, v = st["K"], st["V"]
    if st["paged"]:
        used = st["table"][:, :(n + st["page"] - 1) // st["page"]].long()
        k, v = (x[used].transpose(1, 2).reshape(B, Hkv, -1, d) for x in (k, v))
    k, v = k[:, :, :n].float(), v[:, :, :n].float()
    q = st["Q"].float().view(B, Hkv, -1, d)
    vis = torch.arange(n, device="cuda") < st["k_lens"].view(-1, 1, 1, 1)
    p1, l1 = _plain_map(q, k, 0, vis)
    p2, l2 = _plain_map(q, k, 1, vis)
    O = (p1 - st["lam"].view(Hkv, -1, 1) * p2) @ v
    return O.view(B, Hq, 1, d).to(BF), torch.stack([l1, l2], -1).view(B, Hq, 2)


def _rotate(x, cos, sin, maps, rope, interleaved):
    """Rotates the first ``rope`` elements of each of the head row's ``maps`` parts."""
    T, H, d = x.shape
    y = x.clone().view(T, H, maps, d // maps)
    cos, sin = cos[:, None, None], sin[:, None, None]
    if interleaved:
        a, b = y[..., 0:rope:2].clone(), y[..., 1:rope:2].clone()
        y[..., 0:rope:2], y[..., 1:rope:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = y[..., :rope // 2].clone(), y[..., rope // 2:rope].clone()
        y[..., :rope // 2], y[..., rope // 2:rope] = a * cos - b * sin, b * cos + a * sin
    return y.view(T, H, d)


def _plain_append(st):
    n, page = st["n_tok"], st["page"]
    row = st["row"]
    cos, sin = st["cos"][row], st["sin"][row]
    args = (cos, sin, st["maps"], st["rope"], st["interleaved"])
    st["Q_out"][:n] = _rotate(st["Q"][:n].float(), *args).to(BF)
    pg = st["table"][st["seq"], row // page].long()
    st["Kp"][pg, :, row % page] = _rotate(st["K"][:n].float(), *args).to(BF)
    st["Vp"][pg, :, row % page] = st["V"][:n]
    return st["Q_out"], st["Kp"], st["Vp"]


# ------------------------------------------------------------------ one pass


def _workspace_bytes(attn, st):
    B, Hq, Hkv, d = st["B"], st["Hq"], st["Hkv"], st["d"]
    if st["op"] == "append":
        return attn.attn_kv_append_paged_workspace_size()
    if st["op"] == "decode":
        L = st["table"].shape[1] * st["page"] if st["paged"] else st["Lmax"]
        return attn.attn_decode_diff_workspace_size(B, Hq, Hkv, L, d)
    size = attn.attn_fwd_diff_workspace_size if st["op"] == "fwd" else \
        attn.attn_bwd_diff_workspace_size
    return size(B, Hq, Hkv, st["Lq"], st["Lk"], d)


def run(state):
    st = state
    if not own:
        return {"append": _plain_append, "fwd": _plain_fwd, "bwd": _plain_bwd,
                "decode": _plain_decode}[st["op"]](st)
    import exact_io_aware_46_b200 as attn

    if "ws" not in st:  # a program keeps its workspace from call to call
        st["ws"] = torch.zeros(_workspace_bytes(attn, st), dtype=torch.uint8, device="cuda")
    if st["op"] == "append":
        attn.attn_kv_append_paged(st["K"], st["V"], st["Kp"], st["Vp"], st["table"], st["k_lens"],
                                  cu_seqlens=st["cu"], Q=st["Q"], Q_out=st["Q_out"],
                                  cos=st["cos"], sin=st["sin"], maps=st["maps"],
                                  interleaved=st["interleaved"], workspace=st["ws"])
        return st["Q_out"], st["Kp"], st["Vp"]
    if st["op"] == "fwd":
        return attn.attn_fwd_diff(st["Q"], st["K"], st["V"], st["lam"], causal=st["causal"],
                                  k_lens=st["k_lens"], workspace=st["ws"])
    if st["op"] == "bwd":
        return attn.attn_bwd_diff(st["Q"], st["K"], st["V"], st["lam"], st["O"], st["O2"],
                                  st["dO"], st["lse"], causal=st["causal"], k_lens=st["k_lens"],
                                  workspace=st["ws"])
    if st["paged"]:
        return attn.attn_fwd_splitkv_decode_diff_paged(
            st["Q"], st["K"], st["V"], st["table"], st["lam"], st["k_lens"], O=st["O"],
            lse=st["lse"], workspace=st["ws"])
    return attn.attn_fwd_splitkv_decode_diff(st["Q"], st["K"], st["V"], st["lam"], st["k_lens"],
                                             O=st["O"], lse=st["lse"], workspace=st["ws"])


# ------------------------------------------------------------------ the definition in 64 bits


def _def_fwd(c, q, k, v, lam, kl):
    """One query head of one sequence: (O, O2, lse [2, Lq]) by torch's softmax in 64 bits."""
    Lq, Lk, h = q.shape[0], k.shape[0], c["d"] // 2
    hide = torch.zeros(Lq, Lk, dtype=torch.bool, device=q.device)
    hide[:, kl:] = True
    if c["causal"]:
        hide |= torch.ones(Lq, Lk, dtype=torch.bool, device=q.device).triu(Lk - Lq + 1)
    o, ls = [], []
    for m in (slice(0, h), slice(h, 2 * h)):
        s = (torch.einsum("id,jd->ij", q[:, m], k[:, m]) / math.sqrt(h)).masked_fill(hide, -math.inf)
        o.append(torch.einsum("ij,jd->id", s.softmax(-1), v))
        ls.append(torch.logsumexp(s, -1))
    return o[0] - lam * o[1], o[1], torch.stack(ls)


def _cache_rows(st, name, b):
    """The visible rows [k_len, Hkv, d] of one sequence's cache."""
    n = st["lens_host"][b]
    if not st["paged"]:
        return st[name][b, :, :n].transpose(0, 1)
    nb = (n + st["page"] - 1) // st["page"]
    x = st[name][st["table"][b, :nb].long()]
    return x.transpose(1, 2).reshape(nb * st["page"], st["Hkv"], st["d"])[:n]


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    d64 = torch.float64
    B, Hq, d = c["B"], c["Hq"], c["d"]
    G = Hq // c["Hkv"]
    if c["op"] == "append":
        q, kp, vp = (st[n].to(d64) for n in ("Q_out", "Kp", "Vp"))
        n, past = _append_sizes(c)
        part, half = d // c["maps"], c["rope"] // 2
        # element pairs of a head row that share an angle
        base = torch.arange(c["maps"], device=q.device)[:, None] * part
        i = torch.arange(half, device=q.device)
        ia = (base + (2 * i if c["interleaved"] else i)).flatten()
        ib = (base + (2 * i + 1 if c["interleaved"] else i + half)).flatten()
        t0 = 0
        for b in range(B):
            rows = torch.arange(past[b], past[b] + n[b], device=q.device)
            z = torch.complex(st["cos"][rows].to(d64), st["sin"][rows].to(d64))
            z = z.repeat(1, c["maps"])[:, None]

            def turn(x):
                x = x[t0:t0 + n[b]].to(d64)
                w = torch.complex(x[..., ia], x[..., ib]) * z
                x[..., ia], x[..., ib] = w.real, w.imag
                return x

            q[t0:t0 + n[b]] = turn(st["Q"])
            pages = st["table"][b].long().repeat_interleave(c["page"])[rows]
            kp[pages, :, rows % c["page"]] = turn(st["K"])
            vp[pages, :, rows % c["page"]] = st["V"][t0:t0 + n[b]].to(d64)
            t0 += n[b]
        return q, kp, vp
    if c["op"] == "decode":
        O = torch.empty(B, Hq, 1, d, dtype=d64, device="cuda")
        lse = torch.empty(B, Hq, 2, dtype=d64, device="cuda")
        for b in range(B):
            k, v = _cache_rows(st, "K", b), _cache_rows(st, "V", b)
            for g in range(c["Hkv"]):
                kg, vg = k[:, g].to(d64), v[:, g].to(d64)
                for hq in range(g * G, (g + 1) * G):
                    o, _, ls = _def_fwd(dict(d=d, causal=False), st["Q"][b, hq].to(d64), kg, vg,
                                        st["lam"][hq].to(d64), kg.shape[0])
                    O[b, hq], lse[b, hq] = o, ls[:, 0]
        return O, lse
    q, k, v = (st[n].to(d64) for n in "QKV")
    lam = st["lam"].to(d64)
    if c["op"] == "fwd":
        O, O2 = torch.empty_like(q), torch.empty_like(q)
        lse = torch.empty(B, Hq, 2, c["Lq"], dtype=d64, device="cuda")
        for b in range(B):
            for hq in range(Hq):
                O[b, hq], O2[b, hq], lse[b, hq] = _def_fwd(
                    c, q[b, hq], k[b, hq // G], v[b, hq // G], lam[hq], st["lens_host"][b])
        return O, O2, lse
    # gradients by automatic differentiation of the definition
    dQ, dK, dV, dlam = (torch.zeros_like(t) for t in (q, k, v, lam))
    for b in range(B):
        for hq in range(Hq):
            leaves = [t.clone().requires_grad_() for t in (q[b, hq], k[b, hq // G], v[b, hq // G],
                                                           lam[hq])]
            o = _def_fwd(c, *leaves, st["lens_host"][b])[0]
            gq, gk, gv, gl = torch.autograd.grad(o, leaves, st["dO"][b, hq].to(d64))
            dQ[b, hq] = gq
            dK[b, hq // G] += gk
            dV[b, hq // G] += gv
            dlam[hq] += gl
    return dQ, dK, dV, dlam
