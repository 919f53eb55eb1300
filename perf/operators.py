"""What is measured of the operators around a served or trained attention layer.

Four operators, by the "op" of a case:

- chunk:  attention of each request's new tokens over its cached keys (the new
          tokens' own keys are in the cache already), through a page table or
          contiguous, bf16 or e4m3 cache, optionally with a sliding window and
          logits capped by a tanh;
- train:  RMS norm of every query and key head and the position rotation in one
          pass over the flat shared-prefix layout, with its gradients;
- append: the serving form of the same pass: queries out, keys and values
          written (e4m3: quantised) into their cache rows;
- read:   cached rows read back (dequantised) into dense bf16 keys and values.

``run`` computes them in elementary torch operations when ``own`` is false and
through ``shared_prefix_attention_b200`` when it is true.
"""
import math
import random

import torch

own = False

F8 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # four requests decoding one token each over short histories: latency
        dict(name="chunk-decode", op="chunk", B=4, nq=1, ctx=900, ragged=True, Hq=32, Hkv=8, d=128,
             paged=True, cache="bf16", window=0, cap=0.0, lens=1),
        # a serving step that mixes short and long pieces over 16k histories
        dict(name="chunk-mixed", op="chunk", B=8, nq=512, ctx=16384, ragged=True, Hq=32, Hkv=8,
             d=128, paged=True, cache="bf16", window=0, cap=0.0, lens=2),
        # one long prompt's next piece, its history in one contiguous range
        dict(name="chunk-long", op="chunk", B=1, nq=2048, ctx=16384, ragged=False, Hq=32, Hkv=8,
             d=128, paged=False, cache="bf16", window=0, cap=0.0, lens=3),
        # pieces of 1024 tokens over e4m3 histories through a page table
        dict(name="chunk-e4m3", op="chunk", B=4, nq=1024, ctx=8192, ragged=True, Hq=32, Hkv=8,
             d=128, paged=True, cache="e4m3", window=0, cap=0.0, lens=4),
        # a layer with capped logits and a sliding window, 64-wide heads
        dict(name="chunk-capped", op="chunk", B=3, nq=777, ctx=6000, ragged=True, Hq=16, Hkv=16,
             d=64, paged=True, cache="bf16", window=4096, cap=30.0, lens=5),
        # a GRPO group in training: every suffix's positions go on from the prefix
        dict(name="train-grpo", op="train", groups=1, P=2048, N=8, S=512, Hq=16, Hkv=16, d=128,
             rot=128, interleaved=False, dtype="bf16"),
        # two packed groups of the large prefill
        dict(name="train-large", op="train", groups=2, P=8192, N=16, S=1024, Hq=32, Hkv=8, d=128,
             rot=128, interleaved=False, dtype="bf16"),
        # a small fp32 check model: odd length, half of each head rotated in pairs
        dict(name="train-small", op="train", groups=1, P=129, N=8, S=81, Hq=4, Hkv=2, d=64, rot=32,
             interleaved=True, dtype="f32"),
        # one decoding step of 32 requests into an e4m3 cache: latency
        dict(name="append-decode", op="append", T=32, pad=0, Hq=32, Hkv=8, d=128, rot=128,
             interleaved=False, cache="e4m3", ntok=8192),
        # a prefill piece with padding behind its last sequence
        dict(name="append-chunk", op="append", T=8192, pad=77, Hq=32, Hkv=8, d=128, rot=128,
             interleaved=False, cache="e4m3", ntok=16384),
        # a short cached range back into dense tensors
        dict(name="read-short", op="read", n=300, Hkv=8, d=128, cache="bf16", ntok=16384),
        # a request's whole e4m3 history back into dense bf16
        dict(name="read-long", op="read", n=65536, Hkv=8, d=128, cache="e4m3", ntok=131072),
    ]


HEADS = [(32, 8), (16, 16), (8, 2), (8, 1), (24, 8), (28, 4), (5, 1)]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "train", "append", "read"])
    Hq, Hkv = rng.choice(HEADS)
    d = rng.choice([64, 128, 128])
    rot = rng.choice([d, d, d // 2])
    if op == "chunk":
        cap = rng.choice([0.0, 0.0, 30.0, 50.0])
        window = rng.choice([0, 0, _log(rng, 64, 8192)])
        while True:
            c = dict(op="chunk", B=_log(rng, 1, 16), nq=_log(rng, 1, 2048), ctx=_log(rng, 1, 16384),
                     ragged=True, Hq=Hq, Hkv=Hkv, d=d, paged=rng.random() < 0.7,
                     cache=rng.choice(["bf16", "e4m3"]), window=window, cap=cap,
                     lens=rng.randrange(1 << 20))
            if c["B"] * Hq * c["nq"] * (c["nq"] + c["ctx"]) <= 1 << 30:
                return c
    if op == "train":
        return dict(op="train", groups=rng.choice([1, 2]), P=_log(rng, 16, 4096), N=_log(rng, 1, 16),
                    S=_log(rng, 1, 1024), Hq=Hq, Hkv=Hkv, d=d, rot=rot,
                    interleaved=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "append":
        T = _log(rng, 1, 8192)
        return dict(op="append", T=T, pad=rng.randrange(0, 1 + T // 4), Hq=Hq, Hkv=Hkv, d=d, rot=rot,
                    interleaved=rng.random() < 0.5, cache=rng.choice(["bf16", "e4m3"]),
                    ntok=T + rng.randrange(1, 8192))
    n = _log(rng, 1, 65536)
    return dict(op="read", n=n, Hkv=Hkv, d=d, cache=rng.choice(["bf16", "e4m3"]),
                ntok=n + rng.randrange(0, 65536))


# ------------------------------------------------------------------ inputs

def _lens(case):
    """New tokens and cached keys (these included) of each request."""
    r = random.Random(case["lens"])
    q, kv = [], []
    for b in range(case["B"]):
        whole = b == 0 or not case["ragged"]  # one request has the full sizes
        n = case["nq"] if whole else r.randint(1, case["nq"])
        h = case["ctx"] if whole else r.randint(0, case["ctx"])
        q.append(n)
        kv.append(n + h)
    return q, kv


def _indptr(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _cache(gen, ntok, Hkv, d, kind):
    """Key and value caches and their scales (rotated, normed keys are of unit size)."""
    k, v = (torch.randn(ntok, Hkv, d, device="cuda", dtype=torch.bfloat16, generator=gen)
            for _ in range(2))
    if kind == "bf16":
        return k, v, None, None
    ks, vs = 0.021, 0.017
    return (k.float() / ks).clamp(-448, 448).to(F8), (v.float() / vs).clamp(-448, 448).to(F8), ks, vs


def _angles(npos, rot):
    """cos and sin of every position's rotation, [npos, rot] fp32 (angles in 64 bits)."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = torch.arange(npos, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _tokens(case):
    return case["groups"] * (case["P"] + case["N"] * case["S"])


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    i32 = dict(device="cuda", dtype=torch.int32)
    st = dict(case=case)
    op, d, Hkv = case["op"], case["d"], case["Hkv"]
    if op == "chunk":
        ql, kl = _lens(case)
        n, nk = sum(ql), sum(kl)
        q = torch.randn(n, case["Hq"], d, device="cuda", generator=g)
        # capped layers are the ones whose logits grow large
        st["q"] = (q * (6.0 if case["cap"] else 1.0)).bfloat16()
        ntok = nk + nk // 4 if case["paged"] else nk
        st["k"], st["v"], st["ks"], st["vs"] = _cache(g, ntok, Hkv, d, case["cache"])
        st["table"] = (torch.randperm(ntok, device="cuda", generator=g)[:nk].to(torch.int32)
                       if case["paged"] else None)
        st["qo"], st["kv"] = torch.tensor(_indptr(ql), **i32), torch.tensor(_indptr(kl), **i32)
        st["nmax"], st["lmax"] = max(ql), max(kl)
        if own:
            import shared_prefix_attention_b200 as psa
            st["plan"] = psa.plan_chunk(ql, kl, case["Hq"], Hkv, d, window=case["window"])
        return st
    if op == "train":
        T, Hq, dt = _tokens(case), case["Hq"], DTYPES[case["dtype"]]
        # the projection's output: queries, keys and values of a token side by side
        x = torch.randn(T, (Hq + 2 * Hkv) * d, device="cuda", generator=g, dtype=dt)
        st["q"] = x[:, :Hq * d].unflatten(1, (Hq, d))
        st["k"] = x[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
        st["dq"] = torch.randn(T, Hq, d, device="cuda", generator=g, dtype=dt)
        st["dk"] = torch.randn(T, Hkv, d, device="cuda", generator=g, dtype=dt)
        one = torch.arange(case["P"], **i32)
        more = torch.arange(case["P"], case["P"] + case["S"], **i32).repeat(case["N"])
        st["pos"] = torch.cat([one, more]).repeat(case["groups"])
        st["cs"] = _angles(case["P"] + case["S"], case["rot"])
    elif op == "append":
        T, Hq, ntok = case["T"], case["Hq"], case["ntok"]
        x = torch.randn(T, (Hq + 2 * Hkv) * d, device="cuda", generator=g, dtype=torch.bfloat16)
        st["q"] = x[:, :Hq * d].unflatten(1, (Hq, d))
        st["kn"] = x[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
        st["vn"] = x[:, (Hq + Hkv) * d:].unflatten(1, (Hkv, d))
        st["k"], st["v"], st["ks"], st["vs"] = _cache(g, ntok, Hkv, d, case["cache"])
        st["slots"] = torch.randperm(ntok, device="cuda", generator=g)[:T].to(torch.int32)
        st["slots"][T - case["pad"]:] = -1
        st["pos"] = torch.randint(0, 16384, (T,), device="cuda", generator=g).to(torch.int32)
        st["cs"] = _angles(16384, case["rot"])
    else:
        st["k"], st["v"], st["ks"], st["vs"] = _cache(g, case["ntok"], Hkv, d, case["cache"])
        st["rows"] = torch.randperm(case["ntok"], device="cuda", generator=g)[:case["n"]].to(torch.int32)
        return st
    st["qw"] = 1 + 0.1 * torch.randn(d, device="cuda", generator=g)
    st["kw"] = 1 + 0.1 * torch.randn(d, device="cuda", generator=g)
    return st


EPS = 1e-6


# ------------------------------------------------------------------ plain forms

def _rotate(x, cs, inter, sign=1.0):
    """x [T, H, d] fp32 with its first rot elements rotated by cs [T, rot]; sign -1: back."""
    rot = cs.shape[1]
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:] * sign
    y = x.clone()
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, a * s + b * c
    return y


def _norm_rope(x, w, cs, inter):
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return _rotate(x * r * w, cs, inter)


def _norm_rope_grad(x, dy, w, cs, inter):
    x, g = x.float(), _rotate(dy.float(), cs, inter, -1.0)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xh = x * r
    wg = w * g
    return r * (wg - xh * (wg * xh).mean(-1, keepdim=True)), (g * xh).sum((0, 1))


def _rows(cache, idx, scale):
    """Rows of a cache as the fp32 values they stand for."""
    if cache.dtype == F8:
        return cache.view(torch.uint8)[idx].view(F8).float() * scale
    return cache[idx].float()


def _plain_chunk(st):
    case = st["case"]
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    qo, kv = st["qo"].long(), st["kv"].long()
    nq, nk = qo[1:] - qo[:-1], kv[1:] - kv[:-1]
    i = torch.arange(st["nmax"], device="cuda")
    j = torch.arange(st["lmax"], device="cuda")
    rows = (qo[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)       # [B, nmax]
    keys = (kv[:-1, None] + j).clamp(max=int(sum(_lens(case)[1])) - 1)  # [B, lmax]
    if st["table"] is not None:
        keys = st["table"].long()[keys]
    q = st["q"][rows].float().unflatten(2, (Hkv, Hq // Hkv)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    k = _rows(st["k"], keys, st["ks"]).transpose(1, 2)               # [B, Hkv, lmax, d]
    v = _rows(st["v"], keys, st["vs"]).transpose(1, 2)
    s = (q @ k.transpose(2, 3)) * d ** -0.5                          # [B, Hkv, G * nmax, lmax]
    if case["cap"]:
        s = case["cap"] * torch.tanh(s / case["cap"])
    at = (nk - nq)[:, None] + i                                      # a row's own position
    see = (j <= at[..., None]) & (j < nk[:, None, None])
    if case["window"]:
        see &= j > at[..., None] - case["window"]
    s = s.unflatten(2, (Hq // Hkv, st["nmax"])).masked_fill(~see[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(s - m)
    del s
    l = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).unflatten(2, (Hq // Hkv, st["nmax"])) / l
    lse = (m + l.log())[..., 0]
    real = i < nq[:, None]                                           # [B, nmax]
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[real]
    return o.to(torch.bfloat16), lse.permute(0, 3, 1, 2).flatten(2, 3)[real]


def _plain_append(st):
    case = st["case"]
    cs = st["cs"][st["pos"].long()]
    inter = case["interleaved"]
    live = st["slots"] >= 0
    at = st["slots"][live].long()
    k = _norm_rope(st["kn"], st["kw"], cs, inter)[live]
    v = st["vn"].float()[live]
    if case["cache"] == "e4m3":
        st["k"].view(torch.uint8)[at] = (k / st["ks"]).clamp(-448, 448).to(F8).view(torch.uint8)
        st["v"].view(torch.uint8)[at] = (v / st["vs"]).clamp(-448, 448).to(F8).view(torch.uint8)
    else:
        st["k"][at] = k.to(torch.bfloat16)
        st["v"][at] = v.to(torch.bfloat16)
    return _norm_rope(st["q"], st["qw"], cs, inter).to(torch.bfloat16), st["k"], st["v"]


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        import shared_prefix_attention_b200 as psa
        if op == "chunk":
            return psa.chunk(st["q"], st["k"], st["v"], st["plan"], case["d"] ** -0.5,
                             kv_indices=st["table"], logit_cap=case["cap"], k_scale=st["ks"],
                             v_scale=st["vs"])
        if op == "train":
            how = dict(q_weight=st["qw"], k_weight=st["kw"], eps=EPS, interleaved=case["interleaved"])
            y = psa.qk_norm_rope(st["q"], st["k"], st["pos"], st["cs"], **how)
            return y, psa.qk_norm_rope_bwd(st["q"], st["k"], st["dq"], st["dk"], st["pos"], st["cs"],
                                           **how)
        if op == "append":
            q = psa.cache_append(st["q"], st["kn"], st["vn"], st["k"], st["v"], st["slots"],
                                 positions=st["pos"], cos_sin=st["cs"], q_weight=st["qw"],
                                 k_weight=st["kw"], eps=EPS, interleaved=case["interleaved"],
                                 k_scale=st["ks"], v_scale=st["vs"])
            return q, st["k"], st["v"]
        return psa.cache_read(st["k"], st["v"], st["rows"], k_scale=st["ks"], v_scale=st["vs"])
    if op == "chunk":
        return _plain_chunk(st)
    if op == "train":
        cs, inter = st["cs"][st["pos"].long()], case["interleaved"]
        dt = st["q"].dtype
        yq = _norm_rope(st["q"], st["qw"], cs, inter).to(dt)
        yk = _norm_rope(st["k"], st["kw"], cs, inter).to(dt)
        dq, dqw = _norm_rope_grad(st["q"], st["dq"], st["qw"], cs, inter)
        dk, dkw = _norm_rope_grad(st["k"], st["dk"], st["kw"], cs, inter)
        return (yq, yk), (dq.to(dt), dk.to(dt), dqw, dkw)
    if op == "append":
        return _plain_append(st)
    rows = st["rows"].long()
    return tuple(_rows(st[c], rows, st[c + "s"]).to(torch.bfloat16) for c in "kv")


# ------------------------------------------------------------------ work and 64 bits

def _pairs(case):
    """Visible (query, key) pairs and the cached keys that some query sees."""
    pairs = keys = 0
    w = case["window"]
    for n, L in zip(*_lens(case)):
        h = L - n
        first = max(0, h + 1 - w) if w else 0
        keys += L - first
        # query i sees min(h + i + 1, w) keys
        full = n if not w else max(0, min(n, w - h))
        pairs += full * h + full * (full + 1) // 2 + (n - full) * w
    return pairs, keys


def work(case):
    d, Hkv = case["d"], case["Hkv"]
    one = 1 if case.get("cache") == "e4m3" else 2
    if case["op"] == "chunk":
        pairs, keys = _pairs(case)
        n = sum(_lens(case)[0])
        return {"bytes": 2 * keys * Hkv * d * one + n * case["Hq"] * (4 * d + 4)
                + (4 * keys if case["paged"] else 0), "flops": 4 * d * case["Hq"] * pairs}
    if case["op"] == "train":
        x = _tokens(case) * (case["Hq"] + Hkv) * d
        size = 4 if case["dtype"] == "f32" else 2
        # forward and gradients are two calls: x in, y out; x and dy in, dx out
        return {"bytes": 5 * x * size + 2 * 4 * (case["P"] + case["S"]) * case["rot"], "flops": 24 * x}
    if case["op"] == "append":
        T, live = case["T"], case["T"] - case["pad"]
        return {"bytes": T * case["Hq"] * d * 4 + live * Hkv * d * 2 * (2 + one)
                + min(T, 16384) * case["rot"] * 4 + 8 * T,
                "flops": 10 * (T * case["Hq"] + 2 * live * Hkv) * d}
    return {"bytes": 2 * case["n"] * Hkv * d * (2 + one) + 4 * case["n"],
            "flops": 2 * case["n"] * Hkv * d}


def _rope64(x, w, cs, inter):
    """Norm and rotation as one complex product per pair, in 64 bits."""
    x = x.double()
    y = x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * w.double()
    h = cs.shape[1] // 2
    turn = torch.complex(cs[:, :h].double(), cs[:, h:].double())[:, None]
    head, rest = y[..., :2 * h], y[..., 2 * h:]
    pairs = head.unflatten(-1, (h, 2)) if inter else head.unflatten(-1, (2, h)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    head = z.flatten(-2) if inter else z.transpose(-1, -2).flatten(-2)
    return torch.cat([head, rest], -1)


def exact(case, seed):
    st = prepare_plain(case, seed)
    op = case["op"]
    if op == "read":
        rows = st["rows"].long()
        return tuple(_rows(st[c], rows, 1.0).double() * (st[c + "s"] or 1.0) for c in "kv")
    if op == "train":
        cs, inter = st["cs"][st["pos"].long()], case["interleaved"]
        y, dx, dw = [], [], []
        for c in "qk":
            x = st[c].double().requires_grad_()
            w = st[c + "w"].double().requires_grad_()
            out = _rope64(x, w, cs, inter)
            gx, gw = torch.autograd.grad(out, (x, w), st["d" + c].double())
            y.append(out.detach())
            dx.append(gx)
            dw.append(gw)
        return tuple(y), (dx[0], dx[1], dw[0], dw[1])
    if op == "append":
        cs, inter = st["cs"][st["pos"].long()], case["interleaved"]
        at = st["slots"].long()
        at = at[at >= 0]
        n = at.numel()
        k = _rope64(st["kn"], st["kw"], cs, inter)[:n]
        v = st["vn"].double()[:n]
        out = [_rope64(st["q"], st["qw"], cs, inter)]
        for c, x in (("k", k), ("v", v)):
            if case["cache"] == "e4m3":
                full = st[c].float().double()
                full[at] = (x / st[c + "s"]).clamp(-448, 448).to(F8).double()
            else:
                full = st[c].double()
                full[at] = x
            out.append(full)
        return tuple(out)
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    n = st["q"].shape[0]
    o = torch.empty(n, Hq, d, device="cuda", dtype=torch.float64)
    lse = torch.empty(n, Hq, device="cuda", dtype=torch.float64)
    ql, kl = _lens(case)
    q0 = k0 = 0
    for nq, L in zip(ql, kl):
        idx = torch.arange(k0, k0 + L, device="cuda")
        if st["table"] is not None:
            idx = st["table"][idx].long()
        k = _rows(st["k"], idx, 1.0).double() * (st["ks"] or 1.0)
        v = _rows(st["v"], idx, 1.0).double() * (st["vs"] or 1.0)
        far = (L - nq + torch.arange(nq, device="cuda"))[:, None] - torch.arange(L, device="cuda")
        hide = far < 0
        if case["window"]:
            hide |= far >= case["window"]
        for h in range(Hq):
            s = st["q"][q0:q0 + nq, h].double() @ k[:, h // (Hq // Hkv)].T / math.sqrt(d)
            if case["cap"]:
                s = case["cap"] * torch.tanh(s / case["cap"])
            s[hide] = -math.inf
            z = torch.logsumexp(s, 1)
            o[q0:q0 + nq, h] = torch.exp(s - z[:, None]) @ v[:, h // (Hq // Hkv)]
            lse[q0:q0 + nq, h] = z
        q0 += nq
        k0 += L
    return o, lse


def prepare_plain(case, seed):
    """The inputs alone, without the framework's plan."""
    global own
    kept, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = kept
