"""Chunk attention on the GPU against its formula in 64 bits.

Tolerances.  With A = sum_j p_j |v_j| / l (p the weights, l their sum):
rounding each weight to 16 bits moves o by at most h A, h = 2^-8 (bf16) or
2^-11 (f16, e4m3 caches), and the store by at most 2^-8 |o|.  A logit is a sum
of d products accumulated in fp32 (each partial sum truncated or rounded: at
most d 2^-23 S, S = scale sum_d |q_d k_d|), scaled and exponentiated with
relative errors of a few 2^-23 of its size: together at most e = (d + 16) 2^-23
(S + 1); a relative change e of each weight moves o by at most 2 e A and the
lse by e.  A cap adds 2^-20 c (its error is absolute)."""
import numpy as np
import pytest
import torch

import shared_prefix_attention_b200 as psa

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


def reference(q, k, v, ql, kl, table, scale, window, cap):
    """(o, lse, A, S) of every new token in 64 bits; k, v the values the
    cache stands for."""
    Hq, d = q.shape[1:]
    Hkv = k.shape[1]
    G = Hq // Hkv
    o, lse, A, S = [], [], [], []
    q0 = k0 = 0
    for n, L in zip(ql, kl):
        idx = torch.arange(k0, k0 + L, device="cuda")
        if table is not None:
            idx = table[idx].long()
        kk, vv = k[idx].double(), v[idx].double()
        qq = q[q0:q0 + n].double().unflatten(1, (Hkv, G))
        s = torch.einsum("nhgd,lhd->hgnl", qq, kk) * scale
        S.append((torch.einsum("nhgd,lhd->hgnl", qq.abs(), kk.abs()) * scale).amax(-1)
                 .permute(2, 0, 1).flatten(1) if L else torch.zeros(n, Hq, device="cuda"))
        if cap:
            s = cap * torch.tanh(s / cap)
        at = L - n + torch.arange(n, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")
        see = j <= at
        if window:
            see &= j > at - window
        s = s.masked_fill(~see, -float("inf"))
        z = torch.logsumexp(s, -1)
        p = torch.exp(s - z[..., None])
        o.append(torch.einsum("hgnl,lhd->nhgd", p, vv).flatten(1, 2))
        A.append(torch.einsum("hgnl,lhd->nhgd", p, vv.abs()).flatten(1, 2))
        lse.append(z.permute(2, 0, 1).flatten(1))
        q0 += n
        k0 += L
    return tuple(torch.cat(x) for x in (o, lse, A, S))


def make(ql, kl, Hq, Hkv, d, paged, kind, seed, qscale=1.0, spare=37):
    g = torch.Generator().manual_seed(seed)
    n, nk = sum(ql), sum(kl)
    q = (torch.randn(n, Hq, d, generator=g) * qscale).bfloat16().cuda()
    ntok = nk + spare
    k, v = (torch.randn(ntok, Hkv, d, generator=g).bfloat16().cuda() for _ in range(2))
    ks = vs = None
    if kind == "e4m3":
        ks, vs = 0.021, 0.017
        k, v = ((x.float() / s).clamp(-448, 448).to(F8) for x, s in ((k, ks), (v, vs)))
    table = torch.randperm(ntok, generator=g)[:nk].int().cuda() if paged else None
    # rows no request owns hold NaN: nothing may read them into a result
    unused = torch.ones(ntok, dtype=torch.bool, device="cuda")
    unused[table.long() if paged else slice(0, nk)] = False
    for c in (k, v):
        if kind == "e4m3":
            c.view(torch.uint8)[unused] = 0x7f
        else:
            c[unused] = float("nan")
    return q, k, v, ks, vs, table


def values(c, s):
    return c.double() if s is None else c.float().double() * float(np.float32(s))


def check(o, lse, ref, d, cap, h, what):
    ro, rl, A, S = ref
    e = (d + 16) * 2.0 ** -23 * (S + 1) + 2.0 ** -20 * cap
    assert torch.isfinite(o.float()).all() and torch.isfinite(lse).all(), what
    err = (lse.double() - rl).abs() - e
    assert float(err.max()) <= 0, f"{what}: lse over its bound by {float(err.max()):.3e}"
    tol = h * A + 2.0 ** -8 * ro.abs() + 2 * e[..., None] * A
    err = (o.double() - ro).abs() - tol
    assert float(err.max()) <= 0, f"{what}: o over its bound by {float(err.max()):.3e}"


CASES = [
    # qo lens, kv lens, Hq, Hkv, d, paged, cache, window, cap
    ([1], [1], 8, 2, 128, True, "bf16", 0, 0.0),
    ([1, 1, 1, 1], [901, 583, 2, 508], 32, 8, 128, True, "bf16", 0, 0.0),
    ([1, 0, 3], [5000, 0, 129], 28, 4, 128, True, "e4m3", 0, 0.0),
    ([5], [5], 5, 1, 64, False, "bf16", 0, 0.0),
    ([64, 65, 1], [64, 200, 128], 32, 8, 128, False, "bf16", 0, 0.0),
    ([200], [1333], 16, 16, 64, True, "bf16", 100, 0.0),
    ([300, 17], [300, 1000], 24, 8, 128, True, "bf16", 0, 30.0),
    ([257, 40], [1500, 40], 8, 1, 128, True, "e4m3", 64, 50.0),
    ([130, 2], [700, 4000], 28, 4, 64, True, "e4m3", 0, 0.0),
    ([777], [2000], 16, 16, 64, True, "bf16", 512, 30.0),
    ([513, 100, 31], [2048, 777, 5000], 32, 8, 128, True, "bf16", 0, 0.0),
    ([400], [3000], 8, 2, 128, False, "e4m3", 0, 0.0),
    ([9, 1, 33], [40, 77, 33], 4, 4, 128, True, "bf16", 1, 0.0),
    ([33], [9000], 64, 1, 64, True, "bf16", 0, 0.0),
    ([3], [700], 128, 1, 128, False, "bf16", 300, 0.0),
]


@pytest.mark.parametrize("ql,kl,Hq,Hkv,d,paged,kind,window,cap", CASES)
def test_parity(ql, kl, Hq, Hkv, d, paged, kind, window, cap):
    scale = d ** -0.5
    q, k, v, ks, vs, table = make(ql, kl, Hq, Hkv, d, paged, kind, sum(kl),
                                  6.0 if cap else 1.0)
    plan = psa.plan_chunk(ql, kl, Hq, Hkv, d, window)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = psa.chunk(q, k, v, plan, scale, kv_indices=table, logit_cap=cap, k_scale=ks,
                       v_scale=vs, status=st)
    assert psa.read_status(st) == 0
    ref = reference(q, values(k, ks), values(v, vs), ql, kl, table, scale, window, cap)
    check(o, lse, ref, d, cap, 2.0 ** -11 if ks else 2.0 ** -8, str((ql, kl)))
    o2, lse2 = psa.chunk(q, k, v, plan, scale, kv_indices=table, logit_cap=cap, k_scale=ks,
                         v_scale=vs)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)  # every sum has a fixed order
