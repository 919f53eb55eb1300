"""Chunk attention where the softmax weights are hard to hold: one key far above
many small ones, logits that are infinite or at the largest cap."""
import ctypes
import math

import pytest
import torch

import shared_prefix_attention_b200 as psa
from test_chunk_gpu import F8, reference, values

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # half a step of fp32


def see_of(n, L):
    at = L - n + torch.arange(n, device="cuda")[:, None]
    return torch.arange(L, device="cuda") <= at


@pytest.mark.parametrize("n,L,Hq,Hkv,d,paged,cap,share", [
    (1, 16500, 8, 2, 128, True, 0.0, 0.99),
    (3, 65536, 4, 1, 64, False, 0.0, 0.99),
    (300, 16384, 8, 2, 128, True, 0.0, 0.99),
    (200, 40000, 4, 4, 64, True, 0.0, 0.9),
    (2, 20000, 8, 1, 128, True, 50.0, 0.99),
    (260, 16384, 4, 2, 128, False, 50.0, 0.99),
])
@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
def test_one_dominant_key_of_value_zero(n, L, Hq, Hkv, d, paged, cap, share, kind):
    """The first key takes about `share` of the weight and adds nothing; the output is
    what the many keys far below it leave.  Bound: each weight is off by half a
    step (2^-11 of it in f16, over e4m3 caches, else 2^-8), in f16 at least by
    2^-32 of the largest weight, which is 1 / l of the whole; logits and the
    store as in the parity test."""
    g = torch.Generator().manual_seed(L + n)
    scale = d ** -0.5
    ks, vs = (0.125, 0.03125) if kind == "e4m3" else (None, None)
    q = torch.zeros(n, Hq, d)
    q[..., 0] = torch.linspace(7.5, 8.5, n * Hq).view(n, Hq)  # the others' weights are equal
    q = q.bfloat16().cuda()
    k, v = torch.randn(L + 40, Hkv, d, generator=g), 1.0 + torch.randn(L + 40, Hkv, d, generator=g)
    k[..., 0] = 0.0
    table = torch.randperm(L + 40, generator=g)[:L].int() if paged else None
    first = int(table[0]) if paged else 0
    gap = math.log(L * share / (1 - share))
    if cap:
        gap = cap * math.atanh(gap / cap)
    k[first] = 0.0
    k[first, :, 0] = gap / (8.0 * scale)
    v[first] = 0.0
    if kind == "e4m3":
        k, v = (k / ks).clamp(-448, 448).to(F8).cuda(), (v / vs).clamp(-448, 448).to(F8).cuda()
    else:
        k, v = k.bfloat16().cuda(), v.bfloat16().cuda()
    table = table.cuda() if paged else None
    # one list: the blocks' keys are not cut, whose pieces have maxima of their own
    data, info = psa.build_chunk_plan([n], [L], Hq, Hkv, d, n_ctas=1)
    plan = psa.ChunkPlan(info, torch.from_numpy(data).cuda(),
                         psa.lib().psa_chunk_workspace_size(ctypes.byref(info)))
    o, lse = psa.chunk(q, k, v, plan, scale, kv_indices=table, logit_cap=cap, k_scale=ks,
                       v_scale=vs)
    kk, vv = values(k, ks), values(v, vs)
    ro, rl, A, S = reference(q, kk, vv, [n], [L], table, scale, 0, cap)
    at = torch.arange(L, device="cuda") if table is None else table.long()
    s = torch.einsum("nhgd,lhd->hgnl", q.double().unflatten(1, (Hkv, Hq // Hkv)), kk[at]) * scale
    if cap:
        s = cap * torch.tanh(s / cap)
    see = see_of(n, L)
    top = s.masked_fill(~see, -math.inf).amax(-1).permute(2, 0, 1).flatten(1)
    total = torch.einsum("nl,lhd->nhd", see.double(), vv[at].abs()).repeat_interleave(Hq // Hkv, 1)
    least = 2.0 ** -32 * torch.exp(top - rl)[..., None] * total if ks else 0.0
    h = 2.0 ** -11 if ks else 2.0 ** -8
    e = (d + 16) * 2.0 ** -23 * (S + 1) + 24 * U * cap
    assert float(((lse.double() - rl).abs() - e).max()) <= 0
    tol = h * A + least + 2.0 ** -8 * ro.abs() + 2 * e[..., None] * A
    over = float(((o.double() - ro).abs() / tol).max())
    assert over <= 1, f"{over:.2f} times the bound, o off by " \
        f"{float((o.double() - ro).norm() / ro.norm()):.2%}"


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,L", [(1, 1), (3, 300), (300, 500)])
def test_infinite_logits_reach_the_cap(n, L, kind):
    """c tanh(+-inf / c) is +-c: keys of one infinite element (bf16 caches), and
    products beyond fp32, weigh as keys at the cap, in whole and in partial
    tiles; a row that sees nothing else has their mean.  Weights and values are
    few and small, so the bound is the rounding of weights and store."""
    Hq, Hkv, d, cap = 4, 2, 128, 5.0
    g = torch.Generator().manual_seed(n + L)
    q = torch.zeros(n, Hq, d)
    q[..., 0] = torch.where(torch.rand(n, Hq, generator=g) < 0.5, -1.0, 1.0)
    q[..., 1] = 1.0
    k = torch.zeros(L, Hkv, d)
    k[..., 1] = torch.randint(-2, 3, (L, Hkv), generator=g).float()
    far = torch.rand(L, Hkv, generator=g) < 0.3
    far[:max(1, L // 4)] = True  # the first rows see these alone
    v = torch.randint(-4, 5, (L, Hkv, d), generator=g).float()
    ks = vs = None
    if kind == "bf16":
        k[..., 0] = torch.where(far, -math.inf, 0.0)
        q, k, v, scale = q.bfloat16().cuda(), k.bfloat16().cuda(), v.bfloat16().cuda(), 1.0
        logits = k.double()
    else:
        ks = vs = 1.0
        k[..., 0] = torch.where(far, -256.0, 0.0)
        scale = 2.0 ** 100  # with the scale 256 is beyond any cap; 2 * 2^100 as well
        q, k, v = q.bfloat16().cuda(), k.to(F8).cuda(), v.to(F8).cuda()
        logits = k.float().double()
    o, lse = psa.chunk(q, k, v, psa.plan_chunk([n], [L], Hq, Hkv, d), scale, logit_cap=cap,
                       k_scale=ks, v_scale=vs)
    G = Hq // Hkv
    qq = q.double().unflatten(1, (Hkv, G))
    s = (qq[..., 0, None] * logits[..., 0].T[None, :, None]).nan_to_num(0.0, posinf=1e30, neginf=-1e30)
    s = (s + qq[..., 1, None] * logits[..., 1].T[None, :, None]) * scale  # [n, Hkv, G, L]
    s = cap * torch.tanh(s / cap)
    s = s.masked_fill(~see_of(n, L)[:, None, None], -math.inf)
    rl = torch.logsumexp(s, -1)
    p = torch.exp(s - rl[..., None])
    vv = v.float().double()
    ro = torch.einsum("nhgl,lhd->nhgd", p, vv).flatten(1, 2)
    A = torch.einsum("nhgl,lhd->nhgd", p, vv.abs()).flatten(1, 2)
    e = 24 * U * cap + 2.0 ** -20
    assert torch.isfinite(lse).all() and torch.isfinite(o.float()).all()
    assert float((lse.double() - rl.flatten(1)).abs().max()) <= e
    tol = (2.0 ** -8 + 2 * e) * A + 2.0 ** -8 * ro.abs() + 1e-30
    assert float(((o.double() - ro).abs() - tol).max()) <= 0


@pytest.mark.parametrize("cap", [1000.0, 50.0])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_error_of_the_capped_logit(cap, kind):
    """Logits that are exact in fp32 (one product each), strongly negative and
    positive ones mixed, at the largest cap: what is left is the error of c
    tanh(s / c).  Four reciprocals come from one: with U half a step, 1 / (1 + e)
    carries 7 U (the sum, three products, two for the reciprocal, two more
    products less one that cancels), the exponential's 4 U and the 4 U of its
    argument's factors count a quarter of it; all that twice the cap, and the
    products with c, the offset and the last sum add 6 U of the cap: 24 U c.  The
    log-sum-exp is rounded as a partial's, as the row's and in the change of base."""
    Hq, Hkv, d, n, L = 4, 2, 64, 40, 1000
    g = torch.Generator().manual_seed(int(cap))
    q = torch.zeros(n, Hq, d, dtype=torch.bfloat16)
    q[..., 0] = torch.randint(64, 96, (n, Hq), generator=g).bfloat16()
    pick = torch.tensor([-12.0, -3.0, -0.125, 0.0, 0.25, 10.0, 11.0, 12.0])
    k = torch.zeros(L, Hkv, d)
    k[..., 0] = pick[torch.randint(0, 8, (L, Hkv), generator=g)]
    v = torch.randint(-8, 9, (L, Hkv, d), generator=g).float()
    scale = cap / 256.0  # 96 * 12 / 256: up to 4.5 caps
    ks = vs = None
    if kind == "e4m3":
        ks = vs = 1.0
        k, v = k.to(F8).cuda(), v.to(F8).cuda()
    else:
        k, v = k.bfloat16().cuda(), v.bfloat16().cuda()
    q = q.cuda()
    o, lse = psa.chunk(q, k, v, psa.plan_chunk([n], [L], Hq, Hkv, d), scale, logit_cap=cap,
                       k_scale=ks, v_scale=vs)
    ro, rl, A, _ = reference(q, values(k, ks), values(v, vs), [n], [L], None, scale, 0, cap)
    e = 24 * U * cap + 4 * U * rl.abs()
    assert float(((lse.double() - rl).abs() - e).max()) <= 0
    h = 2.0 ** -11 if ks else 2.0 ** -8
    tol = (h + 2 * e[..., None]) * A + 2.0 ** -8 * ro.abs()
    assert float(((o.double() - ro).abs() - tol).max()) <= 0
