"""Chunk attention where the softmax weights are hard to hold: one key far above
many small ones."""
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
