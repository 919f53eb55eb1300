"""The operators of a layer run together, as they are used: a prompt cached and
attended piece by piece, then decoded; a training step from the projection's
output to its gradient.  Compared with the formulas in 64 bits; the bounds add
up those of the single steps (each says its own in its test)."""
import pytest
import torch

import shared_prefix_attention_b200 as psa
from test_chunk_gpu import F8, reference, values
from test_qk_norm_rope_gpu import EPS, forward64, weight

pytestmark = pytest.mark.gpu


def angles(npos, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(npos, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().cuda()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_serving(kind):
    """Two requests: prompts in pieces of 100 tokens into a paged cache, then
    three decoding steps, each step one append and one chunk call.  The rows
    that chunk sees are the cache's own, so it has chunk's own bound, and every
    cached row is read back as it was written."""
    Hq, Hkv, d, lens, piece, steps = 8, 2, 128, [250, 37], 100, 3
    g = torch.Generator().manual_seed(21)
    ks, vs = (0.021, 0.017) if kind == "e4m3" else (None, None)
    ntok = 400
    k = torch.zeros(ntok, Hkv, d, dtype=torch.bfloat16, device="cuda")
    if kind == "e4m3":
        k = k.to(F8)
    v = k.clone()
    pages = torch.randperm(ntok, generator=g).int().cuda()
    row = [pages[:270], pages[270:]]
    cs = angles(300, d)
    qw, kw = weight(g, d), weight(g, d)
    total = [n + steps for n in lens]
    x = [torch.randn(n, (Hq + 2 * Hkv) * d, generator=g).bfloat16().cuda() for n in total]
    done = [0, 0]
    h = 2.0 ** -11 if ks else 2.0 ** -8
    while done != total:
        new = [min(piece, n - a) if a < n else (1 if a < t else 0)
               for a, n, t in zip(done, lens, total)]
        xs = torch.cat([x[b][done[b]:done[b] + new[b]] for b in range(2)])
        pos = torch.cat([torch.arange(done[b], done[b] + new[b]) for b in range(2)]).int().cuda()
        slots = torch.cat([row[b][done[b]:done[b] + new[b]] for b in range(2)])
        q = xs[:, :Hq * d].unflatten(1, (Hq, d))
        kn = xs[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
        vn = xs[:, (Hq + Hkv) * d:].unflatten(1, (Hkv, d))
        qr = psa.cache_append(q, kn, vn, k, v, slots, pos, cs, qw, kw, EPS, k_scale=ks,
                              v_scale=vs)
        done = [a + n for a, n in zip(done, new)]
        table = torch.cat([row[b][:done[b]] for b in range(2)])
        plan = psa.plan_chunk(new, done, Hq, Hkv, d)
        o, lse = psa.chunk(qr, k, v, plan, d ** -0.5, kv_indices=table, k_scale=ks, v_scale=vs)
        ro, rl, A, S = reference(qr, values(k, ks), values(v, vs), new, done, table, d ** -0.5, 0,
                                 0.0)
        e = (d + 16) * 2.0 ** -23 * (S + 1)
        assert float(((lse.double() - rl).abs() - e).max()) <= 0
        tol = h * A + 2.0 ** -8 * ro.abs() + 2 * e[..., None] * A
        assert float(((o.double() - ro).abs() - tol).max()) <= 0
    kk, vv = psa.cache_read(k, v, row[0][:total[0]], ks, vs)
    kn = x[0][:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
    vn = x[0][:, (Hq + Hkv) * d:].unflatten(1, (Hkv, d))
    pos = torch.arange(total[0], device="cuda")
    kref, mag = forward64(kn, kw, cs, pos, False)
    # half a step of the cache's type, half a step of bf16 on the way back, and
    # the row's own fp32 error
    step = 2.0 ** -4 if ks else 2.0 ** -8
    low = (2.0 ** -10 if ks else 0.0)
    for got, ref, s, m in ((kk, kref, ks, mag), (vv, vn.double(), vs, vn.double().abs())):
        tol = (step + 2.0 ** -8) * 1.01 * ref.abs() + low * (s or 0.0) + 2.0 ** -19 * m
        assert float(((got.double() - ref).abs() - tol).max()) <= 0


def test_training_step():
    """qk_norm_rope -> prefill -> its gradients -> gradients of qk_norm_rope,
    against autograd in 64 bits over every [prefix; suffix] row's keys.  Bar:
    the prefill gradients' own (relative Frobenius error 2e-2) for dq, dk, dv
    and for the weights' sums."""
    P, N, S, Hq, Hkv, d = 130, 3, 70, 4, 2, 64
    T = P + N * S
    g = torch.Generator().manual_seed(31)
    x = torch.randn(T, (Hq + 2 * Hkv) * d, generator=g).bfloat16().cuda()
    q = x[:, :Hq * d].unflatten(1, (Hq, d))
    k = x[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
    v = x[:, (Hq + Hkv) * d:].unflatten(1, (Hkv, d)).contiguous()
    do = torch.randn(T, Hq, d, generator=g).bfloat16().cuda()
    pos = torch.cat([torch.arange(P), torch.arange(P, P + S).repeat(N)]).int().cuda()
    cs, qw, kw = angles(P + S, d), weight(g, d), weight(g, d)
    segs = psa.spec_flat(P, N, S)
    scale = d ** -0.5

    qr, kr = psa.qk_norm_rope(q, k, pos, cs, qw, kw, EPS)
    o, lse = psa.prefill(qr, kr, v, psa.plan_prefill(segs, [0, T], d), scale)
    dqr, dkr, dv = psa.prefill_bwd(qr, kr, v, o, lse, do, psa.plan_prefill_bwd(segs, [0, T], d),
                                   scale)
    dx = torch.zeros_like(x)
    dq = dx[:, :Hq * d].unflatten(1, (Hq, d))
    dk = dx[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
    _, _, dqw, dkw = psa.qk_norm_rope_bwd(q, k, dqr, dkr, pos, cs, qw, kw, EPS, dq=dq, dk=dk)

    leaves = [t.double().requires_grad_() for t in (q, k, v, qw, kw)]
    q64, k64, v64, qw64, kw64 = leaves
    yq, _ = forward64(q64, qw64, cs, pos, False)
    yk, _ = forward64(k64, kw64, cs, pos, False)
    at = torch.arange(T, device="cuda")
    seg = torch.where(at < P, 0, 1 + (at - P) // S)
    see = (at[:, None] >= at) & ((seg[:, None] == seg) | (at < P))
    s = torch.einsum("nhgd,lhd->hgnl", yq.unflatten(1, (Hkv, Hq // Hkv)), yk) * scale
    p = torch.softmax(s.masked_fill(~see, -float("inf")), -1)
    ref = torch.einsum("hgnl,lhd->nhgd", p, v64).flatten(1, 2)
    want = torch.autograd.grad(ref, leaves, do.double())
    for name, got, r in zip(("dq", "dk", "dv", "dqw", "dkw"), (dq, dk, dv, dqw, dkw), want):
        err = float((got.double() - r).norm() / r.norm())
        assert err <= 2e-2, f"{name}: {err:.3e}"
