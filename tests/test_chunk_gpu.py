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


def small(seed=1, ql=(100, 3), kl=(700, 300), Hq=8, Hkv=2, d=128, paged=True, kind="bf16", **kw):
    ql, kl = list(ql), list(kl)
    q, k, v, ks, vs, table = make(ql, kl, Hq, Hkv, d, paged, kind, seed, **kw)
    return ql, kl, q, k, v, ks, vs, table, psa.plan_chunk(ql, kl, Hq, Hkv, d)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_bad_pages_read_as_zeros_and_are_reported(kind):
    """Entries outside the cache (a hole, an index behind the end) in a whole
    tile and in the last, partial one."""
    ql, kl, q, k, v, ks, vs, table, plan = small(kind=kind)
    bad = table.clone()
    bad[[5, 640, 699, 700, 999]] = torch.tensor([-1, k.shape[0], -2**31, 2**31 - 1, -7],
                                                dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = psa.chunk(q, k, v, plan, 0.1, kv_indices=bad, k_scale=ks, v_scale=vs, status=st)
    assert psa.read_status(st) == psa.PSA_ERR_INVALID_ARG
    kz = torch.cat([values(k, ks), torch.zeros_like(values(k[:1], ks))])
    vz = torch.cat([values(v, vs), torch.zeros_like(values(v[:1], vs))])
    at = torch.where((bad < 0) | (bad >= k.shape[0]), k.shape[0], bad)
    ref = reference(q, kz, vz, ql, kl, at, 0.1, 0, 0.0)
    check(o, lse, ref, 128, 0.0, 2.0 ** -11 if ks else 2.0 ** -8, "bad pages")
    # without a status word nothing else changes
    o2, _ = psa.chunk(q, k, v, plan, 0.1, kv_indices=bad, k_scale=ks, v_scale=vs)
    assert torch.equal(o, o2)


def test_rows_behind_the_last_sequence_are_left_alone():
    ql, kl, q, k, v, _, _, table, plan = small()
    qq = torch.cat([q, torch.full((9, 8, 128), float("nan"), dtype=q.dtype, device="cuda")])
    o = torch.full_like(qq, 7.0)
    lse = torch.full(qq.shape[:2], 7.0, device="cuda")
    psa.chunk(qq, k, v, plan, 0.1, kv_indices=table, out=o, lse=lse)
    want, wl = psa.chunk(q, k, v, plan, 0.1, kv_indices=table)
    assert torch.equal(o[:-9], want) and torch.equal(lse[:-9], wl)
    assert (o[-9:] == 7).all() and (lse[-9:] == 7).all()


@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_nan_key_reaches_the_rows_that_see_it_and_no_other(cap):
    ql, kl, q, k, v, _, _, table, plan = small(ql=(300,), kl=(500,))
    o, lse = psa.chunk(q, k, v, plan, 0.1, kv_indices=table, logit_cap=cap)
    k[int(table[420])] = float("nan")
    on, ln = psa.chunk(q, k, v, plan, 0.1, kv_indices=table, logit_cap=cap)
    assert torch.equal(on[:220], o[:220]) and torch.equal(ln[:220], lse[:220])
    assert torch.isnan(on[220:].float()).all() and torch.isnan(ln[220:]).all()


def test_lowest_logits_and_equal_keys():
    """Logits far below zero, and rows whose keys are all alike (the mean)."""
    ql, kl, q, k, v, _, _, table, plan = small()
    k[:] = -100.0
    q[:] = 100.0
    o, lse = psa.chunk(q, k, v, plan, 1.0, kv_indices=table)
    ref = reference(q, k.double(), v.double(), ql, kl, table, 1.0, 0, 0.0)
    assert torch.isfinite(o.float()).all()
    assert float(((o.double() - ref[0]).abs() - 2.0 ** -7 * ref[2]).max()) <= 0
    # lse = -1.28e6 + log n: a step of fp32 there is 1/8
    assert float((lse.double() - ref[1]).abs().max()) <= 0.5


def test_misaligned_output_and_given_buffers():
    """Outputs on 16-byte (not 32-byte) boundaries, a caller's workspace."""
    ql, kl, q, k, v, _, _, table, plan = small(ql=(300,), kl=(300,), paged=False)
    want, wl = psa.chunk(q, k, v, plan, 0.1)
    buf = torch.zeros(q.numel() + 8, dtype=q.dtype, device="cuda")
    o = buf[8:].view(q.shape)
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    got, gl = psa.chunk(q, k, v, plan, 0.1, out=o, workspace=ws)
    assert got.data_ptr() == o.data_ptr() and torch.equal(o, want) and torch.equal(gl, wl)
    with pytest.raises(psa.PsaError) as e:
        psa.chunk(q, k, v, plan, 0.1, workspace=ws[:plan.workspace_bytes - 1])
    assert e.value.status == psa.PSA_ERR_WORKSPACE


def test_refused_arguments():
    ql, kl, q, k, v, ks, vs, table, plan = small()
    for args in ((q.float(), k, v, plan), (q[:, :4], k, v, plan), (q, k[:, :1], v, plan),
                 (q, k.float(), v, plan), (q, k.transpose(0, 1), v, plan), (q, k, v[:-1], plan)):
        with pytest.raises(ValueError):
            psa.chunk(*args, 0.1, kv_indices=table)
    with pytest.raises(ValueError):
        psa.chunk(q, k, v, plan, 0.1, kv_indices=table[:-1])
    with pytest.raises(ValueError):
        psa.chunk(q, k, v, plan, 0.1, kv_indices=table.long())
    for kw in (dict(logit_cap=-1.0), dict(logit_cap=float("inf"))):
        with pytest.raises(psa.PsaError):
            psa.chunk(q, k, v, plan, 0.1, kv_indices=table, **kw)
    with pytest.raises(psa.PsaError):
        psa.chunk(q, k, v, plan, 0.0, kv_indices=table)
    with pytest.raises(psa.PsaError):
        psa.chunk(q, k[:50], v[:50], plan, 0.1)  # no table, and a cache of too few rows
    with pytest.raises(psa.PsaError):
        psa.chunk(q[:-1], k, v, plan, 0.1, kv_indices=table)


def test_two_graphs_and_an_eager_call_at_once():
    """Two captured calls replayed on two streams and an eager one on a third,
    all in flight together; captured replays see new inputs."""
    sets = [small(seed=s, ql=(200, 64), kl=(3000, 2000)) for s in (1, 2, 3)]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for (ql, kl, q, k, v, _, _, table, plan), s in zip(sets[:2], streams):
        with torch.cuda.stream(s):
            psa.chunk(q, k, v, plan, 0.1, kv_indices=table)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                outs.append(psa.chunk(q, k, v, plan, 0.1, kv_indices=table))
        graphs.append(g)
    torch.cuda.synchronize()
    for x in sets:
        x[2].mul_(-1.5)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            _, _, q, k, v, _, _, table, plan = sets[2]
            eager = psa.chunk(q, k, v, plan, 0.1, kv_indices=table)
    torch.cuda.synchronize()
    for (ql, kl, q, k, v, _, _, table, plan), got in zip(sets, outs + [eager]):
        want = psa.chunk(q, k, v, plan, 0.1, kv_indices=table)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("captured", [False, True])
def test_layers_in_a_row_share_a_workspace(captured):
    """Eight calls, each one's queries the output of the one before, all over
    one workspace whose partials each call's join reads: nothing of a call may
    begin before the call before it is done."""
    ql, kl, q, k, v, _, _, table, plan = small(seed=7, ql=(300, 1, 64), kl=(4000, 900, 64))
    assert plan.info.n_joins > 0
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")

    def layers():
        x, every = q, []
        for i in range(8):
            x, l = psa.chunk(x, k, v, plan, 0.3 + 0.1 * i, kv_indices=table, workspace=ws)
            every += [x, l]
        return every

    if captured:
        layers()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = layers()
        ws.fill_(0xff)
        for _ in range(3):
            g.replay()
    else:
        got = layers()
    x = q
    for i in range(8):
        torch.cuda.synchronize()
        want = psa.chunk(x, k, v, plan, 0.3 + 0.1 * i, kv_indices=table)
        torch.cuda.synchronize()
        assert torch.equal(got[2 * i], want[0]) and torch.equal(got[2 * i + 1], want[1])
        x = want[0]


def test_cache_rows_beyond_32_bit_offsets():
    """Rows whose byte offsets pass 2^32: appended, attended, read back."""
    Hq, Hkv, d, n = 4, 2, 128, 130
    ntok = (1 << 32) // (Hkv * d * 2) + 1000
    g = torch.Generator().manual_seed(5)
    k, v = (torch.empty(ntok, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rows = (ntok - 1 - torch.randperm(900, generator=g)[:n]).int().cuda()
    q = torch.randn(n, Hq, d, generator=g).bfloat16().cuda()
    kn, vn = (torch.randn(n, Hkv, d, generator=g).bfloat16().cuda() for _ in range(2))
    assert torch.equal(psa.cache_append(q, kn, vn, k, v, rows), q)
    kk, vv = psa.cache_read(k, v, rows)
    assert torch.equal(kk, kn) and torch.equal(vv, vn)
    plan = psa.plan_chunk([n], [n], Hq, Hkv, d)
    o, lse = psa.chunk(q, k, v, plan, 0.1, kv_indices=rows)
    want, wl = psa.chunk(q, kn, vn, plan, 0.1)
    assert torch.equal(o, want) and torch.equal(lse, wl)


def test_debug_build_agrees():
    """The bounds-checked library on the same calls, with and without split
    blocks."""
    for kw in (dict(), dict(ql=(3,), kl=(90,)), dict(ql=(9000,), kl=(9000,), Hq=32, Hkv=8)):
        ql, kl, q, k, v, _, _, table, plan = small(**kw)
        want, wl = psa.chunk(q, k, v, plan, 0.1, kv_indices=table)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        with psa.use_library(psa.DEBUG_LIB_PATH):
            got, gl = psa.chunk(q, k, v, plan, 0.1, kv_indices=table, status=st)
            torch.cuda.synchronize()
        assert psa.read_status(st) == 0
        assert torch.equal(got, want) and torch.equal(gl, wl)


def test_agrees_with_the_verify_entry():
    """Draft tokens whose keys are cached already are a chunk: the extend form
    of verify on the cache without them gives the same rows (two kernels, each
    within its own bound)."""
    ql, kl = [4, 2], [900, 130]
    q, k, v, _, _, _ = make(ql, kl, 8, 2, 128, False, "bf16", 9)
    o, lse = psa.chunk(q, k, v, psa.plan_chunk(ql, kl, 8, 2, 128), 0.1)
    new = torch.tensor([896, 897, 898, 899, 1028, 1029], device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.cat([torch.arange(896, **i32), torch.arange(900, 1028, **i32)])
    o2, lse2 = psa.verify_extend(q, k[new], v[new], k, v, torch.tensor([0, 4, 6], **i32), 4,
                                 torch.tensor([0, 896, 1024], **i32), 896, 0.1, kv_indices=table)
    ref = reference(q, k.double(), v.double(), ql, kl, None, 0.1, 0, 0.0)
    tol = 2 * (2.0 ** -8 * ref[2] + 2.0 ** -8 * ref[0].abs()) + 1e-4
    assert float(((o.double() - o2.double()).abs() - tol).max()) <= 0
    assert float((lse - lse2).abs().max()) <= 1e-3
