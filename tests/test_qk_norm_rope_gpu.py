"""Norm and rotation of query and key heads, its gradients, the cache append
and the cache read on the GPU, against the formulas in 64 bits.

Tolerances.  U = 2^-24 is half a step of fp32 (relative).  A row's mean of
squares is a sum of d fp32 products (8 in a lane, then log2(d / 8) shuffles):
relative error <= 13 U, and r = rsqrt of it <= 9 U with the function's own
error; x r w and the pair's products and sum add 5 U of |a| + |b|.  So before
the final rounding an element is off by at most 16 U (|a| + |b|) = 2^-20 (|a|
+ |b|), (a, b) the normed pair; the store rounds by at most half a step."""
import numpy as np
import pytest
import torch

import shared_prefix_attention_b200 as psa

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F8 = torch.float8_e4m3fn
EPS = 1e-6


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def angles(npos, rot, gen):
    a = torch.rand(npos, rot // 2, generator=gen, dtype=torch.float64) * 6.28
    return torch.cat([a.cos(), a.sin()], 1).float().cuda()


def split_pairs(y, rot, inter):
    """(a, b, rest) of the rotated elements."""
    head = y[..., :rot]
    if inter:
        return head[..., 0::2], head[..., 1::2], y[..., rot:]
    return head[..., :rot // 2], head[..., rot // 2:], y[..., rot:]


def join_pairs(a, b, rest, inter):
    head = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return torch.cat([head, rest], -1)


def forward64(x, w, cs, pos, inter):
    """(result, bound on |a| + |b| of every element's pair) in 64 bits."""
    y = x.double()
    if w is not None:
        y = y / (y.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * w.double()
    if cs is None:
        return y, y.abs().detach()
    rot = cs.shape[1]
    t = cs.double()[pos.long()][:, None]
    c, s = t[..., :rot // 2], t[..., rot // 2:]
    a, b, rest = split_pairs(y, rot, inter)
    m = (a.abs() + b.abs()).detach()
    return (join_pairs(a * c - b * s, a * s + b * c, rest, inter),
            join_pairs(m, m, rest.abs().detach(), inter))


def check(got, ref, mag, dtype, what):
    tol = half_step(dtype) * (ref.abs() + 16 * U * mag) + 16 * U * mag
    bad = (got.double() - ref).abs() - tol
    assert torch.isfinite(got.float()).all(), what
    assert float(bad.max()) <= 0, f"{what}: over the bound by {float(bad.max()):.3e}"


def make(T, Hq, Hkv, d, dtype, seed, strided=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, (Hq + 2 * Hkv) * d + 16, generator=g).to(dtype).cuda()
    if not strided:
        return (g, *(torch.randn(T, h, d, generator=g).to(dtype).cuda() for h in (Hq, Hkv, Hkv)))
    q = x[:, :Hq * d].unflatten(1, (Hq, d))
    k = x[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
    v = x[:, (Hq + Hkv) * d:(Hq + 2 * Hkv) * d].unflatten(1, (Hkv, d))
    return g, q, k, v


def weight(g, d, dtype=torch.float32):
    return (1 + 0.2 * torch.randn(d, generator=g)).to(dtype).cuda()


CASES = [
    # T, Hq, Hkv, d, rot, interleaved, dtype, weight dtype, strided
    (1, 4, 1, 64, 64, False, torch.bfloat16, torch.float32, True),
    (7, 32, 8, 128, 128, False, torch.bfloat16, torch.bfloat16, True),
    (300, 5, 1, 128, 64, True, torch.bfloat16, torch.float32, False),
    (129, 28, 4, 64, 32, False, torch.float32, torch.float32, True),
    (2500, 3, 3, 128, 16, True, torch.float32, torch.bfloat16, False),
    (33, 6, 2, 256, 256, False, torch.bfloat16, torch.float32, True),
    (65, 2, 2, 256, 48, True, torch.float32, torch.float32, True),
    (5000, 16, 16, 64, 64, True, torch.bfloat16, torch.float32, True),
]


@pytest.mark.parametrize("T,Hq,Hkv,d,rot,inter,dtype,wdt,strided", CASES)
def test_forward(T, Hq, Hkv, d, rot, inter, dtype, wdt, strided):
    g, q, k, _ = make(T, Hq, Hkv, d, dtype, T + d, strided)
    qw, kw = weight(g, d, wdt), weight(g, d, wdt)
    cs = angles(57, rot, g)
    pos = torch.randint(0, 57, (T,), generator=g).int().cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    yq, yk = psa.qk_norm_rope(q, k, pos, cs, qw, kw, EPS, inter, status=st)
    assert psa.read_status(st) == 0
    for got, x, w in ((yq, q, qw), (yk, k, kw)):
        ref, mag = forward64(x, w, cs, pos, inter)
        check(got, ref, mag, dtype, f"T={T} d={d}")


@pytest.mark.parametrize("norm,rope", [(True, False), (False, True), (False, False)])
def test_forward_parts(norm, rope):
    """Only the norm, only the rotation, neither (a copy); one weight missing."""
    g, q, k, _ = make(40, 8, 2, 128, torch.bfloat16, 3)
    qw = weight(g, 128) if norm else None
    cs = angles(9, 128, g) if rope else None
    pos = torch.randint(0, 9, (40,), generator=g).int().cuda() if rope else None
    yq, yk = psa.qk_norm_rope(q, k, pos, cs, q_weight=qw, eps=EPS)
    for got, x, w in ((yq, q, qw), (yk, k, None)):
        ref, mag = forward64(x, w, cs, pos, False)
        check(got, ref, mag, torch.bfloat16, f"norm={norm} rope={rope}")
    if not norm and not rope:
        assert torch.equal(yq, q) and torch.equal(yk, k)


def test_forward_in_place_and_non_finite():
    """Dense tensors may be their own outputs; an infinity behind the rotated
    part stays itself and spoils no other element without a norm."""
    g, q, k, _ = make(50, 4, 4, 64, torch.bfloat16, 4, strided=False)
    cs, pos = angles(50, 32, g), torch.arange(50).int().cuda()
    q[3, 1, 60] = float("inf")
    want = psa.qk_norm_rope(q, k, pos, cs)
    assert torch.isinf(want[0][3, 1, 60]) and int(torch.isfinite(want[0]).logical_not().sum()) == 1
    got = psa.qk_norm_rope(q, k, pos, cs, q_out=q, k_out=k)
    assert torch.equal(got[0], want[0]) and got[0].data_ptr() == q.data_ptr()
    assert torch.equal(got[1], want[1])


def test_zero_rows_and_zero_tokens():
    g, q, k, _ = make(10, 4, 2, 128, torch.bfloat16, 5)
    q, k = q.clone(), k.clone()
    q[4], k[2, 1] = 0, 0
    w = weight(g, 128)
    yq, yk = psa.qk_norm_rope(q, k, None, None, w, w, EPS)
    assert not yq[4].any() and not yk[2, 1].any()
    dq, dk, dqw, dkw = psa.qk_norm_rope_bwd(q, k, torch.ones_like(q), torch.ones_like(k), None,
                                            None, w, w, EPS)
    for t in (dq, dk, dqw, dkw):
        assert torch.isfinite(t.float()).all()
    e = torch.empty(0, 4, 128, dtype=torch.bfloat16, device="cuda")
    yq, yk = psa.qk_norm_rope(e, e, None, None, w, w)
    assert yq.shape == (0, 4, 128)
    out = psa.qk_norm_rope_bwd(e, e, e, e, None, None, w, w)
    assert not out[2].any() and not out[3].any()  # sums over nothing
    cs, none = angles(4, 128, g), torch.empty(0, dtype=torch.int32, device="cuda")
    assert psa.qk_norm_rope(e, e, none, cs, w, w)[0].shape == (0, 4, 128)
    c = torch.zeros(3, 4, 128, dtype=torch.bfloat16, device="cuda")
    assert psa.cache_append(e, e, e, c, c.clone(), none, none, cs, w, w).shape == (0, 4, 128)
    with pytest.raises(ValueError):
        psa.qk_norm_rope(q, k, torch.zeros(10, dtype=torch.int32, device="cuda"), cs[:0])


def test_bad_position_is_reported_and_skipped():
    g, q, k, _ = make(6, 2, 2, 64, torch.bfloat16, 6)
    cs = angles(8, 64, g)
    for bad in (-1, 8):
        pos = torch.tensor([0, 1, bad, 3, 4, 7], dtype=torch.int32, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        yq = torch.full((6, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        yk = yq.clone()
        psa.qk_norm_rope(q, k, pos, cs, q_out=yq, k_out=yk, status=st)
        assert psa.read_status(st) == psa.PSA_ERR_INVALID_ARG
        assert (yq[2] == 7).all() and (yk[2] == 7).all()
        ref, mag = forward64(q, None, cs, pos.clamp(0, 7), False)
        keep = [0, 1, 3, 4, 5]
        check(yq[keep], ref[keep], mag[keep], torch.bfloat16, "others")


def bwd64(x, dy, w, cs, pos, inter):
    """(dx, dw, bound of dx's terms, bound of dw's sum) by autograd in 64 bits."""
    xx = x.double().requires_grad_()
    ww = w.double().requires_grad_() if w is not None else None
    y, _ = forward64(xx, ww, cs, pos, inter)
    grads = torch.autograd.grad(y, (xx, ww) if w is not None else (xx,), dy.double())
    # magnitudes: |g| of the turned-back gradient is at most |a| + |b|
    dyd = dy.double()
    if cs is not None:
        a, b, rest = split_pairs(dyd, cs.shape[1], inter)
        m = a.abs() + b.abs()
        gm = join_pairs(m, m, rest.abs(), inter)
    else:
        gm = dyd.abs()
    if w is None:
        return grads[0], None, gm, None
    xd = x.double()
    r = (xd.pow(2).mean(-1, keepdim=True) + EPS).rsqrt()
    wg = w.double().abs() * gm
    terms = r * (wg + xd.abs() * r * r * (wg * xd.abs()).mean(-1, keepdim=True))
    return grads[0], grads[1], terms, (gm * xd.abs() * r).sum((0, 1))


@pytest.mark.parametrize("T,Hq,Hkv,d,rot,inter,dtype,wdt,strided", CASES)
def test_backward(T, Hq, Hkv, d, rot, inter, dtype, wdt, strided):
    """dx: the two terms carry the norm's 13 + 9 U three times over and the
    mean of d products another 13 U: 64 U of their magnitudes bounds it.  dw:
    every addend is off by at most 32 U of its magnitude and takes part in at
    most (rows / 8 + 128) fp32 additions (a lane's own rows, then lanes,
    warps and blocks)."""
    g, q, k, _ = make(T, Hq, Hkv, d, dtype, T + d, strided)
    qw, kw = weight(g, d, wdt), weight(g, d, wdt)
    cs = angles(57, rot, g)
    pos = torch.randint(0, 57, (T,), generator=g).int().cuda()
    dyq = torch.randn(T, Hq, d, generator=g).to(dtype).cuda()
    dyk = torch.randn(T, Hkv, d, generator=g).to(dtype).cuda()
    # dq, dk as slices of one gradient tensor
    buf = torch.full((T, (Hq + Hkv) * d + 8), 7.0, dtype=dtype, device="cuda")
    dq = buf[:, :Hq * d].unflatten(1, (Hq, d))
    dk = buf[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = psa.qk_norm_rope_bwd(q, k, dyq, dyk, pos, cs, qw, kw, EPS, inter, dq=dq, dk=dk,
                               status=st)
    assert psa.read_status(st) == 0
    assert (buf[:, (Hq + Hkv) * d:] == 7).all()
    for x, dy, w, dx, dw in ((q, dyq, qw, out[0], out[2]), (k, dyk, kw, out[1], out[3])):
        rx, rw, terms, wsum = bwd64(x, dy, w, cs, pos, inter)
        tol = half_step(dtype) * (rx.abs() + 64 * U * terms) + 64 * U * terms
        assert float(((dx.double() - rx).abs() - tol).max()) <= 0
        tol = (32 + T * x.shape[1] / 8 + 128) * U * wsum
        assert float(((dw.double() - rw).abs() - tol).max()) <= 0
    again = psa.qk_norm_rope_bwd(q, k, dyq, dyk, pos, cs, qw, kw, EPS, inter)
    for a, b in zip(out, again):
        assert torch.equal(a, b)  # a fixed order of every sum


@pytest.mark.parametrize("Hq,Hkv,d,inter", [(9, 1, 128, False), (2, 3, 64, True)])
def test_backward_of_many_tokens(Hq, Hkv, d, inter):
    """Enough tokens that every warp takes whole ones."""
    test_backward(40001, Hq, Hkv, d, d, inter, torch.bfloat16, torch.float32, True)


@pytest.mark.parametrize("captured", [False, True])
def test_backwards_in_a_row_share_a_workspace(captured):
    """The sum over a call's partial weight gradients against the next call,
    which writes its own partials to the same place."""
    calls = []
    ws = torch.empty(296 * 128 * 4, dtype=torch.uint8, device="cuda")
    for i in range(6):
        g, q, k, _ = make(700, 8, 2, 128, torch.bfloat16, 100 + i)
        calls.append((q, k, torch.randn_like(q.contiguous()), torch.randn_like(k.contiguous()),
                      torch.arange(700, device="cuda").int(), angles(700, 128, g),
                      weight(g, 128), weight(g, 128)))

    def run():
        return [psa.qk_norm_rope_bwd(*c, EPS, False, workspace=ws) for c in calls]

    if captured:
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run()
        ws.fill_(0xff)
        for _ in range(3):
            graph.replay()
    else:
        got = run()
    for c, a in zip(calls, got):
        torch.cuda.synchronize()
        for x, y in zip(a, psa.qk_norm_rope_bwd(*c, EPS, False)):
            assert torch.equal(x, y)


def test_backward_against_differences():
    """Central differences of the forward kernel itself, fp32: a step h moves
    <y, dy> by h dx + O(h^3); with |values| ~ 1 and sums of 2 * 64 terms the
    forward's fp32 error over 2 h is at most 128 * 4 U / h."""
    g, q, k, _ = make(3, 1, 1, 64, torch.float32, 9, strided=False)
    qw, kw = weight(g, 64), weight(g, 64)
    cs, pos = angles(3, 32, g), torch.arange(3).int().cuda()
    dyq, dyk = torch.randn(3, 1, 64, generator=g).cuda(), torch.randn(3, 1, 64, generator=g).cuda()

    def loss(q, k, qw, kw):
        yq, yk = psa.qk_norm_rope(q, k, pos, cs, qw, kw, EPS)
        return float((yq.double() * dyq.double()).sum() + (yk.double() * dyk.double()).sum())

    grads = psa.qk_norm_rope_bwd(q, k, dyq, dyk, pos, cs, qw, kw, EPS)
    h = 2.0 ** -8
    args = [q, k, qw, kw]
    for i, gr in enumerate(grads):
        flat = gr.flatten()
        for j in range(0, flat.numel(), 5):
            hi, lo = args[i].clone(), args[i].clone()
            hi.view(-1)[j] += h
            lo.view(-1)[j] -= h
            d = (loss(*args[:i], hi, *args[i + 1:]) - loss(*args[:i], lo, *args[i + 1:])) / (2 * h)
            # third derivative of x / rms(x): at most ~8 |dy| |w| per element
            assert abs(d - float(flat[j])) <= 128 * 4 * U / h + 8 * h * h + 1e-6, (i, j)


# ------------------------------------------------------------------ cache append and read

def as_cache(x, kind):
    return x.to(torch.bfloat16) if kind == "bf16" else x.clamp(-448, 448).to(F8)


@pytest.mark.parametrize("T,Hq,Hkv,d,rot,inter,kind", [
    (1, 4, 1, 128, 128, False, "e4m3"),
    (32, 32, 8, 128, 64, True, "bf16"),
    (300, 28, 4, 64, 64, False, "e4m3"),
    (77, 5, 1, 256, 128, False, "bf16"),
    (1500, 8, 8, 128, 128, True, "e4m3"),
])
def test_append(T, Hq, Hkv, d, rot, inter, kind):
    g, q, k, v = make(T, Hq, Hkv, d, torch.bfloat16, T, strided=True)
    ntok = T + 100
    kc = as_cache(torch.randn(ntok, Hkv, d, generator=g), kind).cuda()
    vc = as_cache(torch.randn(ntok, Hkv, d, generator=g), kind).cuda()
    slots = torch.randperm(ntok, generator=g)[:T].int()
    pad = T // 7
    slots[T - pad:] = -1
    slots = slots.cuda()
    qw, kw = weight(g, d), weight(g, d)
    cs = angles(64, rot, g)
    pos = torch.randint(0, 64, (T,), generator=g).int().cuda()
    ks, vs = (0.021, 0.0046) if kind == "e4m3" else (None, None)
    k0, v0 = kc.view(torch.uint8).clone(), vc.view(torch.uint8).clone()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    yq = psa.cache_append(q, k, v, kc, vc, slots, pos, cs, qw, kw, EPS, inter, ks, vs, status=st)
    assert psa.read_status(st) == 0
    ref, mag = forward64(q, qw, cs, pos, inter)
    check(yq, ref, mag, torch.bfloat16, "queries")  # padded tokens' queries too
    live = slots >= 0
    at = slots[live].long()
    untouched = torch.ones(ntok, dtype=torch.bool, device="cuda")
    untouched[at] = False
    assert torch.equal(kc.view(torch.uint8)[untouched], k0[untouched])
    assert torch.equal(vc.view(torch.uint8)[untouched], v0[untouched])
    kref, kmag = forward64(k, kw, cs, pos, inter)
    for c, ref, mag, s in ((kc, kref, kmag, ks), (vc, v.double(), v.double().abs() * 0, vs)):
        ref, mag = ref[live], mag[live]
        if kind == "bf16":
            check(c[at], ref, mag, torch.bfloat16, "cache")
            continue
        got = c.view(torch.uint8)[at].view(F8).double()
        want = (ref / s).clamp(-448, 448)
        off = (16 * mag / s + 2 * want.abs()) * U  # the row's error and the division's
        step = torch.maximum(2.0 ** -4 * (want.abs() + off), torch.full_like(want, 2.0 ** -10))
        assert float(((got - want).abs() - step - off).max()) <= 0


def test_append_without_queries_or_norm_copies():
    g, q, k, v = make(20, 4, 2, 128, torch.bfloat16, 12)
    kc = torch.zeros(30, 2, 128, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    slots = torch.randperm(30, generator=g)[:20].int().cuda()
    assert psa.cache_append(None, k, v, kc, vc, slots) is None
    assert torch.equal(kc[slots.long()], k) and torch.equal(vc[slots.long()], v)


def test_append_saturates_and_keeps_nan():
    k = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    k[0, 0, :5] = torch.tensor([1e4, -1e4, float("inf"), float("nan"), 1.0])
    kc = torch.zeros(2, 1, 64, dtype=torch.uint8, device="cuda").view(F8)
    vc = kc.clone()
    psa.cache_append(None, k, k, kc, vc, torch.ones(1, dtype=torch.int32, device="cuda"),
                     k_scale=1.0, v_scale=0.5)
    got = kc[1, 0, :5].float().cpu()
    assert got[0] == 448 and got[1] == -448 and got[2] == 448 and torch.isnan(got[3])
    assert got[4] == 1 and vc[1, 0, 4].float() == 2
    assert not kc[0].view(torch.uint8).any()


def test_append_bad_slot_is_reported_and_skipped():
    g, q, k, v = make(3, 2, 2, 64, torch.bfloat16, 13)
    buf = torch.zeros(12, 2, 64, dtype=torch.bfloat16, device="cuda")
    kc, vc = buf[2:6], torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    yq = psa.cache_append(q, k, v, kc, vc,
                          torch.tensor([1, 4, 3], dtype=torch.int32, device="cuda"), status=st)
    assert psa.read_status(st) == psa.PSA_ERR_INVALID_ARG
    assert torch.equal(kc[1], k[0]) and torch.equal(kc[3], k[2]) and not kc[0].any()
    assert not buf[6:].any() and not buf[:2].any() and torch.equal(yq, q)


@pytest.mark.parametrize("n,Hkv,d,kind", [(1, 1, 64, "bf16"), (300, 8, 128, "e4m3"),
                                          (4097, 3, 256, "e4m3"), (999, 4, 64, "bf16")])
def test_read(n, Hkv, d, kind):
    g = torch.Generator().manual_seed(n)
    ntok = n + 50
    kc = as_cache(torch.randn(ntok, Hkv, d, generator=g) * 3, kind).cuda()
    vc = as_cache(torch.randn(ntok, Hkv, d, generator=g) * 3, kind).cuda()
    rows = torch.randint(0, ntok, (n,), generator=g).int().cuda()  # repeats allowed
    ks, vs = (0.021, 3.7) if kind == "e4m3" else (None, None)
    k, v = psa.cache_read(kc, vc, rows, ks, vs)
    for got, c, s in ((k, kc, ks), (v, vc, vs)):
        if kind == "bf16":
            assert torch.equal(got, c[rows.long()])
        else:
            # one fp32 product, rounded to bf16: the scale as fp32
            ref = c.view(torch.uint8)[rows.long()].view(F8).double() * float(np.float32(s))
            assert float(((got.double() - ref).abs() - (2.0 ** -8 + U * 2) * ref.abs()).max()) <= 0


def test_read_bad_rows_and_empty():
    kc = torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = psa.cache_read(kc, kc, torch.tensor([0, -1, 4, 3], dtype=torch.int32, device="cuda"),
                          status=st)
    assert psa.read_status(st) == psa.PSA_ERR_INVALID_ARG
    assert k[0].all() and k[3].all() and not k[1:3].any() and not v[1:3].any()
    k, v = psa.cache_read(kc, kc, torch.empty(0, dtype=torch.int32, device="cuda"))
    assert k.shape == (0, 2, 64)


def test_append_then_read_through_a_graph_on_another_stream():
    """Captured, replayed with new inputs, on a stream of its own."""
    g, q, k, v = make(64, 8, 2, 128, torch.bfloat16, 15)
    kc = torch.zeros(100, 2, 128, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    slots = torch.randperm(100, generator=g)[:64].int().cuda()
    cs, pos = angles(64, 128, g), torch.arange(64).int().cuda()
    w = weight(g, 128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        psa.cache_append(q, k, v, kc, vc, slots, pos, cs, w, w, EPS)
        with torch.cuda.graph(graph, stream=s):
            yq = psa.cache_append(q, k, v, kc, vc, slots, pos, cs, w, w, EPS)
            kk, vv = psa.cache_read(kc, vc, slots)
    torch.cuda.current_stream().wait_stream(s)
    q.mul_(-0.5)
    k.mul_(2.0).add_(0.25)
    v.neg_()
    graph.replay()
    want_q, want_k = psa.qk_norm_rope(q, k, pos, cs, w, w, EPS)
    torch.cuda.synchronize()
    assert torch.equal(yq, want_q) and torch.equal(kk, want_k) and torch.equal(vv, v)


@pytest.mark.parametrize("T,Hq,Hkv,d,dtype", [
    (7, 5, 1, 128, torch.bfloat16),
    (9, 2, 2, 128, torch.bfloat16),
    (40, 9, 3, 64, torch.bfloat16),
    (6, 3, 1, 256, torch.bfloat16),
    (5, 3, 1, 256, torch.float32),
    (11, 5, 2, 64, torch.float32),
    (40001, 9, 1, 128, torch.bfloat16),
])
def test_backward_without_eps(T, Hq, Hkv, d, dtype, monkeypatch):
    """eps = 0 is a norm like any other where no row is zero, also where a
    token's heads do not fill a warp's last group of rows."""
    monkeypatch.setitem(globals(), "EPS", 0.0)
    test_backward(T, Hq, Hkv, d, d, False, dtype, torch.float32, True)
