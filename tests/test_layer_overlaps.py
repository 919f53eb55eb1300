"""Buffers that overlap: what the calls around a layer refuse, on the host, and
the placements in place and side by side that they take."""
import ctypes

import pytest
import torch

import shared_prefix_attention_b200 as psa
from test_chunk_plan import BAD_HOW, _append, _chunk, _how, _info, _read
from test_qk_norm_rope_gpu import EPS, angles, weight

P = ctypes.c_void_p
BAD = psa.PSA_ERR_INVALID_ARG
MB = 1 << 20
T, HQ, HKV, D = 4, 8, 2, 128
QB, KB = T * HQ * D * 2, T * HKV * D * 2  # bytes of dense queries, of dense keys


def _fwd(**kw):
    a = dict(q=MB, qs=HQ * D, k=2 * MB, ks=HKV * D, qo=3 * MB, ko=4 * MB, how=_how())
    a.update(kw)
    return psa.lib().psa_qk_norm_rope_fwd(P(a["q"]), a["qs"], P(a["k"]), a["ks"], psa.PSA_BF16, T,
                                          HQ, HKV, D, ctypes.byref(a["how"]), P(a["qo"]),
                                          P(a["ko"]), None, None)


def _bwd(**kw):
    a = dict(q=MB, qs=HQ * D, k=2 * MB, ks=HKV * D, gq=3 * MB, gk=4 * MB, dq=5 * MB, dqs=HQ * D,
             dk=6 * MB, dks=HKV * D, how=_how())
    a.update(kw)
    return psa.lib().psa_qk_norm_rope_bwd(P(a["q"]), a["qs"], P(a["k"]), a["ks"], P(a["gq"]),
                                          P(a["gk"]), psa.PSA_BF16, T, HQ, HKV, D,
                                          ctypes.byref(a["how"]), P(a["dq"]), a["dqs"],
                                          P(a["dk"]), a["dks"], None, None, P(256), MB, None, None)


def test_norm_and_rotation_refuse_overlaps():
    wide = (HQ + 2 * HKV) * D  # a projection's row
    for kw in (dict(qo=MB + 16), dict(qo=MB + QB - 16), dict(qo=MB - QB + 16), dict(ko=2 * MB + 256),
               dict(qo=2 * MB), dict(ko=MB), dict(ko=3 * MB), dict(ko=3 * MB + QB - 16),
               dict(qs=wide, qo=MB), dict(qs=wide, qo=MB + 2 * HQ * D)):
        assert _fwd(**kw) == BAD, kw
    for kw in (dict(dq=3 * MB + 16), dict(dq=MB + 16), dict(dq=4 * MB), dict(dk=3 * MB),
               dict(dk=5 * MB + QB - 16), dict(dq=MB, dqs=wide), dict(dq=2 * MB),
               # slices of one tensor that run into one another
               dict(dqs=wide, dk=5 * MB + 2 * HQ * D - 16, dks=wide),
               dict(dqs=wide, dk=5 * MB + 2 * (wide - HKV * D) + 16, dks=wide)):
        assert _bwd(**kw) == BAD, kw


def test_cache_rows_refuse_overlaps():
    ok = dict(q=MB, k=2 * MB, v=3 * MB, kc=4 * MB, vc=5 * MB, slots=16, qo=6 * MB)
    row = HKV * D * 2
    for kw in (dict(vc=4 * MB), dict(vc=4 * MB + 7 * row), dict(kc=2 * MB), dict(kc=2 * MB - 7 * row),
               dict(vc=3 * MB + row), dict(kc=MB), dict(vc=6 * MB), dict(qo=MB + 16),
               dict(qo=2 * MB), dict(qo=3 * MB)):
        assert _append(**{**ok, **kw}) == BAD, kw
    # and what is refused whatever the addresses
    for kw in (dict(T=-1), dict(Hkv=0), dict(Hq=0), dict(ntok=-1), dict(ntok=2**31), dict(k=None),
               dict(v=None), dict(kc=None), dict(vc=8), dict(slots=None), dict(slots=2),
               dict(ks=255), dict(vs=0), dict(qo=None), dict(sc=(-1.0, 1.0)), dict(sc=(1.0, 1e-39))):
        assert _append(**{**ok, **kw}) == BAD, kw
    for kw in BAD_HOW:
        assert _append(**ok, how=_how(**kw)) == BAD, kw
    ok = dict(kc=MB, vc=2 * MB, rows=16, k=3 * MB, v=4 * MB)
    for kw in (dict(k=MB), dict(v=2 * MB + 7 * row), dict(k=2 * MB - row), dict(v=3 * MB + row),
               dict(n=-1), dict(Hkv=0), dict(ntok=-1), dict(kc=None), dict(vc=8), dict(rows=None),
               dict(rows=1), dict(k=None), dict(v=8), dict(sc=(1.0, 0.0))):
        assert _read(**{**ok, **kw}) == BAD, kw


def test_attention_refuses_an_output_over_a_cache():
    rows, cache = 300 * 8 * 128 * 2, 2000 * 2 * 128 * 2
    at = dict(q=64 * MB, k=MB, v=8 * MB)
    for o in (MB, 8 * MB + cache - 16, MB - rows + 16):
        assert _chunk(**at, o=o) == BAD, o


def test_attention_refuses_overlaps_of_lse_and_workspace():
    at = dict(q=64 * MB, k=MB, v=8 * MB, o=128 * MB, lse=192 * MB, ws=256 * MB)
    rows, lse, cache = 300 * 8 * 128 * 2, 300 * 8 * 4, 2000 * 2 * 128 * 2
    info = _info()
    need = psa.lib().psa_chunk_workspace_size(ctypes.byref(info))
    assert need > 256
    for kw in (dict(lse=64 * MB), dict(lse=64 * MB + rows - 4), dict(lse=128 * MB), dict(lse=MB + 4),
               dict(lse=128 * MB - lse + 4), dict(lse=8 * MB + cache - 4),
               dict(ws=64 * MB), dict(ws=128 * MB + 256), dict(ws=MB), dict(ws=8 * MB),
               dict(ws=192 * MB), dict(ws=128 * MB - (need - 256)), dict(lse=256 * MB + need - 4)):
        assert _chunk(info=info, **{**at, **kw}) == BAD, kw


def test_gradients_refuse_overlaps_of_weight_gradients_and_workspace():
    at = dict(q=MB, k=2 * MB, gq=3 * MB, gk=4 * MB, dq=5 * MB, dk=6 * MB, dqw=7 * MB, dkw=8 * MB,
              ws=9 * MB)
    need = psa.lib().psa_qk_norm_rope_bwd_workspace_size(D)

    def call(**kw):
        a = {**at, **kw}
        return psa.lib().psa_qk_norm_rope_bwd(
            P(a["q"]), HQ * D, P(a["k"]), HKV * D, P(a["gq"]), P(a["gk"]), psa.PSA_BF16, T, HQ, HKV, D,
            ctypes.byref(_how()), P(a["dq"]), HQ * D, P(a["dk"]), HKV * D, P(a["dqw"]), P(a["dkw"]),
            P(a["ws"]), MB, None, None)

    for w in ("dqw", "dkw"):
        for x in ("q", "k", "gq", "gk", "dq", "dk", "ws"):
            assert call(**{w: at[x]}) == BAD, (w, x)
        assert call(**{w: 5 * MB + QB - 4}) == BAD
    assert call(dkw=7 * MB + D * 4 - 4) == BAD  # on one another
    for x in ("q", "k", "gq", "gk", "dq", "dk"):
        assert call(ws=at[x]) == BAD, x
        assert call(ws=at[x] - (need - 256)) == BAD, x


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 500])
def test_gradients_in_place_and_between(T):
    """dq and dk over the upstream gradients, over the inputs, and beside the
    values' slice of the tensor that the inputs are slices of."""
    Hq, Hkv, d = 6, 2, 128
    g = torch.Generator().manual_seed(T)
    cs, pos = angles(T, d, g), torch.arange(T, device="cuda").int()
    qw, kw = weight(g, d), weight(g, d)

    def qkv():
        t = torch.empty(T, (Hq + 2 * Hkv) * d, dtype=torch.bfloat16, device="cuda")
        return t, t[:, :Hq * d].unflatten(1, (Hq, d)), \
            t[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))

    whole, q, k = qkv()
    whole.copy_(torch.randn(whole.shape, generator=g))
    gq = torch.randn(T, Hq, d, generator=g).bfloat16().cuda()
    gk = torch.randn(T, Hkv, d, generator=g).bfloat16().cuda()
    args = (pos, cs, qw, kw, EPS, False)
    want = psa.qk_norm_rope_bwd(q, k, gq, gk, *args)
    a, b = gq.clone(), gk.clone()
    got = psa.qk_norm_rope_bwd(q, k, a, b, *args, dq=a, dk=b)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    other, q2, k2 = qkv()
    other.copy_(whole)
    got = psa.qk_norm_rope_bwd(q2, k2, gq, gk, *args, dq=q2, dk=k2)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert torch.equal(other[:, (Hq + Hkv) * d:], whole[:, (Hq + Hkv) * d:])
    # dk where the values were
    other.copy_(whole)
    dk = other[:, (Hq + Hkv) * d:].unflatten(1, (Hkv, d))
    got = psa.qk_norm_rope_bwd(q2, k2, gq, gk, *args, dk=dk)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert torch.equal(other[:, :(Hq + Hkv) * d], whole[:, :(Hq + Hkv) * d])
    with pytest.raises(psa.PsaError):
        psa.qk_norm_rope_bwd(q2, k2, gq, gk, *args, dq=q2, dk=q2[:, 2:4])
