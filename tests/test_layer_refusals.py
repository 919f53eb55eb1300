"""What the calls around a layer refuse, one bad argument at a time in a call
that is good otherwise.  The good call gets past every check to the launch,
which a machine without a GPU answers with PSA_ERR_CUDA; the addresses are made
up, so where there is a GPU nothing of this runs."""
import ctypes

import pytest
import torch

import shared_prefix_attention_b200 as psa
from test_chunk_plan import CASES

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")

P = ctypes.c_void_p
BAD, UNSUPPORTED, WS = psa.PSA_ERR_INVALID_ARG, psa.PSA_ERR_UNSUPPORTED, psa.PSA_ERR_WORKSPACE
MB = 1 << 20
NAN, INF = float("nan"), float("inf")


def how(**kw):
    h = psa.NormRope(40 * MB, 41 * MB, 8, 64, 0, 42 * MB, 43 * MB, psa.PSA_F32, 1e-6)
    for k, v in kw.items():
        setattr(h, k, v)
    return h


BAD_HOW = [dict(positions=None), dict(positions=40 * MB + 2), dict(cos_sin=41 * MB + 4),
           dict(n_positions=-1), dict(rot_dim=0), dict(rot_dim=-16), dict(rot_dim=8),
           dict(rot_dim=144), dict(q_weight=42 * MB + 8), dict(k_weight=43 * MB + 8),
           dict(weight_dtype=7), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF)]


def ref(x):
    return ctypes.byref(x) if x is not None else None


def forward(q=MB, qs=1024, k=2 * MB, ks=256, dtype=psa.PSA_BF16, T=4, Hq=8, Hkv=2, d=128, qo=3 * MB,
            ko=4 * MB, h=how()):
    return psa.lib().psa_qk_norm_rope_fwd(P(q), qs, P(k), ks, dtype, T, Hq, Hkv, d, ref(h), P(qo),
                                          P(ko), None, None)


def gradients(q=MB, qs=1024, k=2 * MB, ks=256, gq=3 * MB, gk=4 * MB, dtype=psa.PSA_BF16, T=4, Hq=8,
              Hkv=2, d=128, h=how(), dq=5 * MB, dqs=1024, dk=6 * MB, dks=256, dqw=7 * MB,
              dkw=8 * MB, ws=9 * MB, n=MB):
    return psa.lib().psa_qk_norm_rope_bwd(P(q), qs, P(k), ks, P(gq), P(gk), dtype, T, Hq, Hkv, d,
                                          ref(h), P(dq), dqs, P(dk), dks, P(dqw), P(dkw), P(ws), n,
                                          None, None)


def append(q=MB, qs=1024, k=2 * MB, ks=256, v=3 * MB, vs=256, T=4, Hq=8, Hkv=2, d=128, h=how(),
           kc=4 * MB, vc=5 * MB, n=8, slots=6 * MB, sc=None, qo=7 * MB):
    sc = psa.KvScales(*sc) if sc else None
    return psa.lib().psa_cache_append(P(q), qs, P(k), ks, P(v), vs, T, Hq, Hkv, d, ref(h), P(kc),
                                      P(vc), n, P(slots), ref(sc), P(qo), None, None)


def read(kc=MB, vc=2 * MB, cached=8, rows=3 * MB, n=4, Hkv=2, d=128, sc=None, k=4 * MB, v=5 * MB):
    sc = psa.KvScales(*sc) if sc else None
    return psa.lib().psa_cache_read(P(kc), P(vc), cached, P(rows), n, Hkv, d, ref(sc), P(k), P(v),
                                    None, None)


INFO = psa.build_chunk_plan([300], [2000], 8, 2, 128)[1]


def chunk(q=MB, k=4 * MB, v=8 * MB, cached=2000, table=12 * MB, sc=None, o=16 * MB, lse=20 * MB,
          T=300, scale=0.1, cap=0.0, info=INFO, plan=24 * MB, ws=64 * MB, n=1 << 40):
    sc = psa.KvScales(*sc) if sc else None
    return psa.lib().psa_chunk_fwd(P(q), P(k), P(v), cached, P(table), ref(sc), P(o), P(lse), T,
                                   scale, cap, ref(info), P(plan), P(ws), n, None, None)


GOOD = [
    (forward, [dict(), dict(dtype=psa.PSA_F32), dict(qs=1536, ks=1536), dict(q=None, qo=None),
               dict(k=None, ko=None), dict(h=how(cos_sin=None, positions=None)), dict(d=64, qs=512),
               dict(h=how(q_weight=None, k_weight=None, weight_dtype=9, eps=-1.0)),
               dict(h=how(eps=0.0)), dict(qo=MB), dict(d=256, qs=2048, ks=512)]),
    (gradients, [dict(), dict(dtype=psa.PSA_F32), dict(dqw=None, dkw=None), dict(dq=3 * MB),
                 dict(dqs=1536, dks=1536, dk=5 * MB + 2048), dict(dq=MB, dk=2 * MB),
                 dict(n=296 * 128 * 4)]),
    (append, [dict(), dict(q=None, qo=None), dict(sc=(0.5, 2.0)), dict(h=None), dict(qo=MB)]),
    (read, [dict(), dict(sc=(0.5, 2.0)), dict(vc=MB), dict(d=64), dict(d=256)]),
    (chunk, [dict(), dict(table=None), dict(sc=(0.5, 2.0)), dict(lse=None), dict(cap=1000.0),
             dict(T=301), dict(cached=10), dict(v=4 * MB)]),
]


@pytest.mark.parametrize("call,kw", [(c, kw) for c, kws in GOOD for kw in kws])
def test_good_calls_reach_the_launch(call, kw):
    assert call(**kw) == psa.PSA_ERR_CUDA


@pytest.mark.parametrize("case", CASES)
def test_every_plan_is_taken(case):
    info = psa.build_chunk_plan(*case)[1]
    assert chunk(info=info, T=info.n_rows, cached=1, q=1 << 40, k=2 << 40, v=3 << 40, o=4 << 40,
                 lse=5 << 40, ws=6 << 40) == psa.PSA_ERR_CUDA


@pytest.mark.parametrize("kw", [
    dict(q=None, k=None), dict(dtype=5), dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(h=None),
    dict(q=MB + 8), dict(k=2 * MB + 8), dict(qs=1023), dict(qs=1028), dict(qs=0), dict(qs=-1024),
    dict(ks=128), dict(ks=260), dict(qo=None), dict(ko=None), dict(qo=3 * MB + 8),
    dict(ko=4 * MB + 4), dict(dtype=psa.PSA_F32, qs=1022),
    *(dict(h=how(**x)) for x in BAD_HOW)])
def test_forward_refuses(kw):
    assert forward(**kw) == BAD


@pytest.mark.parametrize("kw", [
    dict(q=None, k=None, dqw=None, dkw=None), dict(dtype=5), dict(T=-1), dict(Hq=0), dict(Hkv=0),
    dict(h=None), dict(q=MB + 8), dict(k=2 * MB + 8), dict(gq=3 * MB + 8), dict(gk=4 * MB + 8),
    dict(dq=5 * MB + 8), dict(dk=6 * MB + 8), dict(qs=1016), dict(qs=1028), dict(ks=252),
    dict(dqs=1016), dict(dqs=1028), dict(dks=128), dict(gq=None), dict(gk=None), dict(dq=None),
    dict(dk=None), dict(dqw=7 * MB + 2), dict(dkw=8 * MB + 1), dict(q=None), dict(k=None),
    dict(h=how(q_weight=None)), dict(h=how(k_weight=None)),
    *(dict(h=how(**x)) for x in BAD_HOW)])
def test_gradients_refuse(kw):
    assert gradients(**kw) == BAD


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(Hkv=0), dict(Hq=0), dict(n=-1), dict(n=2**31), dict(k=None), dict(v=None),
    dict(k=2 * MB + 8), dict(v=3 * MB + 8), dict(q=MB + 8), dict(kc=None), dict(vc=None),
    dict(kc=4 * MB + 8), dict(vc=5 * MB + 8), dict(slots=None), dict(slots=6 * MB + 2),
    dict(ks=252), dict(ks=260), dict(vs=0), dict(qs=1016), dict(qo=None), dict(qo=7 * MB + 8),
    dict(sc=(-1.0, 1.0)), dict(sc=(1.0, 0.0)), dict(sc=(NAN, 1.0)), dict(sc=(1.0, INF)),
    dict(sc=(1e-39, 1.0)), dict(sc=(1.0, 1e-39)), *(dict(h=how(**x)) for x in BAD_HOW)])
def test_append_refuses(kw):
    assert append(**kw) == BAD


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(Hkv=0), dict(Hkv=2**30), dict(cached=-1), dict(cached=2**31), dict(kc=None),
    dict(vc=None), dict(kc=MB + 8), dict(vc=2 * MB + 8), dict(rows=None), dict(rows=3 * MB + 1),
    dict(k=None), dict(v=None), dict(k=4 * MB + 8), dict(v=5 * MB + 8), dict(sc=(1.0, 0.0)),
    dict(sc=(NAN, 1.0))])
def test_read_refuses(kw):
    assert read(**kw) == BAD


@pytest.mark.parametrize("kw", [
    dict(info=None), dict(T=299), dict(T=-1), dict(cached=-1), dict(cached=2**31),
    dict(cached=1999, table=None), dict(scale=0.0), dict(scale=-1.0), dict(scale=INF),
    dict(scale=NAN), dict(scale=3e38), dict(scale=1.0, cap=1e-39), dict(cap=-1.0), dict(cap=NAN),
    dict(cap=INF), dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(plan=None),
    dict(q=MB + 8), dict(k=4 * MB + 8), dict(v=8 * MB + 8), dict(o=16 * MB + 8),
    dict(plan=24 * MB + 8), dict(lse=20 * MB + 2), dict(table=12 * MB + 2), dict(sc=(0.0, 1.0)),
    dict(sc=(1.0, INF)), dict(sc=(1e-30, 1.0), scale=1e-30)])
def test_chunk_refuses(kw):
    assert chunk(**kw) == BAD


def test_what_is_not_supported_or_has_no_workspace():
    for call in (forward, gradients, append, read):
        for d in (0, 32, 96, 512):
            assert call(d=d) == UNSUPPORTED
    assert chunk(cap=1001.0) == UNSUPPORTED
    for kw in (dict(ws=None), dict(ws=64 * MB + 128), dict(n=255)):
        assert gradients(**{**kw, **({"ws": 9 * MB + 128} if kw.get("ws") else {})}) == WS
        assert chunk(**kw) == WS
    assert gradients(n=296 * 128 * 4 - 1) == WS
    need = psa.lib().psa_chunk_workspace_size(ctypes.byref(INFO))
    assert chunk(n=need) == psa.PSA_ERR_CUDA and chunk(n=need - 1) == WS


def test_nothing_to_do_is_no_error():
    assert forward(T=0) == append(T=0) == read(n=0) == psa.PSA_OK
    assert append(T=0, h=how(positions=None)) == forward(T=0, h=how(positions=None)) == psa.PSA_OK
    assert chunk(info=psa.build_chunk_plan([0], [7], 8, 2, 128)[1], q=None, T=0) == psa.PSA_OK
