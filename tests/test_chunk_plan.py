"""The chunk planner and the host-side checks of the layer operators.  No GPU:
the plan is host data, and every call below is refused before any CUDA call."""
import ctypes

import numpy as np
import pytest
import torch

import shared_prefix_attention_b200 as psa

MAGIC = 0x50534343


def decode(data, info):
    """(lists, units, joins) of a plan."""
    assert data[0] == MAGIC and data[1] == info.n_ctas and data[2] == info.n_units
    assert data[3] == info.n_joins and len(data) == info.len
    lists = data[8:8 + info.n_ctas + 1]
    at = (8 + info.n_ctas + 1 + 3) // 4 * 4
    units = data[at:at + 12 * info.n_units].reshape(-1, 12)
    joins = data[at + 12 * info.n_units:].reshape(-1, 8)
    return lists, units, joins


CASES = [
    ([1], [1], 8, 2, 128, 0),
    ([1, 1, 1, 1], [901, 583, 2, 508], 32, 8, 128, 0),
    ([1, 0, 3], [5000, 0, 129], 28, 4, 128, 0),
    ([64, 65, 1, 63, 128, 129], [64, 200, 128, 4000, 128, 129], 32, 8, 128, 0),
    ([777, 638], [6777, 2730], 16, 16, 64, 4096),
    ([300], [5000], 5, 1, 64, 1),
    ([2048], [18432], 32, 8, 128, 0),
    ([9] * 40, list(range(9, 4009, 100)), 24, 8, 128, 300),
    ([3], [100000], 128, 1, 128, 0),
    ([1] * 300, [17 * i + 1 for i in range(300)], 8, 1, 64, 0),
]


@pytest.mark.parametrize("n_ctas", [1, 7, 148])
@pytest.mark.parametrize("ql,kl,Hq,Hkv,d,window", CASES)
def test_plan_covers_every_row_and_key_once(ql, kl, Hq, Hkv, d, window, n_ctas):
    data, info = psa.build_chunk_plan(ql, kl, Hq, Hkv, d, window, n_ctas)
    G = Hq // Hkv
    tph = 128 // G
    lists, units, joins = decode(data, info)
    assert info.n_rows == sum(ql) and info.n_keys == sum(kl) and info.n_ctas <= n_ctas
    assert lists[0] == 0 and lists[-1] == len(units) and (np.diff(lists) >= 0).all()
    # the query blocks: request, tokens, keys
    want = {}
    q0 = k0 = 0
    for n, L in zip(ql, kl):
        for i in range(0, n, 2 * tph):
            m = min(n - i, 2 * tph)
            pos = L - n + i
            lo = max(0, pos - window + 1) if window else 0
            for h in range(Hkv):
                want[(q0 + i, h)] = (m, pos, k0, lo, pos + m)
        q0 += n
        k0 += L
    pieces = {}
    for u in units.tolist():
        pieces.setdefault((u[0], u[3]), []).append(u)
    assert set(pieces) == set(want)
    ends = {}
    rows = np.zeros(info.part_rows, dtype=np.int64)
    for key, us in pieces.items():
        m, pos, kv0, lo, hi = want[key]
        us.sort(key=lambda u: u[5])
        twin = m <= tph
        for u in us:
            assert (u[1], u[2], u[4], bool(u[7])) == (m, pos, kv0, twin)
            assert u[5] < u[6] and (u[5] - lo) % 128 == 0
        assert us[0][5] == lo and us[-1][6] == hi
        assert all(a[6] == b[5] for a, b in zip(us, us[1:]))
        # partials: one per piece and, in a twin, half; none for a final block
        n_part = len(us) * (2 if twin else 1)
        if len(us) == 1 and (not twin or hi - lo <= 128):
            assert us[0][8] == -1
            continue
        per = m * G * (2 if twin else 1)
        parts = sorted(u[8] for u in us)
        assert parts == [parts[0] + i * per for i in range(len(us))]
        rows[parts[0]:parts[0] + n_part * m * G] += 1
        ends[key] = (parts[0], m * G, n_part)
    assert (rows == 1).all()
    assert {(j[0], j[2]): (j[3], j[1], j[4]) for j in joins.tolist()} == ends
    assert info.max_join_rows == max([j[1] for j in joins.tolist()], default=0)
    need = info.part_rows * d * 4 + info.part_rows * 4
    ws = psa.lib().psa_chunk_workspace_size(ctypes.byref(info))
    assert ws >= max(need, 256) and ws % 256 == 0


def test_plan_balances_long_work():
    """The longest list holds at most a tenth more tiles than the mean."""
    data, info = psa.build_chunk_plan([2048], [18432], 32, 8, 128)
    lists, units, _ = decode(data, info)
    tiles = [(u[6] - u[5] + 127) // 128 for u in units.tolist()]
    loads = [sum(tiles[lists[c]:lists[c + 1]]) for c in range(info.n_ctas)]
    assert max(loads) <= 1.1 * sum(loads) / 148


def test_empty_plans():
    for ql, kl in (([], []), ([0], [0]), ([0, 0], [5, 0])):
        data, info = psa.build_chunk_plan(ql, kl, 8, 2, 128)
        assert info.n_rows == 0 and info.n_units == 0 and info.n_keys == sum(kl)


@pytest.mark.parametrize("ql,kl,Hq,Hkv,d,window,n_ctas,status", [
    ([2], [1], 8, 2, 128, 0, 148, psa.PSA_ERR_INVALID_ARG),     # its own keys are missing
    ([-1], [4], 8, 2, 128, 0, 148, psa.PSA_ERR_INVALID_ARG),
    ([1], [4], 6, 4, 128, 0, 148, psa.PSA_ERR_INVALID_ARG),
    ([1], [4], 0, 1, 128, 0, 148, psa.PSA_ERR_INVALID_ARG),
    ([1], [4], 8, 2, 128, -1, 148, psa.PSA_ERR_INVALID_ARG),
    ([1], [4], 8, 2, 128, 0, 0, psa.PSA_ERR_INVALID_ARG),
    ([1], [4], 8, 2, 256, 0, 148, psa.PSA_ERR_UNSUPPORTED),
    ([1], [4], 129, 1, 128, 0, 148, psa.PSA_ERR_UNSUPPORTED),
    ([1, 1], [2**31 - 1, 2**31 - 1], 8, 2, 128, 0, 148, psa.PSA_ERR_INVALID_ARG),
    ([1], [2**31 - 100], 8, 2, 128, 0, 148, psa.PSA_ERR_INVALID_ARG),
])
def test_plan_refusals(ql, kl, Hq, Hkv, d, window, n_ctas, status):
    with pytest.raises(psa.PsaError) as e:
        psa.build_chunk_plan(ql, kl, Hq, Hkv, d, window, n_ctas)
    assert e.value.status == status


def test_plan_capacity():
    info = psa.ChunkInfo()
    one = np.array([1], dtype=np.int32)
    p = one.ctypes.data_as(ctypes.c_void_p)
    out = np.full(4, -7, dtype=np.int32)
    rc = psa.lib().psa_build_chunk_plan(p, p, 1, 8, 2, 128, 0, 148,
                                        out.ctypes.data_as(ctypes.c_void_p), 4,
                                        ctypes.byref(info))
    assert rc == psa.PSA_ERR_CAPACITY and info.len > 4 and (out == -7).all()
    assert psa.lib().psa_build_chunk_plan(None, p, 1, 8, 2, 128, 0, 148, None, 0,
                                          ctypes.byref(info)) == psa.PSA_ERR_INVALID_ARG


# ------------------------------------------------------------------ host checks of the calls

P = ctypes.c_void_p


def _info(**kw):
    _, info = psa.build_chunk_plan([300], [2000], 8, 2, 128)
    for k, v in kw.items():
        setattr(info, k, v)
    return info


def _chunk(**kw):
    a = dict(q=16, k=16, v=16, ntok=2000, table=None, sc=None, o=1 << 30, lse=None, T=300, scale=0.1,
             cap=0.0, info=_info(), plan=16, ws=256, wsb=1 << 40)
    a.update(kw)
    sc = ctypes.byref(psa.KvScales(*a["sc"])) if a["sc"] else None
    return psa.lib().psa_chunk_fwd(P(a["q"]), P(a["k"]), P(a["v"]), a["ntok"], P(a["table"]), sc,
                                   P(a["o"]), P(a["lse"]), a["T"], a["scale"], a["cap"],
                                   ctypes.byref(a["info"]) if a["info"] else None, P(a["plan"]),
                                   P(a["ws"]), a["wsb"], None, None)


def test_chunk_host_validation():
    bad = psa.PSA_ERR_INVALID_ARG
    for kw in (dict(info=None), dict(T=299), dict(ntok=1999), dict(ntok=2**31), dict(scale=0.0),
               dict(scale=float("inf")), dict(scale=3e38), dict(scale=1.0, cap=1e-39), dict(cap=-1.0),
               dict(o=16), dict(o=16 + 300 * 8 * 128), dict(cap=float("nan")), dict(q=8),
               dict(q=None), dict(k=None), dict(v=24 + 1), dict(o=None), dict(lse=2),
               dict(table=2), dict(plan=None), dict(plan=8), dict(sc=(0.0, 1.0)),
               dict(sc=(1.0, float("inf")))):
        assert _chunk(**kw) == bad, kw
    assert _chunk(cap=1001.0) == psa.PSA_ERR_UNSUPPORTED
    for kw in (dict(ws=None), dict(ws=128), dict(wsb=255)):
        assert _chunk(**kw) == psa.PSA_ERR_WORKSPACE, kw
    assert _chunk(info=_info(n_rows=0), q=None) == psa.PSA_OK  # nothing to do


def _how(**kw):
    h = psa.NormRope(16, 16, 8, 64, 0, 16, 16, psa.PSA_F32, 1e-6)
    for k, v in kw.items():
        setattr(h, k, v)
    return h


BAD_HOW = (dict(rot_dim=8), dict(rot_dim=144), dict(rot_dim=0), dict(positions=None),
           dict(cos_sin=4), dict(n_positions=-1), dict(q_weight=8), dict(weight_dtype=7),
           dict(eps=-1.0), dict(eps=float("nan")))


def _rope(fn, **kw):
    a = dict(q=16, qs=1024, k=16, ks=256, dt=psa.PSA_BF16, T=4, Hq=8, Hkv=2, d=128, how=_how(),
             qo=16, ko=16, ws=256, wsb=1 << 30, dqw=None)
    a.update(kw)
    how = ctypes.byref(a["how"]) if a["how"] else None
    if fn == "fwd":
        return psa.lib().psa_qk_norm_rope_fwd(P(a["q"]), a["qs"], P(a["k"]), a["ks"], a["dt"],
                                              a["T"], a["Hq"], a["Hkv"], a["d"], how, P(a["qo"]),
                                              P(a["ko"]), None, None)
    return psa.lib().psa_qk_norm_rope_bwd(P(a["q"]), a["qs"], P(a["k"]), a["ks"], P(a["qo"]),
                                          P(a["ko"]), a["dt"], a["T"], a["Hq"], a["Hkv"], a["d"],
                                          how, P(16), a["qs"], P(16), a["ks"], P(a["dqw"]), None,
                                          P(a["ws"]), a["wsb"], None, None)


@pytest.mark.parametrize("fn", ["fwd", "bwd"])
def test_qk_norm_rope_host_validation(fn):
    bad = psa.PSA_ERR_INVALID_ARG
    for kw in (dict(how=None), dict(q=None, k=None), dict(dt=5), dict(T=-1), dict(Hq=0),
               dict(q=8), dict(qs=1023), dict(qs=1028), dict(ks=128), dict(qo=None),
               dict(ko=12)):
        assert _rope(fn, **kw) == bad, kw
    for kw in BAD_HOW:
        assert _rope(fn, how=_how(**kw)) == bad, kw
    assert _rope(fn, d=96) == psa.PSA_ERR_UNSUPPORTED
    if fn == "fwd":
        assert _rope(fn, T=0) == psa.PSA_OK
    else:
        assert _rope(fn, dqw=16, how=_how(q_weight=None)) == bad  # no norm, no gradient
        assert _rope(fn, wsb=16) == psa.PSA_ERR_WORKSPACE
        assert _rope(fn, ws=None) == psa.PSA_ERR_WORKSPACE


def _append(**kw):
    a = dict(q=16, qs=1024, k=16, ks=256, v=16, vs=256, T=4, Hq=8, Hkv=2, d=128, how=_how(),
             kc=16, vc=16, ntok=8, slots=16, sc=None, qo=16)
    a.update(kw)
    sc = ctypes.byref(psa.KvScales(*a["sc"])) if a["sc"] else None
    return psa.lib().psa_cache_append(P(a["q"]), a["qs"], P(a["k"]), a["ks"], P(a["v"]), a["vs"],
                                      a["T"], a["Hq"], a["Hkv"], a["d"],
                                      ctypes.byref(a["how"]) if a["how"] else None, P(a["kc"]),
                                      P(a["vc"]), a["ntok"], P(a["slots"]), sc, P(a["qo"]), None,
                                      None)


def test_cache_append_host_validation():
    bad = psa.PSA_ERR_INVALID_ARG
    for kw in (dict(T=-1), dict(Hkv=0), dict(Hq=0), dict(ntok=-1), dict(ntok=2**31), dict(k=None),
               dict(v=None), dict(kc=None), dict(vc=8), dict(slots=None), dict(slots=2),
               dict(ks=255), dict(vs=0), dict(qo=None), dict(sc=(-1.0, 1.0)),
               dict(sc=(1.0, 1e-39))):
        assert _append(**kw) == bad, kw
    for kw in BAD_HOW:
        assert _append(how=_how(**kw)) == bad, kw
    assert _append(d=80) == psa.PSA_ERR_UNSUPPORTED
    assert _append(T=0) == psa.PSA_OK
    assert _append(T=0, how=_how(positions=None)) == psa.PSA_OK


def _read(**kw):
    a = dict(kc=16, vc=16, ntok=8, rows=16, n=4, Hkv=2, d=128, sc=None, k=16, v=16)
    a.update(kw)
    sc = ctypes.byref(psa.KvScales(*a["sc"])) if a["sc"] else None
    return psa.lib().psa_cache_read(P(a["kc"]), P(a["vc"]), a["ntok"], P(a["rows"]), a["n"],
                                    a["Hkv"], a["d"], sc, P(a["k"]), P(a["v"]), None, None)


def test_cache_read_host_validation():
    bad = psa.PSA_ERR_INVALID_ARG
    for kw in (dict(n=-1), dict(Hkv=0), dict(ntok=-1), dict(kc=None), dict(vc=8), dict(rows=None),
               dict(rows=1), dict(k=None), dict(v=8), dict(sc=(1.0, 0.0))):
        assert _read(**kw) == bad, kw
    assert _read(d=32) == psa.PSA_ERR_UNSUPPORTED
    assert _read(n=0) == psa.PSA_OK


def test_binding_refuses_tensors_that_do_not_fit():
    """There is no CPU path, and shapes, dtypes and strides are checked before
    the library is called."""
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    w = torch.zeros(128)
    with pytest.raises(ValueError):
        psa.qk_norm_rope(x, x, None, None, w, w)
    with pytest.raises(ValueError):
        psa.qk_norm_rope(x.half(), x.half(), None, None)
    with pytest.raises(ValueError):
        psa.qk_norm_rope_bwd(x, x, x, x, None, None, w, w)
    with pytest.raises(ValueError):
        psa.cache_append(x, x, x, x, x, i)
    with pytest.raises(ValueError):
        psa.cache_read(x, x, i)
    with pytest.raises(ValueError):
        psa.cache_read(x, x, i, k_scale=1.0)  # one scale only
    data, info = psa.build_chunk_plan([4], [4], 2, 2, 128)
    plan = psa.ChunkPlan(info, torch.from_numpy(data), 256)
    with pytest.raises(ValueError):
        psa.chunk(x, x, x, plan, 1.0)
    with pytest.raises(ValueError):
        psa.build_chunk_plan([1, 2], [3], 2, 2, 128)


def test_large_batches_are_planned_quickly():
    """4096 decoding requests: one plan per step has to stay cheap."""
    import time
    t = time.perf_counter()
    _, info = psa.build_chunk_plan([1] * 4096, [1000 + i % 700 for i in range(4096)], 32, 8, 128)
    assert info.n_units >= 4096 * 8 and time.perf_counter() - t < 0.5


WIDE = 2**32


@pytest.mark.parametrize("args", [
    ([1], np.array([WIDE + 100]), 8, 2, 128),
    (np.array([WIDE + 1]), [100], 8, 2, 128),
    (torch.tensor([1]), torch.tensor([WIDE + 100]), 8, 2, 128),
    (np.array([1], dtype=np.uint64), np.array([2**64 - 1], dtype=np.uint64), 8, 2, 128),
    ([1], [WIDE + 100], 8, 2, 128),
    ([1], [2**70], 8, 2, 128),
    ([1], [100.5], 8, 2, 128),
    ([0.5], [100], 8, 2, 128),
    ([1], [float("nan")], 8, 2, 128),
    ([[1]], [[100]], 8, 2, 128),
    ([1], [100], WIDE + 8, 2, 128),
    ([1], [100], 8, WIDE + 2, 128),
    ([1], [100], 8, 2, WIDE + 128),
    ([1], [100], 8, 2, 128, 0, WIDE + 148),
    ([1], [100], 8, 2, 128, 4.5),
    ([1], [100], 8, 2, 128, -WIDE),
])
def test_plan_arguments_beyond_32_bits_are_refused(args):
    """No length, head count or window becomes another one on its way to the
    planner's 32-bit integers."""
    with pytest.raises((ValueError, psa.PsaError)):
        psa.build_chunk_plan(*args)


def test_plan_takes_any_integers_and_windows_beyond_every_key():
    want, _ = psa.build_chunk_plan([3, 1], [700, 9], 8, 2, 128)
    for ql, kl in ((np.array([3, 1]), np.array([700, 9], dtype=np.uint16)),
                   (torch.tensor([3, 1]), torch.tensor([700, 9], dtype=torch.int32)),
                   ((3, 1), (700.0, 9.0))):
        assert (psa.build_chunk_plan(ql, kl, 8, 2, 128)[0] == want).all()
    whole = decode(*psa.build_chunk_plan([3, 1], [700, 9], 8, 2, 128, 2**31 - 1))[1]
    for window in (700, WIDE + 5, 2**70):
        data, info = psa.build_chunk_plan([3, 1], [700, 9], 8, 2, 128, window)
        assert (decode(data, info)[1] == whole).all() and info.window >= 700


MB = 1 << 20
APART = dict(q=64 * MB, k=MB, v=8 * MB, o=128 * MB, lse=192 * MB, ws=256 * MB)


@pytest.mark.parametrize("fields", [
    dict(Hq=0), dict(Hkv=0), dict(Hkv=-2), dict(Hq=9), dict(head_dim=0), dict(head_dim=96),
    dict(head_dim=256), dict(Hq=258), dict(window=-1), dict(n_rows=-1), dict(n_keys=299),
    dict(n_keys=2**31), dict(n_ctas=0), dict(n_units=0), dict(n_units=-1), dict(n_joins=-1),
    dict(part_rows=-1), dict(part_rows=0), dict(part_rows=2**31), dict(max_join_rows=0),
    dict(max_join_rows=257), dict(len=8), dict(Hq=2**31 - 2),
])
def test_call_refuses_an_info_that_no_plan_has(fields):
    """The fields of a hand-made or stale info lead to divisions, grids and
    buffer sizes: what cannot come from the planner is refused on the host."""
    info = _info(**fields)
    assert info.n_joins != 0  # split blocks: every field counts
    rc = _chunk(info=info, T=300, ntok=3000, table=16, **APART)
    assert rc in (psa.PSA_ERR_INVALID_ARG, psa.PSA_ERR_UNSUPPORTED)


def test_plan_object_checks_its_lists():
    """Lists that are shorter than the plan's length, or not int32 words, are
    not what a kernel may read."""
    data, info = psa.build_chunk_plan([4], [4], 2, 2, 128)
    whole = torch.from_numpy(data)
    for bad in (whole[:-1], whole.long(), whole.float(), torch.stack([whole, whole], 1)[:, 0]):
        with pytest.raises(ValueError, match="plan"):
            psa.ChunkPlan(info, bad, 256)
    psa.ChunkPlan(info, whole, 256)
    psa.ChunkPlan(info, torch.cat([whole, whole]), 256)
