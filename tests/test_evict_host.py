"""Eviction, what needs no GPU: closed forms of the oracle's accumulated
blending weights and survivor order, argument checks of the C calls and of the
Splatter (all before anything is enqueued), and the score summed over ranks."""

import ctypes
import os
import socket

import numpy as np
import pytest
import torch
import torch.distributed as dist
import torch.multiprocessing as mp

from gaussian_splatting_differentiable_ewa_b200 import api
from gaussian_splatting_differentiable_ewa_b200 import scenes as S
from gaussian_splatting_differentiable_ewa_b200.pipeline import Splatter
from oracle import oracle as O


def _record(u, v, sigma, o):
    """An isotropic splat's record (see gs_projected)."""
    k = np.sqrt(0.5 / np.log(2.0)) / sigma
    r = np.zeros(16, np.float32)
    r[[0, 1, 2, 6, 8, 14]] = u, v, k, k, -np.log2(255.0 * o), o
    return r


def test_oracle_weights_closed_forms():
    """One splat on a pixel centre weighs its opacity there; a second one behind
    it weighs what the first leaves; weights and transmittance sum to one."""
    rec = np.stack([_record(8.5, 8.5, 3.0, 0.6), _record(8.5, 8.5, 3.0, 0.5)])[None]
    ids, ranges = np.array([0, 1], np.uint32), np.array([[0, 2]])
    nc = np.full((1, 16, 16), 2)
    s, m, slack = O.blend_weights(rec, ids, ranges, nc, 16, 16)
    assert m[0] == pytest.approx(0.6, rel=1e-6)
    y, x = np.mgrid[0:16, 0:16]
    q = ((x - 8.0) ** 2 + (y - 8.0) ** 2) / 9.0
    a0, a1 = (np.where(o * np.exp(-q / 2) >= 1 / 255, o * np.exp(-q / 2), 0) for o in (0.6, 0.5))
    assert s[0] == pytest.approx(a0.sum(), rel=1e-6)
    assert s[1] == pytest.approx((a1 * (1 - a0)).sum(), rel=1e-6)
    assert s.sum() + ((1 - a0) * (1 - a1)).sum() == pytest.approx(256.0, rel=1e-7)
    assert np.all(slack >= 0) and np.all(slack < 1e-3 * s)
    # one pixel of weight one half, every other masked
    pw = np.zeros((1, 16, 16), np.float32)
    pw[0, 8, 8] = 0.5
    s1, m1, _ = O.blend_weights(rec, ids, ranges, nc, 16, 16, pw)
    assert s1[0] == pytest.approx(0.3, rel=1e-6) and m1[0] == s1[0]
    assert s1[1] == pytest.approx(0.5 * 0.5 * 0.4, rel=1e-6)
    pw[:] = np.nan
    assert not O.blend_weights(rec, ids, ranges, nc, 16, 16, pw)[0].any()


def test_oracle_survivor_order():
    nan, inf = float("nan"), float("inf")
    s = np.array([1.0, nan, -0.0, 0.0, inf, -inf, 1.0], np.float32)
    order = [4, 0, 6, 2, 3, 5, 1]
    for k in range(8):
        want = np.zeros(7, np.int8)
        want[order[:k]] = 1
        assert np.array_equal(O.evict_select(s, None, k), want), k
    assert O.evict_select(s, [0, 1, 0, 0, 0, 1, 0], 2).tolist() == [0, 1, 0, 0, 0, 1, 0]
    assert O.evict_select(s, [0, 1, 0, 0, 0, 1, 0], 1).tolist() == [0, 1, 0, 0, 0, 0, 0]


P = ctypes.c_void_p(4096)  # aligned, never dereferenced: every call returns first


def _cam(w=64, h=48):
    sc = S.make_scene("fwd_1k_128", n=1)
    c = sc.cameras[0]
    c.width, c.height = w, h
    return api.cameras([c])


def test_blend_weights_arguments():
    L = api.lib()
    size = api.gs_blend_weights_workspace_size
    assert size(0) > 0 and size(-1) == 0 and size(1 << 31) == 0 and size(1000) % 256 == 0
    assert size(1000) - size(0) >= 8000 - 256
    proj = api.GsProjected(4096, None, None)
    bins = api.GsBinned(4096, 4096, None, 10)
    ok = dict(proj=ctypes.byref(proj), bins=ctypes.byref(bins), cams=_cam(), V=1, n=10, nc=P,
              wm=None, pw=None, decay=1.0, s=P, m=None, ws=P, nb=size(10))

    def call(**kw):
        a = {**ok, **kw}
        return L.gs_blend_weights(a["proj"], a["bins"], a["cams"], a["V"], a["n"], a["nc"],
                                  a["wm"], a["pw"], a["decay"], a["s"], a["m"], a["ws"], a["nb"],
                                  None)

    odd = ctypes.c_void_p(4098)
    none = api.GsProjected(None, None, None)
    off = api.GsProjected(4104, None, None)
    no_ids, no_ranges = api.GsBinned(None, 4096, None, 10), api.GsBinned(4096, None, None, 10)
    negative = api.GsBinned(4096, 4096, None, -1)
    for kw in (dict(proj=None), dict(bins=None), dict(V=0), dict(V=33), dict(n=-1), dict(nc=None),
               dict(s=None), dict(ws=None), dict(ws=ctypes.c_void_p(4100)), dict(nb=size(10) - 1),
               dict(decay=-0.5), dict(decay=1.5), dict(decay=float("nan")), dict(nc=odd),
               dict(pw=odd), dict(s=odd), dict(m=odd), dict(proj=ctypes.byref(none)),
               dict(proj=ctypes.byref(off)), dict(bins=ctypes.byref(no_ids)),
               dict(bins=ctypes.byref(no_ranges)), dict(bins=ctypes.byref(negative)),
               dict(cams=None)):
        assert call(**kw) == api.GS_ERR_INVALID_ARG, kw
    assert call(n=1 << 31) == api.GS_ERR_OVERFLOW
    assert call(cams=_cam(65536, 32769)) == api.GS_ERR_OVERFLOW  # more than 2^31 pixels
    assert call(n=0, nc=None, s=None, nb=size(0)) == api.GS_OK  # nothing to do


def test_evict_select_arguments():
    L = api.lib()
    size = api.gs_evict_workspace_size
    assert size(0) > 0 and size(-1) == 0 and size(1 << 31) == 0 and size(10 ** 6) % 256 == 0
    nb = size(10)
    bad = [(None, None, 10, 5, P, P, nb), (P, None, 10, 5, None, P, nb),
           (P, None, 10, 5, P, None, nb), (P, None, 10, 5, P, ctypes.c_void_p(4100), nb),
           (P, None, 10, 5, P, P, nb - 1), (P, None, -1, 5, P, P, nb),
           (P, None, 10, -1, P, P, nb), (ctypes.c_void_p(4098), None, 10, 5, P, P, nb)]
    for a in bad:
        assert L.gs_evict_select(*a, None) == api.GS_ERR_INVALID_ARG, a
    assert L.gs_evict_select(P, None, 1 << 31, 5, P, P, 1 << 40, None) == api.GS_ERR_OVERFLOW
    assert L.gs_evict_select(None, None, 0, 5, None, P, nb, None) == api.GS_OK


def test_evict_compact_arguments():
    L = api.lib()
    nb = api.gs_evict_workspace_size(10)
    a16 = 4096
    full = [a16] * 5

    def call(params=None, m=None, v=None, dec=P, out=full, mo=None, vo=None, cap=10, src=None,
             n_out=None, ws=P, nb=nb):
        g = lambda x: None if x is None else ctypes.byref(api.GsGrads(*x))  # noqa: E731
        p = params if params is not None else api.GsParams(*full, 1, 0, 10, None)
        return L.gs_evict_compact(ctypes.byref(p), g(m), g(v), dec, g(out), g(mo), g(vo), cap,
                                  src, n_out, ws, nb, None)

    hole = lambda k: [None if j == k else a16 for j in range(5)]  # noqa: E731
    skew = lambda k: [a16 + 4 if j == k else a16 for j in range(5)]  # noqa: E731
    bad = [dict(dec=None), dict(out=None), dict(cap=-1), dict(ws=None), dict(nb=nb - 1),
           dict(ws=ctypes.c_void_p(4100)), dict(n_out=ctypes.c_void_p(4100)),
           dict(src=ctypes.c_void_p(4098)),
           # moments: all four or none
           dict(m=full), dict(m=full, v=full), dict(m=full, v=full, mo=full), dict(mo=full),
           dict(m=full, mo=full), dict(m=hole(4), v=full, mo=full, vo=full),
           dict(m=full, v=full, mo=full, vo=skew(1))]
    bad += [dict(out=hole(k)) for k in range(5)]
    bad += [dict(out=skew(k)) for k in (0, 1, 2, 4)]
    bad += [dict(params=api.GsParams(*hole(k), 1, 0, 10, None)) for k in range(5)]
    bad += [dict(params=api.GsParams(*full, 4, 0, 10, None)),
            dict(params=api.GsParams(*full, -1, 0, 10, None)),
            dict(params=api.GsParams(*full, 1, 0, -1, None))]
    for kw in bad:
        assert call(**kw) == api.GS_ERR_INVALID_ARG, kw
    assert call(cap=1 << 31) == api.GS_ERR_OVERFLOW
    big = api.GsParams(*full, 1, 0, 1 << 31, None)
    assert call(params=big) == api.GS_ERR_OVERFLOW


def test_splatter_refuses_on_the_host():
    sp = Splatter(S.make_scene("fwd_1k_128", n=50), device="cpu")
    with pytest.raises(ValueError, match="accumulate_weights"):
        sp.evict(10)
    score = torch.zeros(50)
    for kw in (dict(n_keep=0), dict(n_keep=-3)):
        with pytest.raises(ValueError, match="n_keep"):
            sp.evict(score=score, **kw)
    for bad in (torch.zeros(49), torch.zeros(50, dtype=torch.float64), torch.zeros(50, 1)):
        with pytest.raises(ValueError, match="score"):
            sp.evict(10, score=bad)
    for bad in (torch.zeros(50), torch.zeros(49, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="protect"):
            sp.evict(10, score=score, protect=bad)
    with pytest.raises(ValueError, match="render"):
        sp.accumulate_weights()
    sp._frame_gen = sp._gen            # as after a render
    for bad in (torch.zeros(1, 128, 127), torch.zeros(1, 128, 128, dtype=torch.float64),
                torch.zeros(1, 128, 256)[:, :, ::2]):
        with pytest.raises(ValueError, match="pixel_weight"):
            sp.accumulate_weights(pixel_weight=bad)
    assert sp.weights_status() == api.GS_OK


def _free_port() -> int:
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        return s.getsockname()[1]


def _evict_worker(rank, world, port, out):
    """The Splatter's own eviction on CPU ranks: the two kernels are replaced by
    the oracle's order and torch indexing, the gathering is the product's."""
    os.environ["MASTER_ADDR"], os.environ["MASTER_PORT"] = "127.0.0.1", str(port)
    dist.init_process_group("gloo", rank=rank, world_size=world)
    try:
        n = 40
        sp = Splatter(S.make_scene("fwd_1k_128", n=n), device="cpu")
        sp.shard_optimizer(rank, world)
        sp.weight_sum = torch.arange(n, dtype=torch.float32) * (1.0 if rank == 0 else -2.0)
        lo, hi = sp._shard["lo"], sp._shard["hi"]
        sp.m_flat[lo:hi] = torch.arange(lo, hi, dtype=torch.float32)
        off = sp.flat_offsets["means"]
        seen = {}

        def select(score, protect, n_, n_keep, decisions, ws, stream=None):
            seen["score"] = score.tolist()
            decisions.copy_(torch.from_numpy(O.evict_select(score.numpy(), None, n_keep)))

        def compact(p, m_in, v_in, decisions, o, m_out, v_out, cap, ws, stream=None):
            rows = torch.nonzero(decisions)[:, 0]
            seen["m"] = sp.exp_avg["means"][rows].tolist()
            seen["rows"] = rows.tolist()

        api.gs_evict_select, api.gs_evict_compact = select, compact
        api.gs_get_status = lambda ws, stream=None: api.GS_OK
        d = sp.evict(10)
        out[rank] = dict(seen, d=d.tolist(), n=sp.n, off=off, sum=sp.weight_sum is None,
                         bounds=(sp._shard["lo"], sp._shard["hi"]), total=sp.flat_total)
    finally:
        dist.barrier()
        dist.destroy_process_group()


def test_ranks_evict_alike():
    with mp.Manager() as mgr:
        out = mgr.dict()
        mp.spawn(_evict_worker, args=(2, _free_port(), out), nprocs=2, join=True)
        a, b = out[0], out[1]
    assert a["score"] == b["score"] == [-float(i) for i in range(40)]
    assert a["rows"] == b["rows"] == list(range(10))
    assert a["d"] == b["d"] == [1] * 10 + [0] * 30
    # every rank holds every slice of the moments when the rows move
    assert a["m"] == b["m"] == [[a["off"] + 4.0 * i + c for c in range(4)] for i in range(10)]
    assert a["n"] == b["n"] == 10 and a["sum"] and b["sum"]
    assert a["bounds"][1] == b["bounds"][0] and b["bounds"][1] == b["total"] == a["total"]
