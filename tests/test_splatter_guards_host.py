"""What Splatter.accumulate_weights and Splatter.evict keep track of on the
host, with the C calls replaced: which frame the buffers hold, which scores are
kept up, and what several ranks agree on before they evict."""

import datetime
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

CALLS = ("gs_project", "gs_bin_sort", "gs_rasterize_fwd", "gs_rasterize_bwd", "gs_densify_stats",
         "gs_project_bwd_adam", "gs_adam_step", "gs_l1_dssim", "gs_blend_weights")


@pytest.fixture
def logged(monkeypatch):
    """A Splatter on the CPU whose C calls only append (name, keywords)."""
    log = []
    for name in CALLS:
        monkeypatch.setattr(api, name, lambda *a, _n=name, **k: log.append((_n, k)))
    monkeypatch.setattr(api, "gs_get_status", lambda ws, stream=None: api.GS_OK)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda *a, **k: None)
    return Splatter(S.make_scene("fwd_1k_128", n=50), device="cpu"), log


def test_new_lists_beside_an_old_frame_are_refused(logged):
    """project, bin_sort and ensure_capacity (the pairs fit: nothing is
    reallocated) write the records and lists of other parameters beside the
    last render's n_contrib; every render makes a frame again."""
    sp, log = logged
    dL = torch.zeros_like(sp.image)
    renders = (sp.forward, sp.rasterize_fwd, lambda: sp.train_step(dL),
               lambda: sp.train_step_target(sp.image))
    for render in renders:
        for spoil in (sp.project, sp.bin_sort, sp.ensure_capacity):
            render()
            sp.accumulate_weights()
            spoil()
            before = len(log)
            with pytest.raises(ValueError, match="render"):
                sp.accumulate_weights()
            assert len(log) == before  # nothing was enqueued
    sp.rasterize_fwd()
    sp.accumulate_weights()
    assert log[-1][0] == "gs_blend_weights"


def test_maxima_once_kept_are_kept_up(logged):
    """From the first call with largest=True on, every call decays and raises
    the maxima as it does the sums."""
    sp, log = logged
    sp.rasterize_fwd()
    sp.accumulate_weights(decay=0.5)
    assert sp.weight_max is None and log[-1][1]["weight_max"] is None
    sp.accumulate_weights(decay=0.5, largest=True)
    kept = sp.weight_max
    assert kept is not None and log[-1][1]["weight_max"] is kept
    sp.accumulate_weights(decay=0.5)
    assert sp.weight_max is kept and log[-1][1]["weight_max"] is kept
    assert log[-1][1]["decay"] == 0.5


def _free_port() -> int:
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        return s.getsockname()[1]


def _rank_worker(rank, world, port, out):
    """Evictions that one rank cannot take, then one whose status is an error,
    then the same again: the kernels replaced by the oracle's order."""
    os.environ["MASTER_ADDR"], os.environ["MASTER_PORT"] = "127.0.0.1", str(port)
    dist.init_process_group("gloo", rank=rank, world_size=world,
                            timeout=datetime.timedelta(seconds=20))
    n, status, seen = 40, [api.GS_OK], {}

    def select(score, protect, n_, n_keep, decisions, ws, stream=None):
        seen["score"] = score.tolist()
        decisions.copy_(torch.from_numpy(O.evict_select(score.numpy(), None, n_keep)))

    api.gs_evict_select = select
    api.gs_evict_compact = lambda *a, **k: None
    api.gs_get_status = lambda ws, stream=None: status[0]
    sp = Splatter(S.make_scene("fwd_1k_128", n=n), device="cpu")
    sp.shard_optimizer(rank, world)
    mine = torch.arange(n, dtype=torch.float32) * (1.0 if rank == 0 else -2.0)
    first = rank == 0

    def refused(*a, **k):
        try:
            sp.evict(*a, **k)
        except ValueError as e:
            return str(e)
        return None

    # no rank, then only the first one has accumulated weights
    raised = [refused(10)]
    sp.weight_sum = mine.clone() if first else None
    raised.append(refused(10))
    sp.weight_sum = mine.clone()
    # a budget, a score or a protection that only one rank has, or has wrong
    raised += [refused(10 if first else 0), refused(10 if first else 11),
               refused(10, score=mine if first else None),
               refused(10, score=mine if first else mine[:3]),
               refused(10, protect=torch.zeros(n, dtype=torch.uint8) if first else None)]
    kept = torch.equal(sp.weight_sum, mine)
    # selection reports an error on every rank: their own totals stay
    status[0] = api.GS_ERR_DEVICE_TIMEOUT
    try:
        sp.evict(10)
        failed = False
    except api.GsError:
        failed = True
    kept = kept and torch.equal(sp.weight_sum, mine)
    status[0] = api.GS_OK
    # a score and an optimiser of its own: no rank waits for another
    alone = Splatter(S.make_scene("fwd_1k_128", n=n + rank), device="cpu")
    if first:
        alone.evict(10, score=torch.arange(n + rank, dtype=torch.float32))
    d = sp.evict(10)
    out.put((rank, dict(raised=raised, kept=kept, failed=failed, d=d.tolist(), n=sp.n,
                        score=seen["score"])))
    dist.barrier()
    dist.destroy_process_group()


def test_ranks_refuse_and_retry_alike():
    ctx = mp.get_context("spawn")
    out = ctx.SimpleQueue()
    mp.spawn(_rank_worker, args=(2, _free_port(), out), nprocs=2, join=True)
    got = dict(out.get() for _ in range(2))
    for rank in range(2):
        r = got[rank]
        assert all(r["raised"]), r["raised"]
        assert "accumulate_weights" in r["raised"][0]
        assert r["kept"] and r["failed"] and r["n"] == 10
        assert r["score"] == [-float(i) for i in range(40)]
        assert r["d"] == np.repeat([1, 0], [10, 30]).tolist()
