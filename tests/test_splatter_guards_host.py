"""What Splatter.accumulate_weights and Splatter.evict keep track of on the
host, with the C calls replaced by a log: which frame the buffers hold."""

import pytest
import torch

from gaussian_splatting_differentiable_ewa_b200 import api
from gaussian_splatting_differentiable_ewa_b200 import scenes as S
from gaussian_splatting_differentiable_ewa_b200.pipeline import Splatter

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
