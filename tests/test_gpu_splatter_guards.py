"""Accumulated weights and eviction through the Splatter on the GPU: frames that
graphs render or overwrite."""

import pytest
import torch

from gaussian_splatting_differentiable_ewa_b200 import api
from gaussian_splatting_differentiable_ewa_b200 import scenes as S
from gaussian_splatting_differentiable_ewa_b200.pipeline import Splatter

pytestmark = pytest.mark.gpu


def _splatter(n=2000, stream=None, **kw):
    sp = Splatter(S.make_scene("fwd_100k_800", n=n, width=160, height=120), stream=stream, **kw)
    torch.cuda.synchronize()
    sp.ensure_capacity()
    sp.rasterize_fwd()
    torch.cuda.synchronize()
    return sp


def test_weights_of_moved_parameters_want_their_own_render():
    """Parameters move, ensure_capacity finds room and writes their lists: the
    old frame's weights are gone, the new frame's come with its render."""
    sp = _splatter()
    first = sp.accumulate_weights(decay=0.0).clone()
    gen = sp._gen
    sp.means[:, 0] += 0.05
    sp.ensure_capacity()
    assert sp._gen == gen                      # nothing was reallocated
    with pytest.raises(ValueError, match="render"):
        sp.accumulate_weights(decay=0.0)
    sp.rasterize_fwd()
    second = sp.accumulate_weights(decay=0.0).clone()
    assert not torch.equal(first, second)
    # the weights and the transmittance of the new frame sum to one per pixel:
    # each of n_contrib entries is off by at most four roundings (2^-24)
    tol = float((sp.n_contrib.double() + 4).sum()) * 2.0 ** -22
    assert abs(float(second.double().sum() + sp.final_T.double().sum()) - sp.W * sp.H) <= tol


def test_replayed_calls_count_as_the_calls():
    sp = _splatter()
    want = sp.accumulate_weights(decay=0.0).clone()
    graphs = sp.capture_calls(torch.full_like(sp.image, 1e-3))
    torch.cuda.synchronize()
    assert torch.equal(sp.accumulate_weights(decay=0.0), want)
    for name in ("project", "bin_sort"):
        graphs[name].replay()
        with pytest.raises(ValueError, match="render"):
            sp.accumulate_weights(decay=0.0)
        graphs["bin_sort"].replay()
        graphs["rasterize_fwd"].replay()
        assert torch.equal(sp.accumulate_weights(decay=0.0), want)
        for after in ("rasterize_bwd", "project_bwd", "densify_stats"):
            graphs[after].replay()
            assert torch.equal(sp.accumulate_weights(decay=0.0), want)


def test_host_fed_paths_leave_a_frame():
    """train_from_host and render_to_host replay graphs of their own: their
    last frame can be weighed, after a call that had spoilt the one before."""
    stream = torch.cuda.Stream()
    sp = _splatter(stream=stream)
    shape = tuple(sp.image.shape)
    images = [torch.empty(shape).pin_memory() for _ in range(3)]
    grads = [torch.full(shape, 1e-4).pin_memory() for _ in range(3)]
    with torch.cuda.stream(stream):
        for run in (lambda: sp.render_to_host(images), lambda: sp.train_from_host(grads, images)):
            for _ in range(2):                 # the second time nothing is captured
                run()
                got = sp.accumulate_weights(decay=0.0).clone()
                torch.cuda.synchronize()
                total = float(got.double().sum() + sp.final_T.double().sum())
                tol = float((sp.n_contrib.double() + 4).sum()) * 2.0 ** -22
                assert abs(total - sp.W * sp.H) <= tol
                sp.project()
                with pytest.raises(ValueError, match="render"):
                    sp.accumulate_weights(decay=0.0)
    torch.cuda.synchronize()
    assert sp.status() == api.GS_OK and sp.weights_status() == api.GS_OK


def test_sums_and_maxima_tell_of_the_same_frames():
    """A call without `largest` after one with it forgets and adds the same in
    both scores."""
    sp = _splatter()
    pw = torch.zeros((1, sp.H, sp.W), device="cuda")
    pw[:, :, : sp.W // 2] = 1.0
    sp.accumulate_weights(pixel_weight=pw, largest=True)
    sums, tops = sp.weight_sum.clone(), sp.weight_max.clone()
    sp.accumulate_weights(pixel_weight=1.0 - pw, decay=0.25)
    ws = torch.zeros_like(sp._weights_ws)
    api.gs_blend_weights(sp.c_proj, sp.c_bins, sp.cams, sp.V, sp.n, sp.n_contrib, sums, ws,
                         weight_max=tops, warp_masks=sp.warp_masks, pixel_weight=1.0 - pw,
                         decay=0.25)
    assert torch.equal(sp.weight_sum, sums) and torch.equal(sp.weight_max, tops)
    # a sum holds its largest term but for its last roundings (2^-21 + 2^-23)
    assert torch.all(sp.weight_max <= sp.weight_sum * (1.0 + 2.0 ** -20))


def test_inputs_from_another_stream_are_waited_for():
    """A Splatter on a stream of its own, pixel weights, scores and protection
    still being computed on the caller's stream, and let go of after the call."""
    stream = torch.cuda.Stream()
    sp = _splatter(stream=stream)
    with torch.cuda.stream(stream):
        want = sp.accumulate_weights(decay=0.0).clone()
    torch.cuda.synchronize()

    def late(shape, dtype, value):
        t = torch.zeros(shape, dtype=dtype, device="cuda")
        torch.cuda._sleep(40_000_000)          # some 20 ms
        return t.copy_(value)

    shape = (sp.V, sp.H, sp.W)
    ones = torch.ones(shape, device="cuda")
    # the memory of weights let go of is not handed out while they are read
    for _ in range(3):
        got = sp.accumulate_weights(pixel_weight=late(shape, torch.float32, ones), decay=0.0)
        with torch.cuda.stream(stream):
            first = got.clone()
            torch.cuda._sleep(40_000_000)
        sp.accumulate_weights(pixel_weight=ones.clone(), decay=0.0)
        other = [torch.zeros(shape, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        assert torch.equal(first, want) and torch.equal(got, want) and not any(bool(o.any()) for o in other)
    n, keep = sp.n, 700
    values = torch.arange(n, dtype=torch.float32, device="cuda")
    marked = values < 3
    d = sp.evict(keep, score=late((n,), torch.float32, values),
                 protect=late((n,), torch.bool, marked))
    torch.cuda.synchronize()
    rows = torch.nonzero(d)[:, 0]
    assert torch.equal(rows, torch.cat([torch.arange(3, device="cuda"),
                                        torch.arange(n - keep + 3, n, device="cuda")]))
