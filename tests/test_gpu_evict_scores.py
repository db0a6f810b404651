"""Small accumulated weights, the ones that an eviction orders: every Gaussian's
score against float64 at its own size, however small the pixel weights are,
and totals as large as a call allows.

A call of P = n_views H W pixels adds up block sums in whole units of 2^-k, k the
largest for which P 2^k <= 2^64 - 2^54: a sum of 2^20 units or more is rounded
to them (2^-21 of it at most), a smaller one to 2^-32 of a unit, and from 2^-9
of a unit up that holds the float as it is."""

import numpy as np
import pytest
import torch

from gaussian_splatting_differentiable_ewa_b200 import api
from gaussian_splatting_differentiable_ewa_b200 import scenes as S
from gaussian_splatting_differentiable_ewa_b200.pipeline import Splatter
from oracle import oracle as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _units(pixels):
    k = 63
    while pixels << k > 2 ** 64 - 2 ** 54:
        k -= 1
    return k


def _frame(name, **kw):
    sp = Splatter(S.make_scene(name, **kw))
    sp.ensure_capacity()
    sp.rasterize_fwd()
    torch.cuda.synchronize()
    assert sp.status() == api.GS_OK
    return sp


def _weights(proj, bins, cams, views, n, n_contrib, masks, pixel_weight=None):
    total = torch.full((n,), float("nan"), device="cuda")
    top = torch.full((n,), float("nan"), device="cuda")
    ws = torch.zeros(api.gs_blend_weights_workspace_size(n) // 8, dtype=torch.int64,
                     device="cuda")
    api.gs_blend_weights(proj, bins, cams, views, n, n_contrib, total, ws, weight_max=top,
                         warp_masks=masks, pixel_weight=pixel_weight, decay=0.0)
    assert api.gs_get_status(ws) == api.GS_OK
    return total, top


def _of(sp, pixel_weight=None, masks=True):
    return _weights(sp.c_proj, sp.c_bins, sp.cams, sp.V, sp.n, sp.n_contrib,
                    sp.warp_masks if masks else None, pixel_weight)


FRAMES = [("fwd_1k_128", dict()),
          ("fwd_100k_800", dict(n=3000, width=200, height=152)),
          ("train_6m_8x1080p", dict(n=2500, n_views=3, width=100, height=70))]


@pytest.mark.parametrize("name,kw", FRAMES)
@pytest.mark.parametrize("scale", [None, 1e-4, 1e-6, 1e-12])
def test_small_weights_at_their_own_size(name, kw, scale):
    """|gpu - float64| within the float32 walk's own bound for the Gaussian
    (oracle.blend_weights), its block sums' rounding (2^-21 of each, or half of
    2^-(k + 32) for every block of the frame, below 2^-60 in all) and the last
    rounding."""
    sp = _frame(name, **kw)
    pw = None
    if scale is not None:
        g = np.random.default_rng(5)
        pw = torch.from_numpy((scale * g.random((sp.V, sp.H, sp.W))).astype(np.float32)).cuda()
    want, _, slack = O.blend_weights(
        sp.records.cpu().numpy(), sp.ids.cpu().numpy().view(np.uint32), sp.ranges.cpu().numpy(),
        sp.n_contrib.cpu().numpy(), sp.W, sp.H, None if pw is None else pw.cpu().numpy())
    half = 4 * sp.ranges.shape[0] * 2.0 ** -(_units(sp.V * sp.H * sp.W) + 33)
    assert half <= 2.0 ** -60
    tol = slack + half + (2.0 ** -21 + U) * want
    for masks in (True, False):
        total, top = _of(sp, pw, masks)
        total = total.cpu().numpy()
        assert np.all(np.abs(total - want) <= tol)
        seen = want > tol
        assert seen.sum() > 0.3 * sp.n and np.all(total[seen] > 0)
        assert np.array_equal(total > 0, top.cpu().numpy() > 0)


@pytest.mark.parametrize("name,kw", FRAMES + [
    ("fwd_100k_800", dict(n=5000, width=3840, height=2160))])
def test_scores_scale_with_the_pixel_weights(name, kw):
    """A pixel weight of 2^-j scales every float of the walk exactly, so that the
    scores are the unweighted ones times 2^-j, but for the rounding of the block
    sums on either side (2^-21; the least of them, 1e-4 / 255 > 2^-22 times
    2^-20, is above 2^-9 units) and the last one's."""
    sp = _frame(name, **kw)
    assert 2.0 ** -42 > 2.0 ** -(_units(sp.V * sp.H * sp.W) + 9)
    base, top = _of(sp)
    assert float(base.max()) > 0
    for j in (3, 12, 20):
        pw = torch.full((sp.V, sp.H, sp.W), 2.0 ** -j, device="cuda")
        s, t = _of(sp, pw)
        s, t = s.double() * 2.0 ** j, t.double() * 2.0 ** j
        assert torch.all((s - base.double()).abs() <= 2 * (2.0 ** -21 + U) * base.double())
        assert torch.equal(t, top.double()) and torch.equal(s > 0, base > 0)


def _flat(views, width, height, per_tile=1, ids=1):
    """Every tile lists `per_tile` splats that weigh 0.99 of what is left at
    every pixel: w1 = w2 = 0, 2^8 / 255 clamped."""
    rec = torch.zeros((views, ids, 16), device="cuda")
    rec[:, :, 8] = -8.0
    sc = S.make_scene("fwd_1k_128", n=1)
    c = sc.cameras[0]
    c.width, c.height = width, height
    tiles = views * (-(-width // 16)) * (-(-height // 16))
    edge = torch.arange(tiles + 1, device="cuda") * per_tile
    ranges = torch.stack([edge[:-1], edge[1:]], 1).contiguous()
    lists = torch.zeros(tiles * per_tile, dtype=torch.int32, device="cuda")
    return dict(rec=rec, lists=lists, ranges=ranges,
                proj=api.projected(rec, None, None),
                bins=api.binned(lists, ranges, None, lists.numel()),
                cams=api.cameras([c] * views),
                masks=torch.full((tiles * per_tile,), 15, dtype=torch.uint8, device="cuda"),
                nc=torch.full((views, height, width), per_tile, dtype=torch.int32,
                              device="cuda"))


@pytest.mark.parametrize("views,width,height", [(1, 1, 1), (1, 64, 64), (1, 4096, 2048),
                                                (32, 8192, 8192)])
def test_the_largest_totals_fit(views, width, height):
    """One splat over every pixel at 0.99, up to the 2^31 pixels of the largest
    call. P is a power of two, so every partial sum of equal floats is exact."""
    f = _flat(views, width, height)
    total, top = _weights(f["proj"], f["bins"], f["cams"], views, 1, f["nc"], f["masks"])
    a = float(np.float32(0.99))
    assert float(total) == a * views * width * height and float(top) == a


def test_a_gaussian_listed_many_times_in_a_tile():
    """A list that names one Gaussian 40 times: its weights per pixel are
    1 - 0.01^40 in all, the late ones far below one unit of the coarse total."""
    f = _flat(2, 64, 48, per_tile=40)
    total, top = _weights(f["proj"], f["bins"], f["cams"], 2, 1, f["nc"], f["masks"])
    P = 2 * 64 * 48
    # alpha is 0.99 rounded, so T falls by 1 - alpha = 0.01 (1 +- 99 u) per
    # entry; four roundings per entry and twelve per sum
    assert abs(float(total) - P) <= P * U * (4 * 40 + 12)
    assert float(top) == float(np.float32(0.99))
