"""Eviction on the GPU: accumulated blending weights against a float64 walk of
the same records and lists (and against the rasteriser's own backward), the
survivors against a sort of tuples, the compaction against indexing.

Bars. weight_sum: |gpu - float64| <= slack, the walk's own error bound
(oracle.blend_weights), plus the fixed-point rounding (2^-33 for each of a
tile's four 8 x 8 blocks) and the last rounding (2^-24 relative, of the decayed sum too). weight_max: within the
same slack. Decisions, sources and rows: equal."""

import numpy as np
import pytest
import torch

from gaussian_splatting_differentiable_ewa_b200 import api
from gaussian_splatting_differentiable_ewa_b200 import scenes as S
from gaussian_splatting_differentiable_ewa_b200.pipeline import Splatter
from oracle import oracle as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _ws(nbytes):
    return torch.zeros(-(-nbytes // 8), dtype=torch.int64, device="cuda")


def _frame(name="fwd_100k_800", **kw):
    sp = Splatter(S.make_scene(name, **kw))
    sp.ensure_capacity()
    sp.rasterize_fwd()
    torch.cuda.synchronize()
    assert sp.status() == api.GS_OK
    return sp


def _weights(sp, masks=True, pixel_weight=None, decay=0.0, total=None, top=None, ws=None,
             stream=None):
    total = torch.full((sp.n,), float("nan"), device="cuda") if total is None else total
    top = torch.full((sp.n,), float("nan"), device="cuda") if top is None else top
    ws = _ws(api.gs_blend_weights_workspace_size(sp.n)) if ws is None else ws
    api.gs_blend_weights(sp.c_proj, sp.c_bins, sp.cams, sp.V, sp.n, sp.n_contrib, total, ws,
                         weight_max=top, warp_masks=sp.warp_masks if masks else None,
                         pixel_weight=pixel_weight, decay=decay, stream=stream)
    return total, top, ws


def _reference(sp, pixel_weight=None):
    return O.blend_weights(sp.records.cpu().numpy(), sp.ids.cpu().numpy().view(np.uint32),
                           sp.ranges.cpu().numpy(), sp.n_contrib.cpu().numpy(), sp.W, sp.H,
                           None if pixel_weight is None else pixel_weight.cpu().numpy())


def _pixel_weights(sp, seed):
    """An error map with everything the call has to take: zeros, negatives,
    values above one, NaN and infinities, one tile without any weight."""
    g = np.random.default_rng(seed)
    m = g.random((sp.V, sp.H, sp.W)).astype(np.float32)
    m[g.random(m.shape) < 0.3] = 0.0
    for val in (-1.0, 2.5, np.nan, np.inf, -np.inf, -0.0):
        m[g.random(m.shape) < 0.02] = val
    m[:, :16, :16] = 0.0
    return torch.from_numpy(m).cuda()


CASES = [
    ("fwd_1k_128", dict(), True, False, 0.0),
    ("fwd_1k_128", dict(n=1), True, False, 0.0),
    ("fwd_100k_800", dict(n=3000, width=200, height=152), True, False, 1.0),
    ("fwd_100k_800", dict(n=700, width=37, height=29), False, False, 0.0),
    ("fwd_100k_800", dict(n=900, width=1, height=1), True, False, 0.5),
    ("train_6m_8x1080p", dict(n=2500, n_views=3, width=100, height=70), False, True, 0.9),
    ("train_6m_8x1080p", dict(n=2500, n_views=2, width=129, height=65), True, True, 0.0),
]


@pytest.mark.parametrize("name,kw,masks,weighted,decay", CASES)
def test_weights_match_the_float64_walk(name, kw, masks, weighted, decay):
    sp = _frame(name, **kw)
    pw = _pixel_weights(sp, 3) if weighted else None
    want, want_top, slack = _reference(sp, pw)
    old, old_top = np.zeros(sp.n), np.zeros(sp.n)
    total = top = None
    if decay > 0:
        g = np.random.default_rng(8)
        old = g.random(sp.n).astype(np.float32) * 5
        old_top = g.random(sp.n).astype(np.float32) * 0.2
        total, top = torch.from_numpy(old.copy()).cuda(), torch.from_numpy(old_top.copy()).cuda()
    total, top, ws = _weights(sp, masks, pw, decay, total, top)
    assert api.gs_get_status(ws) == api.GS_OK
    tiles = sp.ranges.shape[0]
    exp = np.float64(np.float32(decay)) * old + want
    tol = slack + 4 * tiles * 2.0 ** -33 + U * exp
    assert np.all(np.abs(total.cpu().numpy() - exp) <= tol)
    exp_top = np.maximum(np.float64(np.float32(decay)) * old_top, want_top)
    assert np.all(np.abs(top.cpu().numpy() - exp_top) <= slack + 2 * U * exp_top)
    assert want.max() > 0


def test_weights_and_transmittance_sum_to_one():
    sp = _frame(n=3000, width=200, height=152)
    total, _, _ = _weights(sp)
    # per pixel at most 2u per entry off one, n_contrib entries
    tol = float((sp.n_contrib.double() + 4).sum()) * 2 * U * 2
    assert abs(float(total.double().sum() + sp.final_T.double().sum()) - sp.W * sp.H) <= tol


@pytest.mark.parametrize("V", [1, 3])
def test_weights_are_the_colour_gradient_of_a_unit_upstream(V):
    """With dL/dimage = 1 in the red plane, dL/dred of a Gaussian is the sum of
    its weights: the backward's own walk (back to front) against this one."""
    sp = _frame("train_6m_8x1080p", n=4000, n_views=V, width=180, height=100)
    dL = torch.zeros_like(sp.image)
    dL[:, 0] = 1.0
    sp.rasterize_bwd(dL, with_params=False)
    want = sp.grad2d[:, :, 6].double().sum(0)
    total, _, _ = _weights(sp)
    err = (total.double() - want).norm() / want.norm()
    # the backward divides by (1 - alpha) to recover T: its stated bar
    assert float(err) <= 1e-4


def test_masks_do_not_change_a_bit_and_calls_repeat():
    sp = _frame(n=5000, width=300, height=211)
    a = _weights(sp, masks=True)
    b = _weights(sp, masks=False)
    c = _weights(sp, masks=True)
    for x, y, z in zip(a[:2], b[:2], c[:2]):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_without_maximum_and_decay_semantics():
    sp = _frame("fwd_1k_128")
    base, _, ws = _weights(sp)
    s = torch.full((sp.n,), float("nan"), device="cuda")
    args = (sp.c_proj, sp.c_bins, sp.cams, sp.V, sp.n, sp.n_contrib, s, ws)
    api.gs_blend_weights(*args, warp_masks=sp.warp_masks, decay=0.0)   # overwrites NaN
    assert torch.equal(s, base)
    api.gs_blend_weights(*args, warp_masks=sp.warp_masks, decay=1.0)
    # the double sum rounded once: twice the fixed-point total within its last bit
    assert torch.all((s.double() - 2 * base.double()).abs() <= 4 * U * base.double())
    # kept maxima below zero or NaN count as zero
    t = torch.full((sp.n,), float("nan"), device="cuda")
    t[::2] = -3.0
    s2 = torch.zeros(sp.n, device="cuda")
    api.gs_blend_weights(*args[:6], s2, ws, weight_max=t, decay=1.0)
    assert torch.equal(t, _weights(sp)[1])


def test_empty_frames_and_single_sides():
    """No Gaussian in view, no pairs, a mask that leaves nothing: zeros (or the
    decayed sums), and nothing written behind the arrays."""
    sc = S.make_scene("fwd_1k_128", n=40)
    sc.means[:, 2] = -5.0                      # all behind the camera
    sp = Splatter(sc)
    sp.ensure_capacity()
    sp.rasterize_fwd()
    buf = torch.full((sp.n + 8,), 7.0, device="cuda")
    _weights(sp, total=buf[:sp.n], decay=0.5)
    assert torch.all(buf[:sp.n] == 3.5) and torch.all(buf[sp.n:] == 7.0)
    sp = _frame("fwd_1k_128")
    zero = torch.zeros((1, 128, 128), device="cuda")
    for pw in (zero, zero + float("nan"), zero - 1.0):
        s, t, _ = _weights(sp, pixel_weight=pw)
        assert not s.any() and not t.any()


@pytest.mark.parametrize("masks", [True, False])
def test_weights_conditions_are_reported(masks):
    """A list entry naming no Gaussian and a range past the ids are clipped and
    reported, with the forward's masks and without."""
    sp = _frame("fwd_1k_128")
    want, _, ws = _weights(sp)
    ids, ranges = sp.ids.clone(), sp.ranges.clone()
    busy = int(torch.argmax(sp.ranges[:, 1] - sp.ranges[:, 0]))
    bins = api.binned(ids, ranges, sp.n_pairs, sp.capacity)
    s = torch.zeros(sp.n, device="cuda")

    def call(b):
        api.gs_blend_weights(sp.c_proj, b, sp.cams, sp.V, sp.n, sp.n_contrib, s, ws, decay=0.0,
                             warp_masks=sp.warp_masks if masks else None)
        return api.gs_get_status(ws)

    first = int(ranges[busy, 0])
    gone = int(ids[first]) & 0xFFFFFFFF
    ids[first] = -1
    assert call(bins) == api.GS_ERR_OVERFLOW
    other = torch.ones(sp.n, dtype=torch.bool, device="cuda")
    other[gone] = False
    assert float(s[gone]) <= float(want[gone]) and torch.all(s[other] >= want[other] - 1e-3)
    ids[first] = gone
    ranges[busy, 1] = sp.capacity + 1
    assert call(bins) == api.GS_ERR_OVERFLOW
    assert float(s.sum()) < float(want.sum())
    ranges[busy, 1] = sp.ranges[busy, 1]
    assert call(bins) == api.GS_OK and torch.equal(s, want)


def _scores(kind, n, seed=0):
    g = np.random.default_rng(seed)
    if kind == "equal":
        return np.full(n, 0.25, np.float32)
    s = np.exp(2 * g.normal(size=n)).astype(np.float32)
    if kind == "ties":
        s[g.random(n) < 0.6] = 0.0
        s[g.random(n) < 0.2] = 1.0
    if kind == "wild":
        s *= np.where(g.random(n) < 0.5, -1, 1).astype(np.float32)
        for v in (0.0, -0.0, np.nan, np.inf, -np.inf, 1e-42, -1e-42, 3.4e38):
            s[g.random(n) < 0.05] = v
        s.view(np.uint32)[g.random(n) < 0.03] = 0xFFC00001   # a NaN with its sign set
    return s


@pytest.mark.parametrize("n", [1, 2, 31, 256, 1023, 1025, 5000, 60001])
@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "wild"])
def test_survivors_match_the_sorted_order(n, kind):
    s = _scores(kind, n, n)
    g = np.random.default_rng(n + 1)
    ws = _ws(api.gs_evict_workspace_size(n))
    # odd addresses: one float, three and one byte off
    score = torch.empty(n + 1, device="cuda")[1:]
    score.copy_(torch.from_numpy(s))
    d = torch.full((n + 11,), 9, dtype=torch.int8, device="cuda")
    masks = [None, (g.random(n) < 0.1).astype(np.uint8) * 200, np.ones(n, np.uint8)]
    for protect in masks:
        p = None
        if protect is not None:
            p = torch.empty(n + 3, dtype=torch.uint8, device="cuda")[3:]
            p.copy_(torch.from_numpy(protect))
        for keep in sorted({0, 1, n // 3, (9 * n) // 10, n - 1, n, n + 5}):
            api.gs_evict_select(score, p, n, keep, d[1:n + 1], ws)
            got = d.cpu().numpy()
            assert np.array_equal(got[1:n + 1], O.evict_select(s, protect, keep)), (keep, p)
            assert got[0] == 9 and np.all(got[n + 1:] == 9)
    assert api.gs_get_status(ws) == api.GS_OK


@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("n,keep", [(131_072, 70_000), (131_073, 131_072), (200_003, 1),
                                    (3_000_001, 1_000_003), (2_097_152, 2_097_151)])
def test_survivors_of_large_sets_with_ties(n, keep, off):
    """Equal scores by the million at the threshold: the lowest indices, across
    blocks, on aligned and on odd addresses."""
    g = torch.Generator(device="cuda").manual_seed(n)
    score = torch.rand(n + off, generator=g, device="cuda")[off:]
    score[torch.rand(n, generator=g, device="cuda") < 0.8] = 0.0
    protect = (torch.rand(n + off, generator=g, device="cuda") < 0.1).to(torch.uint8)[off:]
    d = torch.empty(n + off, dtype=torch.int8, device="cuda")[off:]
    ws = _ws(api.gs_evict_workspace_size(n))
    for p in (None, protect):
        api.gs_evict_select(score, p, n, keep, d, ws)
        s = score if p is None else torch.where(p != 0, torch.inf, score)
        best = torch.sort(s, descending=True, stable=True).indices[:keep]
        want = torch.zeros_like(d)
        want[best] = 1
        assert torch.equal(d, want)
    assert api.gs_get_status(ws) == api.GS_OK
    best = torch.sort(score, descending=True, stable=True).indices[:keep]
    api.gs_evict_select(score, None, n, keep, d, ws)
    want = torch.zeros_like(d)
    want[best] = 1
    assert torch.equal(d, want)


def test_selection_that_waits_in_vain_is_reported():
    """A block of the large selection that never comes to the barrier: the
    others give up in time, and the next call is normal."""
    n = 300_000
    score = torch.arange(n, dtype=torch.float32, device="cuda")
    d = torch.empty(n, dtype=torch.int8, device="cuda")
    ws = _ws(api.gs_evict_workspace_size(n))
    try:
        api.gs_debug_stall(api.GS_STALL_SORT_LOOKBACK, 5, 0.05)
        api.gs_evict_select(score, None, n, n // 2, d, ws)
        assert api.gs_get_status(ws) == api.GS_ERR_DEVICE_TIMEOUT
    finally:
        api.gs_debug_stall(api.GS_STALL_NONE)
    api.gs_evict_select(score, None, n, n // 2, d, ws)
    assert api.gs_get_status(ws) == api.GS_OK
    assert not d[:n // 2].any() and torch.all(d[n // 2:] == 1)


def _sets(n, K, count, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shapes = [(4,), (4,), (4,), (), (K, 3)]
    return [[torch.randn((n,) + s, generator=g, device="cuda") for s in shapes]
            for _ in range(count)]


def _compact(ins, deg, d, cap, guard=3, source=True):
    """gs_evict_compact into arrays with `guard` rows behind the capacity."""
    n = ins[0][0].shape[0]
    outs = [[torch.full((cap + guard,) + x.shape[1:], 5.0, device="cuda") for x in a]
            for a in ins]
    src = torch.full((cap + guard,), -7, dtype=torch.int32, device="cuda")
    n_out = torch.full((1,), -1, dtype=torch.int64, device="cuda")
    ws = _ws(api.gs_evict_workspace_size(n))
    gr = [api.grads(*a) for a in ins[1:]] or [None, None]
    go = [api.grads(*a) for a in outs] + [None, None]
    api.gs_evict_compact(api.params(*ins[0], deg), gr[0], gr[1], d, go[0], go[1], go[2], cap, ws,
                         source=src if source else None, n_out=n_out)
    return outs, src, int(n_out.item()), api.gs_get_status(ws)


@pytest.mark.parametrize("n", [1, 255, 1024, 1025, 40_003])
@pytest.mark.parametrize("deg,count", [(0, 3), (1, 1), (2, 3), (3, 3)])
def test_compaction_equals_indexing(n, deg, count):
    ins = _sets(n, (deg + 1) ** 2, count, seed=n + deg)
    g = torch.Generator(device="cuda").manual_seed(n)
    for share in (0.0, 0.1, 0.85, 1.0):
        d = (torch.rand(n, generator=g, device="cuda") < share).to(torch.int8)
        rows = torch.nonzero(d)[:, 0]
        m = rows.numel()
        outs, src, n_out, st = _compact(ins, deg, d, m)
        assert st == api.GS_OK and n_out == m
        assert torch.equal(src[:m].long(), rows) and torch.all(src[m:] == -7)
        for a, b in zip(ins, outs):
            for x, y in zip(a, b):
                assert torch.equal(y[:m], x[rows])
                assert torch.all(y[m:] == 5.0)       # rows behind the last stay


def test_compaction_capacity_any_nonzero_and_empty():
    n = 5000
    ins = _sets(n, 4, 3)
    d = torch.zeros(n, dtype=torch.int8, device="cuda")
    d[10:4000] = -1
    d[17] = 3
    outs, src, n_out, st = _compact(ins, 1, d, 1500)
    assert st == api.GS_ERR_CAPACITY and n_out == 3990
    assert torch.equal(src[:1500].long(), torch.arange(10, 1510, device="cuda"))
    for a, b in zip(ins, outs):
        for x, y in zip(a, b):
            assert torch.equal(y[:1500], x[10:1510]) and torch.all(y[1500:] == 5.0)
    _, src, n_out, st = _compact(ins, 1, d, 0)                     # no room at all
    assert st == api.GS_ERR_CAPACITY and n_out == 3990 and torch.all(src == -7)
    outs, _, n_out, st = _compact(ins, 1, d, 4100, source=False)   # room to spare
    assert st == api.GS_OK and n_out == 3990
    assert torch.equal(outs[2][4][:3990], ins[2][4][10:4000])
    assert torch.all(outs[2][4][3990:] == 5.0)
    # no Gaussian: the count alone
    empty = [[x[:0] for x in a] for a in ins]
    _, _, n_out, st = _compact(empty, 1, d, 0)
    assert n_out == 0 and st == api.GS_OK


def test_captured_and_replayed_with_new_values():
    """One graph of weights, selection and compaction, replayed after the scores
    and decisions' inputs changed, equals the calls."""
    sp = _frame("fwd_1k_128")
    n, keep = sp.n, 640
    total = torch.zeros(n, device="cuda")
    top = torch.zeros(n, device="cuda")
    ws, ws2 = _ws(api.gs_blend_weights_workspace_size(n)), _ws(api.gs_evict_workspace_size(n))
    pw = torch.ones((1, 128, 128), device="cuda")
    d = torch.empty(n, dtype=torch.int8, device="cuda")
    ins = [[t for _, t in sp.param_list]]
    out = [torch.empty((keep,) + t.shape[1:], device="cuda") for t in ins[0]]
    p, go = api.params(*ins[0], 0), api.grads(*out)

    def calls(stream):
        _weights(sp, pixel_weight=pw, total=total, top=top, ws=ws, stream=stream)
        api.gs_evict_select(total, None, n, keep, d, ws2, stream=stream)
        api.gs_evict_compact(p, None, None, d, go, None, None, keep, ws2, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        calls(side)
    for k in range(3):
        pw.copy_((torch.arange(128 * 128, device="cuda").view(1, 128, 128) % (k + 2) == 0).float())
        g.replay()
        torch.cuda.synchronize()
        s, dd, oo = total.clone(), d.clone(), [x.clone() for x in out]
        calls(None)
        torch.cuda.synchronize()
        assert torch.equal(s, total) and torch.equal(dd, d)
        assert all(torch.equal(x, y) for x, y in zip(oo, out))
        assert np.array_equal(dd.cpu().numpy(), O.evict_select(s.cpu().numpy(), None, keep))


@pytest.mark.parametrize("n", [9000, 150_000, 700_001])
def test_large_sets_captured_and_replayed(n):
    """Selection by the grid and compaction behind its counts in one graph,
    replayed with new scores (ties among them) and new rows."""
    keep = (2 * n) // 3
    score = torch.zeros(n, device="cuda")
    d = torch.empty(n, dtype=torch.int8, device="cuda")
    ws = _ws(api.gs_evict_workspace_size(n))
    ins = _sets(n, 1, 3)
    outs = [[torch.empty((keep,) + x.shape[1:], device="cuda") for x in a] for a in ins]
    src = torch.empty(keep, dtype=torch.int32, device="cuda")
    p, gi, go = api.params(*ins[0], 0), [api.grads(*a) for a in ins], [api.grads(*a) for a in outs]
    side = torch.cuda.Stream()

    def calls():
        api.gs_evict_select(score, None, n, keep, d, ws, stream=side)
        api.gs_evict_compact(p, gi[1], gi[2], d, go[0], go[1], go[2], keep, ws, source=src,
                             stream=side)

    torch.cuda.synchronize()
    calls()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        calls()
    gen = torch.Generator(device="cuda").manual_seed(n)
    for share in (0.0, 0.5, 1.0):
        score.copy_(torch.rand(n, generator=gen, device="cuda"))
        score[torch.rand(n, generator=gen, device="cuda") < share] = 0.0
        for a in ins:
            for x in a:
                x.add_(1.0)
        g.replay()
        torch.cuda.synchronize()
        rows = torch.sort(score, descending=True, stable=True).indices[:keep].sort().values
        assert torch.equal(src.long(), rows)
        for a, b in zip(ins, outs):
            assert all(torch.equal(y, x[rows]) for x, y in zip(a, b))
    assert api.gs_get_status(ws) == api.GS_OK


def test_two_streams_with_their_own_workspaces():
    n = 200_000
    g = torch.Generator(device="cuda").manual_seed(1)
    scores = [torch.rand(n, generator=g, device="cuda") for _ in range(2)]
    want = []
    for s in scores:
        w = torch.zeros(n, dtype=torch.int8, device="cuda")
        w[torch.sort(s, descending=True, stable=True).indices[:n // 2]] = 1
        want.append(w)
    d = [torch.empty(n, dtype=torch.int8, device="cuda") for _ in range(2)]
    ws = [_ws(api.gs_evict_workspace_size(n)) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for k in range(2):
            api.gs_evict_select(scores[k], None, n, n // 2, d[k], ws[k], stream=streams[k])
    torch.cuda.synchronize()
    assert torch.equal(d[0], want[0]) and torch.equal(d[1], want[1])


def test_large_selections_side_by_side():
    """Grids that wait for their own blocks, on streams of different priority,
    beside one another and beside other work: all finish, none gives up."""
    n = 3_000_000
    g = torch.Generator(device="cuda").manual_seed(2)
    scores = [torch.rand(n, generator=g, device="cuda") for _ in range(3)]
    want = []
    for s in scores:
        w = torch.zeros(n, dtype=torch.int8, device="cuda")
        w[torch.sort(s, descending=True, stable=True).indices[:n // 3]] = 1
        want.append(w)
    d = [torch.empty(n, dtype=torch.int8, device="cuda") for _ in range(3)]
    ws = [_ws(api.gs_evict_workspace_size(n)) for _ in range(3)]
    streams = [torch.cuda.Stream(priority=p) for p in (0, -1, 0)]
    busy = torch.cuda.Stream(priority=-1)
    filler = torch.zeros(1 << 24, device="cuda")
    torch.cuda.synchronize()
    for _ in range(30):
        for k in range(3):
            api.gs_evict_select(scores[k], None, n, n // 3, d[k], ws[k], stream=streams[k])
        with torch.cuda.stream(busy):
            filler.add_(1.0)
    torch.cuda.synchronize()
    for k in range(3):
        assert api.gs_get_status(ws[k], streams[k]) == api.GS_OK
        assert torch.equal(d[k], want[k])


def test_splatter_wants_a_frame_of_the_current_set():
    sp = _frame("fwd_1k_128")
    sp.accumulate_weights()
    sp.evict(500)
    with pytest.raises(ValueError, match="render"):
        sp.accumulate_weights()
    sp.ensure_capacity()
    sp.rasterize_fwd()
    assert float(sp.accumulate_weights().sum()) > 0 and sp.weights_status() == api.GS_OK


@pytest.mark.parametrize("bits", [None, 8, 16])
@pytest.mark.parametrize("own_stream", [False, True])
def test_splatter_evicts_what_it_draws_on_least(bits, own_stream):
    """Train, accumulate over two frames, evict, train on: the survivors are the
    heaviest by the accumulated weight, with their parameters and moments, and
    the frame changes by what the evicted ones weighed."""
    stream = torch.cuda.Stream() if own_stream else None
    sc = S.make_scene("fwd_100k_800", n=4000, width=160, height=120)
    sp = Splatter(sc, sh_bits=bits, stream=stream)
    torch.cuda.synchronize()
    sp.ensure_capacity()
    dL = torch.full_like(sp.image, 1e-3)
    torch.cuda.synchronize()
    for _ in range(2):
        sp.train_step(dL)
    sp.forward()
    torch.cuda.synchronize()
    first = sp.accumulate_weights(largest=True).clone() if stream is None else None
    if stream is not None:
        sp.accumulate_weights(largest=True)
    sp.accumulate_weights(pixel_weight=None, decay=0.5, largest=True)
    torch.cuda.synchronize()
    assert sp.weights_status() == api.GS_OK
    w = sp.weight_sum.clone()
    if first is not None:
        assert torch.all((w - 1.5 * first).abs() <= 4 * U * w)
    before = sp.image.clone()
    if bits is not None:
        sp.refresh_sh_float()          # sp.sh is a decoded copy, taken when asked
        torch.cuda.synchronize()
    p = {k: t.clone() for k, t in sp.param_list}
    m = {k: t.clone() for k, t in sp.exp_avg.items() if t is not None}
    v = {k: t.clone() for k, t in sp.exp_avg_sq.items() if t is not None}
    protect = torch.zeros(sp.n, dtype=torch.bool, device="cuda")
    protect[torch.argmin(w)] = True
    torch.cuda.synchronize()
    keep = 3000
    d = sp.evict(keep, protect=protect)
    torch.cuda.synchronize()
    assert np.array_equal(d.cpu().numpy(), O.evict_select(w.cpu().numpy(), protect.cpu().numpy(),
                                                          keep))
    rows = torch.nonzero(d)[:, 0]
    assert sp.n == keep and sp.weight_sum is None
    for k, t in sp.param_list:
        if bits is not None and k == "sh":
            c, b = O.sh_quantize(p["sh"][rows].cpu().numpy(), bits)
            got = sp.sh_codes.cpu().numpy()
            assert np.array_equal((got.view(np.uint16) if bits == 16 else got)[:, :keep],
                                  c[:, :keep])
            continue
        assert torch.equal(t, p[k][rows]), k
        assert torch.equal(sp.exp_avg[k], m[k][rows]) and torch.equal(sp.exp_avg_sq[k],
                                                                      v[k][rows]), k
    sp.ensure_capacity()
    sp.rasterize_fwd()
    torch.cuda.synchronize()
    assert torch.isfinite(sp.image).all() and not torch.equal(sp.image, before)
    sp.train_step(torch.full_like(sp.image, 1e-3))
    torch.cuda.synchronize()
    assert sp.status() == api.GS_OK
    # a budget above the count keeps all; one Gaussian is a set
    s = torch.arange(sp.n, dtype=torch.float32, device="cuda")
    torch.cuda.synchronize()
    assert sp.evict(10 ** 9, score=s).sum() == keep and sp.n == keep
    sp.evict(1, score=s)
    torch.cuda.synchronize()
    assert sp.n == 1
