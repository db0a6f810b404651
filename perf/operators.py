"""Cases and plain forms of the eviction operators: per-Gaussian accumulated
blending weights, and the eviction of the Gaussians that carry the least.

A rendered pixel is a normalised weighting of its tile's list: entry k has the
weight w_k = alpha_k T_k, T_k the product of (1 - alpha_j) over the entries
before it, and the background takes what is left. ``weights`` cases sum those
weights over pixels and views for every Gaussian (and take the largest one);
``select`` cases decide which Gaussians survive a budget by such a score;
``evict`` cases decide and compact the parameters and Adam moments.

With ``own`` the operators are the framework's (gs_blend_weights,
gs_evict_select, gs_evict_compact); without it they are elementary torch
operations. Sizes follow the framework's workloads (1,000 Gaussians at 128 x
128, 100,000 at 800 x 800, 1,000,000 at 1920 x 1080, several views, 3840 x
2160), with odd ones beside them.
"""

import math

import torch

own = False

TILE = 16


# --------------------------------------------------------------------- cases

def listed():
    return [
        # one small frame (the framework's smallest workload): latency
        dict(name="weights_1k_128", op="weights", n=1000, views=1, width=128, height=128,
             sigma_lo=1.0, sigma_hi=8.0, masks=True, weighted=False, decay=0.0, largest=False),
        # an interactive frame with the forward's block masks, sums and maxima
        dict(name="weights_100k_800", op="weights", n=100_000, views=1, width=800, height=800,
             sigma_lo=0.6, sigma_hi=16.0, masks=True, weighted=False, decay=0.0, largest=True),
        # three ragged views under a pixel weight (an error map times a mask),
        # added to a running score that forgets; no block masks kept
        dict(name="weights_77k_3x_ragged", op="weights", n=77_003, views=3, width=791, height=597,
             sigma_lo=0.6, sigma_hi=20.0, masks=False, weighted=True, decay=0.9, largest=True),
        # the framework's benchmark frame
        dict(name="weights_1m_1080p", op="weights", n=1_000_000, views=1, width=1920,
             height=1080, sigma_lo=0.6, sigma_hi=16.0, masks=True, weighted=False, decay=0.0,
             largest=False),
        # a 4K frame, scores kept over steps
        dict(name="weights_2m_4k", op="weights", n=2_000_000, views=1, width=3840, height=2160,
             sigma_lo=0.8, sigma_hi=20.0, masks=True, weighted=False, decay=0.5, largest=False),
        # decisions alone, as quantised-SH states need them: a mid-sized set,
        # a third of it never seen (equal scores, the lowest indices survive)
        dict(name="select_60k", op="select", n=60_001, keep=0.5, zeros=0.6, protect=0.1),
        # decisions over the framework's largest set
        dict(name="select_10m", op="select", n=10_000_000, keep=0.8, zeros=0.1, protect=0.0),
        # a scene just started: latency
        dict(name="evict_1k_sh0", op="evict", n=1000, degree=0, moments=True, keep=0.9,
             zeros=0.05, protect=0.0),
        # every tenth Gaussian goes, newborn ones protected
        dict(name="evict_100k_sh3", op="evict", n=100_000, degree=3, moments=True, keep=0.9,
             zeros=0.2, protect=0.05),
        # a finished scene cut to a delivery budget: parameters only, rows of
        # 27 floats
        dict(name="evict_777k_sh2_params", op="evict", n=777_777, degree=2, moments=False,
             keep=0.4, zeros=0.3, protect=0.0),
        # a training set held to its budget
        dict(name="evict_4m_sh3", op="evict", n=4_000_000, degree=3, moments=True, keep=0.85,
             zeros=0.1, protect=0.02),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["weights", "weights", "select", "evict", "evict"])
    if op == "weights":
        width, height = _log_int(rng, 40, 1900), _log_int(rng, 40, 1080)
        views = rng.choice([1, 1, 2, 3])
        pixels = width * height * views
        # half to twenty pixels per Gaussian and view, as the workloads have
        n = max(1, min(1_000_000, int(pixels / views / math.exp(rng.uniform(math.log(2.0),
                                                                           math.log(20.0))))))
        return dict(op=op, n=n, views=views, width=width, height=height,
                    sigma_lo=round(rng.uniform(0.5, 1.0), 3),
                    sigma_hi=round(rng.uniform(6.0, 20.0), 3), masks=rng.random() < 0.6,
                    weighted=rng.random() < 0.4, decay=rng.choice([0.0, 0.0, 0.5, 0.9, 1.0]),
                    largest=rng.random() < 0.5)
    if op == "select":
        return dict(op=op, n=_log_int(rng, 500, 9_000_000), keep=round(rng.uniform(0.05, 0.98), 3),
                    zeros=round(rng.uniform(0.0, 0.9), 3),
                    protect=rng.choice([0.0, 0.0, 0.03, 0.2]))
    return dict(op=op, n=_log_int(rng, 500, 3_500_000), degree=rng.choice([0, 1, 2, 3, 3]),
                moments=rng.random() < 0.75, keep=round(rng.uniform(0.2, 0.95), 3),
                zeros=round(rng.uniform(0.0, 0.5), 3), protect=rng.choice([0.0, 0.0, 0.05]))


# -------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _frame(case, seed):
    """Projected records, per-tile lists and forward outputs of a synthetic
    frame: what gs_project, gs_bin_sort and gs_rasterize_fwd leave behind."""
    g = _generator(seed)
    n, V, W, H = case["n"], case["views"], case["width"], case["height"]
    rand = lambda *s: torch.rand(*s, generator=g, device="cuda", dtype=torch.float64)  # noqa: E731
    # two thirds of the Gaussians spread over the frame and its border, the
    # rest gathered around its middle
    u = (rand(V, n) * 1.1 - 0.05) * W
    v = (rand(V, n) * 1.1 - 0.05) * H
    mid = rand(V, n) < 1.0 / 3.0
    nu = torch.randn(V, n, generator=g, device="cuda", dtype=torch.float64)
    nv = torch.randn(V, n, generator=g, device="cuda", dtype=torch.float64)
    u = torch.where(mid, W * (0.5 + 0.12 * nu), u)
    v = torch.where(mid, H * (0.5 + 0.12 * nv), v)
    lo, hi = math.log(case["sigma_lo"]), math.log(case["sigma_hi"])
    s1 = torch.exp(lo + (hi - lo) * rand(V, n))
    s2 = torch.clamp(s1 * torch.exp(-1.5 * rand(V, n)), min=0.55)
    s1 = torch.maximum(s1, s2)
    ang = math.pi * rand(V, n)
    logit = torch.randn(n, generator=g, device="cuda", dtype=torch.float64)
    o = torch.sigmoid(logit).expand(V, n)
    depth = 1.0 + 9.0 * rand(V, n).float()
    c, s = torch.cos(ang), torch.sin(ang)
    k1, k2 = (math.sqrt(0.5 * math.log2(math.e)) / x for x in (s1, s2))
    uh, vh = u.float(), v.float()
    w1x, w1y = (k1 * c).float(), (k1 * s).float()
    w2x, w2y = (-k2 * s).float(), (k2 * c).float()
    du, dv = u - uh.double(), v - vh.double()
    c1 = -(w1x.double() * du + w1y.double() * dv).float()
    c2 = -(w2x.double() * du + w2y.double() * dv).float()
    nlo = (-torch.log2(255.0 * o)).float()
    cxx = (s1 * c) ** 2 + (s2 * s) ** 2
    cyy = (s1 * s) ** 2 + (s2 * c) ** 2
    q = 2.0 * math.log(2.0) * -nlo.double()
    qp = q + 0.002 * q.abs() + 1e-4
    hx = torch.where(qp > 0, torch.sqrt(qp.clamp(min=0) * cxx) + 0.01, -1.0).float()
    hy = torch.where(qp > 0, torch.sqrt(qp.clamp(min=0) * cyy) + 0.01, -1.0).float()
    rgb = torch.rand(3, V, n, generator=g, device="cuda")
    records = torch.stack([uh, vh, w1x, w1y, c1, w2x, w2y, c2, nlo, rgb[0], rgb[1], rgb[2], hx,
                           hy, o.float(), torch.zeros_like(uh)], dim=-1).contiguous()
    # tile lists: every tile of the 3-sigma square, by tile, depth, index
    r = torch.ceil(3.0 * s1)
    tx_n, ty_n = -(-W // TILE), -(-H // TILE)
    tx0 = torch.floor((u - r) / TILE).clamp(min=0).long()
    tx1 = torch.floor((u + r) / TILE).clamp(max=tx_n - 1).long()
    ty0 = torch.floor((v - r) / TILE).clamp(min=0).long()
    ty1 = torch.floor((v + r) / TILE).clamp(max=ty_n - 1).long()
    nx, ny = (tx1 - tx0 + 1).clamp(min=0), (ty1 - ty0 + 1).clamp(min=0)
    count = (nx * ny).reshape(-1)
    order = torch.argsort(depth.reshape(-1), stable=True)
    rep = torch.repeat_interleave(order, count[order])
    first = torch.cumsum(count[order], 0) - count[order]
    k = torch.arange(rep.numel(), device="cuda") - torch.repeat_interleave(first, count[order])
    wx = nx.reshape(-1)[rep]
    tile = ((rep // max(n, 1)) * ty_n + ty0.reshape(-1)[rep] + k // wx) * tx_n
    tile = tile + tx0.reshape(-1)[rep] + k % wx
    tile, by = torch.sort(tile, stable=True)
    ids = (rep[by] % max(n, 1)).int()
    tiles = tx_n * ty_n * V
    edge = torch.searchsorted(tile, torch.arange(tiles + 1, device="cuda"))
    ranges = torch.stack([edge[:-1], edge[1:]], dim=1).contiguous()
    st = dict(records=records, ids=ids, ranges=ranges, tiles_x=tx_n, tiles_y=ty_n, tile=tile)
    st["n_contrib"], st["masks"] = _forward(case, st)
    if not case["masks"]:
        st["masks"] = None
    del st["tile"]
    return st, g


def _pixels(case, st, tiles):
    """View and pixel-centre coordinates of the given tiles, [t], [t][256]."""
    per = st["tiles_x"] * st["tiles_y"]
    view, tt = tiles // per, tiles % per
    p = torch.arange(TILE * TILE, device="cuda")
    x = (tt % st["tiles_x"] * TILE)[:, None] + p % TILE
    y = (tt // st["tiles_x"] * TILE)[:, None] + p // TILE
    return view, x, y


def _zq(rec, x, y):
    """-log2(255 alpha) of records [t][k][16] at pixels [t][256]: [t][k][256].
    The border alpha = 1/255 is decided here, so products are taken in 64 bits
    and rounded where the record's definition rounds them."""
    px, py = (x.float() + 0.5)[:, None, :], (y.float() + 0.5)[:, None, :]
    f = lambda i: rec[:, :, i:i + 1]  # noqa: E731
    dx, dy = (px - f(0)).double(), (py - f(1)).double()
    p1 = (f(3).double() * dy + (f(2).double() * dx + f(4).double()).float().double()).float()
    p2 = (f(6).double() * dy + (f(5).double() * dx + f(7).double()).float().double()).float()
    p1, p2 = p1.double(), p2.double()
    return (p1 * p1 + (p2 * p2 + f(8).double()).float().double()).float()


def _forward(case, st):
    """n_contrib of every pixel (the list prefix its compositing used) and the
    8 x 8 pixel blocks every list entry reaches, from a front-to-back walk."""
    W, H, V = case["width"], case["height"], case["views"]
    ranges, ids, records = st["ranges"], st["ids"], st["records"]
    n_contrib = torch.zeros(V, H, W, dtype=torch.int32, device="cuda")
    masks = torch.zeros(max(ids.numel(), 1), dtype=torch.uint8, device="cuda")
    lens = ranges[:, 1] - ranges[:, 0]
    tiles = torch.nonzero(lens > 0)[:, 0]
    p = torch.arange(TILE * TILE, device="cuda")
    block = (p % TILE) // 8 + 2 * ((p // TILE) // 8)
    bit = torch.nn.functional.one_hot(block, 4).to(torch.float32)
    for part in torch.split(tiles, 4096):
        T = torch.ones(part.numel(), TILE * TILE, device="cuda")
        view, x, y = _pixels(case, st, part)
        live = (x < W) & (y < H)
        last = torch.zeros(T.shape, dtype=torch.int32, device="cuda")
        at, step = 0, 32
        idx = torch.arange(part.numel(), device="cuda")
        while idx.numel():
            t = part[idx]
            pos = at + torch.arange(step, device="cuda")
            ok = pos[None, :] < lens[t][:, None]
            where = (ranges[t, 0][:, None] + pos[None, :]).clamp(max=ids.numel() - 1)
            rec = records[view[idx][:, None], ids[where].long()]
            zq = _zq(rec, x[idx], y[idx])
            a = torch.exp2(-zq).div_(255.0).clamp_(max=0.99)
            hit = (zq <= 0) & ok[:, :, None]
            a = torch.where(hit, a, 0.0)
            reach = (hit.float() @ bit > 0).to(torch.uint8)
            masks[where[ok]] = (reach * torch.tensor([1, 2, 4, 8], dtype=torch.uint8,
                                                     device="cuda")).sum(-1).to(torch.uint8)[ok]
            Tn = T[idx][:, None, :] * torch.cumprod(1.0 - a, dim=1)
            go = (Tn >= 1e-4) & live[idx][:, None, :]
            used = hit & go
            here = torch.where(used, (pos + 1)[None, :, None].int(), 0).amax(dim=1)
            last[idx] = torch.maximum(last[idx], here)
            live[idx] &= go[:, -1, :]
            T[idx] = Tn[:, -1, :]
            at += step
            idx = idx[(lens[t] > at) & live[idx].any(dim=1)]
        inside = (x < W) & (y < H)
        vv = view[:, None].expand_as(x)
        n_contrib[vv[inside], y[inside], x[inside]] = last[inside]
    return n_contrib, masks


def prepare(case, seed):
    if case["op"] == "weights":
        st, g = _frame(case, seed)
        n, V, W, H = case["n"], case["views"], case["width"], case["height"]
        st["pixel_weight"] = None
        if case["weighted"]:
            # an error map in [0, 1], a fifth of the frame masked out
            e = torch.rand(V, H, W, generator=g, device="cuda") ** 2
            m = torch.rand(V, H // 8 + 1, W // 8 + 1, generator=g, device="cuda") > 0.2
            m = m.repeat_interleave(8, 1).repeat_interleave(8, 2)[:, :H, :W]
            st["pixel_weight"] = (e * m).contiguous()
        # the score kept from earlier steps
        st["sum0"] = torch.rand(n, generator=g, device="cuda") * 4.0
        st["max0"] = torch.rand(n, generator=g, device="cuda") * 0.1
        # the tiles by the length of the prefix that their pixels used
        pad = torch.zeros(V, st["tiles_y"] * TILE, st["tiles_x"] * TILE, dtype=torch.int32,
                          device="cuda")
        pad[:, :H, :W] = st["n_contrib"]
        per = pad.view(V, st["tiles_y"], TILE, st["tiles_x"], TILE).amax(dim=(2, 4)).reshape(-1)
        used, by = torch.sort(per, stable=True)
        used_host, chunks, a = used.tolist(), [], 0
        while a < len(used_host):
            if used_host[a] == 0:
                a += 1
                continue
            b = a + 1
            while b < len(used_host) and (b + 1 - a) * used_host[b] <= 150_000:
                b += 1
            chunks.append((by[a:b].contiguous(), used_host[b - 1]))
            a = b
        st["chunks"] = chunks
        st["out"] = [torch.empty(n, device="cuda"), torch.empty(n, device="cuda")]
        st["case"] = dict(case)
        return st
    g = _generator(seed)
    n = case["n"]
    score = torch.exp(2.0 * torch.randn(n, generator=g, device="cuda"))
    unseen = torch.rand(n, generator=g, device="cuda") < case["zeros"]
    score[unseen] = 0.0
    protect = None
    if case["protect"] > 0:
        protect = (torch.rand(n, generator=g, device="cuda") < case["protect"]).to(torch.uint8)
    n_keep = max(1, int(n * case["keep"]))
    st = dict(case=dict(case), score=score, protect=protect, n_keep=n_keep,
              decisions=torch.empty(n, dtype=torch.int8, device="cuda"))
    if case["op"] == "evict":
        K = (case["degree"] + 1) ** 2
        shapes = [(4,), (4,), (4,), (), (K, 3)]
        sets = 3 if case["moments"] else 1
        st["inputs"] = [[torch.randn((n,) + s, generator=g, device="cuda") for s in shapes]
                        for _ in range(sets)]
        st["outputs"] = [[torch.empty((n_keep,) + s, device="cuda") for s in shapes]
                         for _ in range(sets)]
        st["source"] = torch.empty(n_keep, dtype=torch.int32, device="cuda")
    return st


# ---------------------------------------------------------------- plain form

def _plain_weights(st):
    case = st["case"]
    n, W, H = case["n"], case["width"], case["height"]
    total = torch.zeros(n, device="cuda")
    largest = torch.zeros(n, device="cuda")
    for tiles, L in st["chunks"]:  # bounds the memory of [tiles][entries][256 pixels]
        view, x, y = _pixels(case, st, tiles)
        inside = (x < W) & (y < H)
        at = (view[:, None] * H + y.clamp(max=H - 1)) * W + x.clamp(max=W - 1)
        used = torch.where(inside, st["n_contrib"].view(-1)[at], 0)
        pos = torch.arange(L, device="cuda")
        where = st["ranges"][tiles, 0][:, None] + pos
        ids = st["ids"][where.clamp(max=st["ids"].numel() - 1)].long()
        zq = _zq(st["records"][view[:, None], ids], x, y)
        take = (zq <= 0) & (pos[None, :, None] < used[:, None, :])
        a = torch.where(take, torch.clamp(torch.exp2(-zq) / 255.0, max=0.99), 0.0)
        T = torch.cumprod(1.0 - a, dim=1)
        w = a.clone()
        w[:, 1:] *= T[:, :-1]
        if st["pixel_weight"] is not None:
            m = st["pixel_weight"].view(-1)[at]
            w *= torch.where(m > 0, m.clamp(max=1.0), 0.0)[:, None, :]
        total.index_add_(0, ids.reshape(-1), w.sum(dim=2).reshape(-1))
        if case["largest"]:
            largest.scatter_reduce_(0, ids.reshape(-1), w.amax(dim=2).reshape(-1), "amax")
    d = case["decay"]
    if d > 0:
        total += d * st["sum0"]
        largest = torch.maximum(largest, d * st["max0"])
    return [total, largest] if case["largest"] else [total]


def _plain_select(st):
    """Which Gaussians survive: the protected ones first, then the highest
    scores, equal ones by the lowest index; NaN goes first."""
    s = torch.where(torch.isnan(st["score"]), -math.inf, st["score"])
    if st["protect"] is not None:
        s = torch.where(st["protect"] != 0, math.inf, s)
    best = torch.sort(s, descending=True, stable=True).indices[:st["n_keep"]]
    decisions = torch.zeros(s.numel(), dtype=torch.int8, device="cuda")
    decisions[best] = 1
    return decisions, best


def _plain_evict(st):
    decisions, best = _plain_select(st)
    source = torch.sort(best).values
    return [decisions, source.int()] + [torch.index_select(x, 0, source)
                                        for arrays in st["inputs"] for x in arrays]


# ---------------------------------------------------------- the framework's

def _handles(st):
    """What a program makes once and keeps beside its buffers: descriptors and
    a workspace."""
    from gaussian_splatting_differentiable_ewa_b200 import api
    c = st["case"]
    if c["op"] == "weights":
        class Cam:
            def as_dict(self):
                return dict(viewmat=[1, 0, 0, 0, 0, 1, 0, 0, 0, 0, 1, 0], fx=c["width"],
                            fy=c["width"], cx=c["width"] / 2, cy=c["height"] / 2,
                            width=c["width"], height=c["height"], campos=[0, 0, 0])
        size = api.gs_blend_weights_workspace_size(c["n"])
        return dict(api=api, cams=api.cameras([Cam()] * c["views"]),
                    proj=api.projected(st["records"], None, None),
                    bins=api.binned(st["ids"], st["ranges"], None, st["ids"].numel()),
                    ws=torch.zeros(-(-size // 8), dtype=torch.int64, device="cuda"))
    size = api.gs_evict_workspace_size(c["n"])
    h = dict(api=api, ws=torch.zeros(-(-size // 8), dtype=torch.int64, device="cuda"))
    if c["op"] == "evict":
        p = st["inputs"][0]
        h["params"] = api.params(*p, c["degree"])
        h["moments"] = [api.grads(*x) for x in st["inputs"][1:]] or [None, None]
        h["out"] = [api.grads(*x) for x in st["outputs"]] + [None, None]
    return h


def _own(st):
    if "handles" not in st:
        st["handles"] = _handles(st)
    h, c = st["handles"], st["case"]
    api, stream = h["api"], torch.cuda.current_stream()
    if c["op"] == "weights":
        total, largest = st["out"]
        if c["decay"] > 0:
            total.copy_(st["sum0"])
            if c["largest"]:
                largest.copy_(st["max0"])
        api.gs_blend_weights(h["proj"], h["bins"], h["cams"], c["views"], c["n"], st["n_contrib"],
                             total, h["ws"], weight_max=largest if c["largest"] else None,
                             warp_masks=st["masks"], pixel_weight=st["pixel_weight"],
                             decay=c["decay"], stream=stream)
        return [total, largest] if c["largest"] else [total]
    api.gs_evict_select(st["score"], st["protect"], c["n"], st["n_keep"], st["decisions"],
                        h["ws"], stream=stream)
    if c["op"] == "select":
        return [st["decisions"]]
    api.gs_evict_compact(h["params"], h["moments"][0], h["moments"][1], st["decisions"],
                         h["out"][0], h["out"][1], h["out"][2], st["n_keep"], h["ws"],
                         source=st["source"], stream=stream)
    return [st["decisions"], st["source"]] + [x for arrays in st["outputs"] for x in arrays]


def run(state):
    if own:
        return _own(state)
    if state["case"]["op"] == "weights":
        return _plain_weights(state)
    if state["case"]["op"] == "select":
        return [_plain_select(state)[0]]
    return _plain_evict(state)


# -------------------------------------------------------------------- bounds

def work(case):
    """Bytes: every input read once, every output written once. Operations of
    ``weights``: 20 per (pixel, entry) that blends -- the quadratic form and
    the exponential (13), the transmittance and the weight (3), its sum and
    the tests (4) -- with the blended entries from the frame's mean coverage."""
    n = case["n"]
    if case["op"] == "weights":
        P = case["views"] * case["width"] * case["height"]
        lo, hi = math.log(case["sigma_lo"]), math.log(case["sigma_hi"])
        # mean s1^2 e^-1.5u, s1 log-uniform and u uniform; the alpha >= 1/255
        # ellipse of opacity one half has q <= 2 ln(127.5)
        s2 = (math.exp(2 * hi) - math.exp(2 * lo)) / (2 * (hi - lo)) * (1 - math.exp(-1.5)) / 1.5
        q = 2 * math.log(127.5)
        cover = case["views"] * n / (1.21 * P) * math.pi * q * s2
        # a covered pixel loses ln(1/(1 - alpha)) ~ 0.5 / ln(127.5) on average;
        # compositing ends at 1e-4
        hits = min(cover, math.log(1e4) * math.log(127.5) / 0.55)
        ids = P / 256 * hits * 2
        out = (1 + case["largest"]) * (2 if case["decay"] > 0 else 1)
        touched = min(n * case["views"], ids)
        nbytes = 64 * touched + ids * (4 + case["masks"]) + 16 * P / 256 + 4 * P + 4 * n * out
        if case["weighted"]:
            nbytes += 4 * P
        return {"bytes": int(nbytes), "flops": int(20 * hits * P)}
    nbytes = n * (4 + 1 + (1 if case["protect"] > 0 else 0))
    if case["op"] == "evict":
        row = 4 * (13 + 3 * (case["degree"] + 1) ** 2) * (3 if case["moments"] else 1)
        nbytes += max(1, int(n * case["keep"])) * (2 * row + 4)
    return {"bytes": int(nbytes), "flops": 0}


# --------------------------------------------------------------------- exact

def exact(case, seed):
    """The weights in 64 bits: every pixel's list walked entry by entry, all
    tiles side by side. An eviction's copies: the rows that outlive n - n_keep
    removals, the removed ones found by a sort of (class, score, -index) from
    the other end. Whole numbers have no such value: None."""
    st = prepare(case, seed)
    if case["op"] == "select":
        return None
    if case["op"] == "evict":
        s, n = st["score"].double(), case["n"]
        rank = torch.arange(n - 1, -1, -1, device="cuda")  # the highest index goes first
        rank = rank[torch.sort(s[n - 1 - torch.arange(n, device="cuda")], stable=True).indices]
        if st["protect"] is not None:
            p = st["protect"][rank] != 0
            rank = torch.cat([rank[~p], rank[p]])
        stays = torch.ones(n, dtype=torch.bool, device="cuda")
        stays[rank[:n - st["n_keep"]]] = False
        return [None, None] + [x[stays].double() for arrays in st["inputs"] for x in arrays]
    n, V, W, H = case["n"], case["views"], case["width"], case["height"]
    rec, ids, ranges = st["records"].double(), st["ids"].long(), st["ranges"]
    total = torch.zeros(n, dtype=torch.float64, device="cuda")
    largest = torch.zeros(n, dtype=torch.float64, device="cuda")
    tx, ty = st["tiles_x"], st["tiles_y"]
    tiles = torch.arange(V * tx * ty, device="cuda")
    limit = torch.zeros(V, ty * TILE, tx * TILE, dtype=torch.int64, device="cuda")
    limit[:, :H, :W] = st["n_contrib"]
    weight = torch.zeros(V, ty * TILE, tx * TILE, dtype=torch.float64, device="cuda")
    weight[:, :H, :W] = 1.0 if st["pixel_weight"] is None else st["pixel_weight"].double()

    def by_tile(a):
        return a.view(V, ty, TILE, tx, TILE).permute(0, 1, 3, 2, 4).reshape(V * ty * tx, -1)

    limit, weight = by_tile(limit), by_tile(weight).clamp(0.0, 1.0)
    longest, order = torch.sort(limit.amax(dim=1), descending=True)
    lane = torch.arange(TILE * TILE, device="cuda")
    px = ((tiles % tx) * TILE)[:, None] + lane % TILE + 0.5
    py = ((tiles // tx % ty) * TILE)[:, None] + lane // TILE + 0.5
    T = torch.ones_like(weight)[order]
    limit, weight, px, py = limit[order], weight[order], px[order], py[order]
    start, view = ranges[order, 0], order // (tx * ty)
    steps = longest.tolist()
    alive = len(steps)
    for k in range(steps[0] if steps else 0):
        while alive and steps[alive - 1] <= k:
            alive -= 1
        i = ids[start[:alive] + k]
        r = rec[view[:alive], i][:, :, None]
        dx, dy = px[:alive] - r[:, 0], py[:alive] - r[:, 1]
        e = (r[:, 2] * dx + r[:, 3] * dy + r[:, 4]) ** 2
        e = e + (r[:, 5] * dx + r[:, 6] * dy + r[:, 7]) ** 2 + r[:, 8]
        a = torch.where((e <= 0) & (k < limit[:alive]), (torch.exp2(-e) / 255.0).clamp(max=0.99),
                        0.0)
        w = a * T[:alive]
        T[:alive] -= w
        w = w * weight[:alive]
        total.index_add_(0, i, w.sum(dim=1))
        largest.scatter_reduce_(0, i, w.amax(dim=1), "amax")
    if case["decay"] > 0:
        d = case["decay"]
        total = total + d * st["sum0"].double()
        largest = torch.maximum(largest, d * st["max0"].double())
    return [total, largest] if case["largest"] else [total]
