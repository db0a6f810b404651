// weights.cu -- accumulated blending weights (gs_blend_weights), sm_100a.
//
// A rendered pixel weighs its tile's list: entry k has alpha_k T_k (lshu.cn
// sec. 3.2 `blend`). This file sums those weights per Gaussian over pixels and
// views, after the forward rasteriser, which left every pixel's list prefix.
//
//  k_weights_begin  totals cleared, kept maxima decayed.
//  k_blend_weights  the walk.
//  k_weights_end    sums <- decayed sums + totals.

#include <cuda_runtime.h>

#include <cmath>

#include "gs_internal.h"

namespace gsb {
namespace {

constexpr float kInv255 = 1.0f / 255.0f;
constexpr int kWarps = 4;  // 8 x 8 pixel blocks of a tile, one warp each

struct WeightGeom {
  Grid g;
  int n;
  int64_t capacity;  // length of ids
  float whole;       // 2^k: whole units of a total in a weight of one
};

__device__ __forceinline__ float2 f2(float x) { return make_float2(x, x); }

// Whether the alpha >= 1/255 ellipse of a record reaches the 8 x 8 block of
// pixels at (xb, yb): the forward rasteriser's test (raster.cu), for a caller
// that kept no masks. The record's box first; then the least value of
// q' = (w1 . d)^2 + (w2 . d)^2 over the rectangle of pixel centres -- 0 with
// the mean inside, else on one of the edges, where q' is a parabola in the
// free coordinate -- against -nlo padded (0.2 % + 0.01) well beyond the float
// rounding of the walk's zq, so no pixel that the walk would take is dropped.
__device__ __noinline__ bool block_reached(const float* r, int xb, int yb) {
  const float4* r4 = reinterpret_cast<const float4*>(r);
  const float4 ra = __ldg(r4), rb = __ldg(r4 + 1), rd = __ldg(r4 + 3);
  const float u = ra.x, v = ra.y, hx = rd.x, hy = rd.y;
  const float xlo = (float)xb + 0.5f, ylo = (float)yb + 0.5f;
  if (!(hx >= 0.f) || !(u + hx >= xlo && u - hx <= xlo + 7.f && v + hy >= ylo &&
                        v - hy <= ylo + 7.f))
    return false;
  const float w1x = ra.z, w1y = ra.w, w2x = rb.y, w2y = rb.z;
  const float a = fmaf(w1x, w1x, w2x * w2x), b = fmaf(w1x, w1y, w2x * w2y);
  const float c = fmaf(w1y, w1y, w2y * w2y), ia = 1.f / a, ic = 1.f / c;
  const float ex0 = xlo - u, ex1 = ex0 + 7.f, ey0 = ylo - v, ey1 = ey0 + 7.f;
  if (ex0 <= 0.f && ex1 >= 0.f && ey0 <= 0.f && ey1 >= 0.f) return true;
  float best = __int_as_float(0x7f800000);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float ex = e ? ex1 : ex0;  // vertical edges
    const float dy = fminf(fmaxf(-b * ex * ic, ey0), ey1);
    best = fminf(best, fmaf(a * ex, ex, fmaf(2.f * b * ex, dy, c * dy * dy)));
    const float ey = e ? ey1 : ey0;  // horizontal edges
    const float dx = fminf(fmaxf(-b * ey * ia, ex0), ex1);
    best = fminf(best, fmaf(c * ey, ey, fmaf(2.f * b * ey, dx, a * dx * dx)));
  }
  return best <= fmaf(-__ldg(r + R_NLO), 1.002f, 0.01f);
}

// Warp sums (or, with MAX, maxima) of kWeightGroup = 4 per-lane values by a
// transposing butterfly: the first two exchanges halve the live values, three
// more finish the one that is left: 6 shuffles instead of 20. Lane l returns
// the result of value 2 ((l>>4)&1) + ((l>>3)&1).
constexpr int kWeightGroup = 4;
template <bool MAX>
__device__ __forceinline__ float warp_reduce4(const float (&v)[kWeightGroup]) {
  const int lane = threadIdx.x & 31;
  const bool h16 = lane & 16, h8 = lane & 8;
  auto op = [](float x, float y) { return MAX ? fmaxf(x, y) : x + y; };
  float a[2];
#pragma unroll
  for (int k = 0; k < 2; ++k)
    a[k] = op(h16 ? v[k + 2] : v[k],
              __shfl_xor_sync(0xffffffffu, h16 ? v[k] : v[k + 2], 16));
  float c = op(h8 ? a[1] : a[0], __shfl_xor_sync(0xffffffffu, h8 ? a[0] : a[1], 8));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) c = op(c, __shfl_xor_sync(0xffffffffu, c, o));
  return c;
}

// 1 where p and x <= 0, else 0.
__device__ __forceinline__ float one_if(bool p, float x) {
  float r;
  asm("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t"
      "set.le.and.f32.f32 %0, %1, 0f00000000, q;\n\t}"
      : "=f"(r)
      : "f"(x), "r"((uint32_t)p));
  return r;
}

// Accumulated blending weights (gs_blend_weights): per list entry the sum (and
// with MAX the largest) over a tile's pixels of m w, w = alpha T the forward's
// weight and m the pixel's weight in [0, 1]. The walk takes zq and alpha by the
// forward's IEEE operations, without colours and without its stop test:
// n_contrib already says how far each pixel composited. T falls by one fma,
// T - alpha T, where the forward rounds 1 - alpha and then T (1 - alpha), so
// that weights are the forward's but for a rounding of T per entry. They are
// linear in T, so T starts at m and the pixel weight costs nothing per entry.
//
// Every warp works by itself on its 8 x 8 pixel block, two pixels per lane:
// it scans the list for the entries that reach its block (the forward's masks,
// or the block test), queues their positions, and takes them 32 at a time.
// The first 48 bytes of the 32 records go to shared memory by 16-byte
// asynchronous copies, three lanes to a record; the warp evaluates all of
// them, four per transposing butterfly, which leaves each entry's result in
// the lane that owns the entry; that lane adds it to the Gaussian's total --
// integers, so totals do not depend on the order in which warps arrive. (A
// maximum of non-negative floats is a maximum of their bits.)
//
// A total has 96 bits: a word of 64 in units of 2^-k and, apart, a word of 32
// in units of 2^-(k + 32) whose carries go to the first. A pixel's weights sum
// to one at most, so the first word holds every total of a frame with
// pixels 2^k < 2^64 (k = 43 at 1080p, 41 at 4K). From 2^20 whole units on a sum
// is rounded to them, 2^-21 of it at most, less than the roundings of the T
// that a weak sum was made with, and costs one atomic; the least sum that a
// frame without pixel weights has, 1e-4 / 255 (2^-21.3), lies above that at
// 1080p and just below at 4K. Smaller sums (of small pixel weights, or of calls
// of more pixels) are held exactly, down to 2^-(k + 9): they are the scores
// that an eviction orders.
// Sending all sums below 2^23 units that way took 0.7 % more at 4K; clearing and
// reading the second word takes 0.3 % there.
//
// The next chunk's records, the one after's ids and the next masks are
// in flight meanwhile; no warp waits for another, and only the last chunk of
// a block is padded.
//
// What bounds it: instruction issue, and the shared-memory reads behind it (a
// read returns 4 bytes to each of 32 lanes per cycle whether or not they share
// an address: 9 cycles of the SM for a record's 36 bytes; the forward's (x, x)
// pairs would take 18). On a 1M-Gaussian 1080p frame (4.4M entries of 8 x 8
// blocks) the whole call takes 0.230 ms at 82 % of the issue slots, the
// forward itself 0.494 ms; on 1000 Gaussians at 128 x 128 three launches take
// 0.015 ms (0.002 more before the walk and the last kernel were allowed to begin
// while the kernel before them ends). What was measured on the way, for the
// 1080p frame: a block staging batches of its tile's list as the forward
// does, 0.290 ms (barriers, and lists padded per batch); bulk copies of the
// records, 0.277 ms (a bulk copy is issued lane by lane); plain loads through
// registers, 0.243 ms; four pixels per lane, 0.251 ms; one warp per thread
// block, 0.233 ms.
constexpr float kWeightRest = 4294967296.f;  // 2^32: units of a rest in a whole one
constexpr float kWeightWhole = 1048576.f;    // 2^20: whole units from which on rests are rounded
constexpr int kWeightQueue = 256;            // positions a warp can hold
constexpr int kWeightAhead = 96;             // positions it wants queued: three chunks
constexpr int kWeightRow = 12;               // floats of a record the walk stages
static_assert(R_NLO < kWeightRow, "the staged part holds the evaluation form");

template <bool MASKS, bool MAX>
__global__ void __launch_bounds__(32 * kWarps) k_blend_weights(
    const float* __restrict__ records, const uint32_t* __restrict__ ids,
    const int64_t* __restrict__ ranges, WeightGeom geo, const uint32_t* __restrict__ n_contrib,
    const uint8_t* __restrict__ wmask_in, const float* __restrict__ pixel_weight,
    unsigned long long* __restrict__ sums, uint32_t* __restrict__ rests,
    uint32_t* __restrict__ largest, uint32_t* __restrict__ status) {
  __shared__ __align__(16) float s_rec[kWarps][2][32][kWeightRow];
  __shared__ __align__(16) uint32_t s_at[kWarps][32];
  __shared__ uint32_t s_queue[kWarps][kWeightQueue];

  const int tile = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the warp's pixel block, and the lane's pixels (px, py) and (px, py + 4)
  const int view = tile / geo.g.tiles_per_view, tt = tile - view * geo.g.tiles_per_view;
  const int ty = tt / geo.g.tiles_x, tx = tt - ty * geo.g.tiles_x;
  const int xb = tx * kTile + 8 * (warp & 1), yb = ty * kTile + 8 * (warp >> 1);
  const int px = xb + (lane & 7), py = yb + (lane >> 3);
  const size_t hw = (size_t)geo.g.width * geo.g.height;
  // a malformed range counts as empty and is reported
  int64_t start = ranges[2 * (int64_t)tile], end = ranges[2 * (int64_t)tile + 1];
  if (start < 0 || end > geo.capacity || end < start) {
    if (threadIdx.x == 0) atomicOr(status, kStatusBounds);
    start = end = 0;
  }
  const float* rec_view = records + (size_t)view * geo.n * GS_RECORD_FLOATS;
  const uint32_t lt = lanemask_lt();

  // a pixel without weight takes no part (a NaN or negative weight counts as
  // none)
  float2 T;
  uint32_t nc[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    nc[i] = 0;
    float m = 1.f;
    if (px < geo.g.width && py + 4 * i < geo.g.height) {
      const size_t pix = (size_t)view * hw + (size_t)(py + 4 * i) * geo.g.width + px;
      nc[i] = n_contrib[pix];
      if (pixel_weight) m = pixel_weight[pix];
      if (!(m > 0.f)) {
        nc[i] = 0;
        m = 0.f;
      }
    }
    (i ? T.y : T.x) = fminf(m, 1.f);
  }
  // the longest prefix among the warp's pixels; positions are 32-bit
  const uint32_t wm = __reduce_max_sync(0xffffffffu, max(nc[0], nc[1]));
  const int64_t used = end - start < (int64_t)wm ? end - start : (int64_t)wm;
  const int limit = (int)(used < (int64_t)0x7fffff00 ? used : (int64_t)0x7fffff00);

  uint32_t* queue = s_queue[warp];
  int head = 0, tail = 0, scan = 0;  // positions consumed, queued, looked at
  uint32_t mk[4];                    // MASKS: the masks of the next 128 positions
  auto load_masks = [&] {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = scan + 32 * i + lane;
      mk[i] = p < limit ? (uint32_t)wmask_in[start + p] : 0u;
    }
  };
  auto push = [&](bool hit, int p) {
    const uint32_t bal = __ballot_sync(0xffffffffu, hit);
    if (hit) queue[(tail + __popc(bal & lt)) & (kWeightQueue - 1)] = (uint32_t)p;
    tail += __popc(bal);
  };
  // queue positions until three chunks are there or the list has ended
  auto fill = [&] {
    while (tail - head < kWeightAhead && scan < limit) {
      if (MASKS) {
#pragma unroll
        for (int i = 0; i < 4; ++i) push((mk[i] >> warp) & 1u, scan + 32 * i + lane);
        scan += 128;
        load_masks();
      } else {
        const int p = scan + lane;
        bool hit = false;
        if (p < limit) {
          const uint32_t id = __ldg(&ids[start + p]);
          // an entry that names no Gaussian goes through, to be reported
          hit = id >= (uint32_t)geo.n ||
                block_reached(rec_view + (size_t)id * GS_RECORD_FLOATS, xb, yb);
        }
        push(hit, p);
        scan += 32;
      }
    }
    __syncwarp();
  };

  // lane l fetches (and adds up) entry `own` of every chunk: the one whose sum
  // the butterflies leave in it
  const int own = 4 * (lane & 7) + 2 * ((lane >> 4) & 1) + ((lane >> 3) & 1);
  constexpr uint32_t kNone = 0xffffffffu;
  struct Own {
    uint32_t id, at;
  };
  auto fetch_ids = [&](int first) {  // of the chunk that starts at queue position `first`
    Own o{kNone, 0u};
    if (first + own < tail) {
      o.at = queue[(first + own) & (kWeightQueue - 1)];
      o.id = __ldg(&ids[start + o.at]);
      if (o.id >= (uint32_t)geo.n) {  // never read outside the records
        atomicOr(status, kStatusBounds);
        o.id = kNone;
      }
    }
    return o;
  };
  auto issue = [&](const Own& o, int buf) {
    float(*rows)[kWeightRow] = s_rec[warp][buf];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2), q = lane & 3;
      const uint32_t id =
          __shfl_sync(0xffffffffu, o.id, (r >> 2) + 16 * ((r >> 1) & 1) + 8 * (r & 1));
      if (id != kNone && q < 3)
        copy_async16(&rows[r][4 * q], rec_view + (size_t)id * GS_RECORD_FLOATS + 4 * q);
    }
    copy_async_commit();
    if (o.id == kNone) {  // no entry, or none with a Gaussian: zq = +inf at every pixel
#pragma unroll
      for (int i = 0; i < 9; ++i) rows[own][i] = i == R_NLO ? __int_as_float(0x7f800000) : 0.f;
    }
  };

  const float pxc = (float)px + 0.5f;
  const float2 pyc = make_float2((float)py + 0.5f, (float)py + 4.5f);
  if (MASKS) load_masks();
  fill();
  Own next = fetch_ids(0);
  issue(next, 0);
  Own after = fetch_ids(32);
  wait_for_previous();  // the totals are cleared
  for (int buf = 0; head < tail; buf ^= 1) {
    const int n = min(32, tail - head);
    const Own mine = next;
    s_at[warp][own] = mine.at;
    head += n;
    // what comes next on its way
    next = after;
    issue(next, buf ^ 1);
    fill();
    after = fetch_ids(head + 32);
    copy_async_wait_but_one();
    __syncwarp();

    float sum = 0.f, top = 0.f;
    const int groups = (n + kWeightGroup - 1) / kWeightGroup;
    for (int g = 0; g < groups; ++g) {
      const float(*rec)[kWeightRow] = &s_rec[warp][buf][kWeightGroup * g];
      const uint4 at4 = *reinterpret_cast<const uint4*>(&s_at[warp][kWeightGroup * g]);
      const uint32_t at[kWeightGroup] = {at4.x, at4.y, at4.z, at4.w};
      float v[kWeightGroup], t[kWeightGroup];  // of -w: -alpha saves sign changes in T (1 - alpha)
#pragma unroll
      for (int k = 0; k < kWeightGroup; ++k) {
        const float4 ra = *reinterpret_cast<const float4*>(&rec[k][0]);  // u v w1x w1y
        const float4 rb = *reinterpret_cast<const float4*>(&rec[k][4]);  // c1 w2x w2y c2
        const float nlo = rec[k][R_NLO];
        const float dx = __fsub_rn(pxc, ra.x);
        const float a1 = __fmaf_rn(ra.z, dx, rb.x), a2 = __fmaf_rn(rb.y, dx, rb.w);
        const float2 dy = make_float2(__fsub_rn(pyc.x, ra.y), __fsub_rn(pyc.y, ra.y));
        const float2 p1 = __ffma2_rn(f2(ra.w), dy, f2(a1));
        const float2 p2 = __ffma2_rn(f2(rb.z), dy, f2(a2));
        const float2 zq = __ffma2_rn(p1, p1, __ffma2_rn(p2, p2, f2(nlo)));
        const float2 raw = __fmul2_rn(make_float2(exp2f(-zq.x), exp2f(-zq.y)), f2(-kInv255));
        const float2 on = make_float2(one_if(at[k] < nc[0], zq.x), one_if(at[k] < nc[1], zq.y));
        const float2 na = __fmul2_rn(on, make_float2(fmaxf(-kAlphaMax, raw.x),
                                                     fmaxf(-kAlphaMax, raw.y)));
        const float2 nw = __fmul2_rn(na, T);
        T = __ffma2_rn(na, T, T);
        v[k] = nw.x + nw.y;
        if (MAX) t[k] = fmaxf(-nw.x, -nw.y);
      }
      const float s = warp_reduce4<false>(v);
      if ((lane & 7) == g) sum = -s;
      if (MAX) {
        const float m = warp_reduce4<true>(t);
        if ((lane & 7) == g) top = m;
      }
    }
    // an entry without a Gaussian sums to 0
    const float units = sum * geo.whole;
    if (units >= kWeightWhole) atomicAdd(&sums[mine.id], __float2ull_rn(units));
    if (MAX && sum > 0.f) atomicMax(&largest[mine.id], __float_as_uint(top));
    // seldom: tested for the warp (a branch per lane: 1.3 % more at 4K)
    const bool small = units > 0.f && units < kWeightWhole;
    if (__any_sync(0xffffffffu, small) && small) {
      uint32_t add = __float2uint_rz(units);
      const uint32_t rest = __float2uint_rn((units - truncf(units)) * kWeightRest);
      if (rest && atomicAdd(&rests[mine.id], rest) + rest < rest) ++add;  // a carry
      if (add) atomicAdd(&sums[mine.id], (unsigned long long)add);
    }
    __syncwarp();  // the chunk's shared memory is free
  }
}

// Before the walk: totals cleared, the kept maxima scaled (a decay of 0 reads
// nothing). A kept maximum below zero or NaN counts as zero.
__global__ void __launch_bounds__(256) k_weights_begin(unsigned long long* __restrict__ sums,
                                                       uint32_t* __restrict__ rests,
                                                       float* __restrict__ largest, int n,
                                                       float decay) {
  let_next_begin();
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  sums[i] = 0ull;
  rests[i] = 0u;
  if (largest) largest[i] = decay > 0.f ? fmaxf(decay * largest[i], 0.f) : 0.f;
}

// After the walk: sum <- decay sum + total, in double, rounded once.
__global__ void __launch_bounds__(256) k_weights_end(const unsigned long long* __restrict__ sums,
                                                     const uint32_t* __restrict__ rests,
                                                     float* __restrict__ weight_sum, int n,
                                                     double unit, float decay) {
  wait_for_previous();
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const double t = fma((double)rests[i], 1.0 / (double)kWeightRest, (double)sums[i]) * unit;
  weight_sum[i] = (float)(decay > 0.f ? fma((double)decay, (double)weight_sum[i], t) : t);
}

}  // namespace

cudaError_t launch_blend_weights(const float* records, const uint32_t* ids, const int64_t* ranges,
                                 int64_t capacity, const Grid& g, int n_views, int n,
                                 const uint32_t* n_contrib, const uint8_t* warp_masks,
                                 const float* pixel_weight, float decay, float* weight_sum,
                                 float* weight_max, uint64_t* sums, uint32_t* status,
                                 cudaStream_t stream) {
  const int64_t tiles = (int64_t)g.tiles_per_view * n_views;
  const unsigned blocks = (unsigned)(((int64_t)n + 255) / 256);
  unsigned long long* acc = reinterpret_cast<unsigned long long*>(sums);
  uint32_t* rests = reinterpret_cast<uint32_t*>(acc + n);
  // the largest 2^k by which the pixels, 2^31 at most, fit 64 bits; 2^-10 of
  // them are left to the roundings of the weights and their sums
  const uint64_t pixels = (uint64_t)g.width * g.height * n_views;
  int k = 63;
  while (pixels > (0ull - (1ull << 54)) >> k) --k;
  k_weights_begin<<<blocks, 256, 0, stream>>>(acc, rests, weight_max, n, decay);
  WeightGeom geo{g, n, capacity, ldexpf(1.f, k)};
  const auto walk = warp_masks ? (weight_max ? k_blend_weights<true, true>
                                             : k_blend_weights<true, false>)
                               : (weight_max ? k_blend_weights<false, true>
                                             : k_blend_weights<false, false>);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess)
    e = launch_dependent(walk, dim3((unsigned)tiles), dim3(32 * kWarps), stream, records,
                         ids, ranges, geo, n_contrib, warp_masks, pixel_weight, acc, rests,
                         reinterpret_cast<uint32_t*>(weight_max), status);
  if (e == cudaSuccess)
    e = launch_dependent(k_weights_end, dim3(blocks), dim3(256), stream,
                         (const unsigned long long*)acc, (const uint32_t*)rests, weight_sum, n,
                         ldexp(1.0, -k), decay);
  return e;
}

}  // namespace gsb
