// evict.cu -- eviction under a budget: which Gaussians survive, and their
// compaction, sm_100a.
//
// Selection keeps the n_keep Gaussians with the highest scores (accumulated
// blending weights, or any score), protected ones first, equal scores by the
// lowest index. A score becomes a 32-bit key whose unsigned order is the
// score's; the threshold is the n_keep-th largest key, found digit by digit
// from counts alone. Of the keys equal to the threshold the first ones in
// index order survive. One launch either way:
//
//  k_ev_select       small sets: one block, the keys in its registers, four
//                    digits of 8 bits.
//  k_ev_select_grid  larger sets: up to one block per SM, launched together;
//                    three digits (11 + 11 + 10 bits) whose counts meet in
//                    global memory, behind a grid barrier with a time limit.
//                    Up to 1.2M Gaussians the keys stay in registers, above
//                    that they are read again for every digit (from L2 up to
//                    some 25M Gaussians).
//
// Compaction moves the survivors' rows in index order:
//
//  k_ev_count   survivors per 256 Gaussians (and per 1024 of those).
//  k_ev_move    every block adds up the survivors before its 256 Gaussians --
//               from the counts, or for small sets from the decisions
//               themselves -- lists its own and copies their rows of one
//               array set (parameters, first or second moments); consecutive
//               threads write consecutive elements of the output.

#include <cuda_runtime.h>

#include "gs_internal.h"

namespace gsb {
namespace {

// Key of a score: unsigned order = score order, -0 and +0 alike, NaN the
// lowest (0), a protected Gaussian the highest (above +infinity).
__device__ __forceinline__ uint32_t ev_key(float score, bool prot) {
  const uint32_t b = __float_as_uint(score);
  uint32_t key = (b >> 31) ? ~b : (b | 0x80000000u);
  if (b == 0x80000000u) key = 0x80000000u;
  if ((b & 0x7fffffffu) > 0x7f800000u) key = 0u;
  return prot ? 0xffffffffu : key;
}

__device__ __forceinline__ uint32_t ev_key_at(const float* score, const uint8_t* protect,
                                              int64_t i) {
  return ev_key(__ldg(&score[i]), protect && protect[i]);
}

// Exclusive sum over the block's threads of x, and the total.
template <int WARPS>
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* s_w, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) s_w[warp] = incl;
  __syncthreads();
  uint32_t w = lane < WARPS ? s_w[lane] : 0u, wi = w;
#pragma unroll
  for (int o = 1; o < WARPS; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, wi, o);
    if (lane >= o) wi += y;
  }
  total = __shfl_sync(0xffffffffu, wi, WARPS - 1);
  return __shfl_sync(0xffffffffu, wi - w, warp) + incl - x;
}

// From the highest digit down, the one in which the wanted key lies: thread t
// holds the counts of bins BINS - 1 - (t PER + k) (0 past the last bin). One
// thread finds it and writes the digit, the rank left within it and its count.
template <int WARPS, uint32_t BINS, int PER>
__device__ __forceinline__ void find_digit(const uint32_t (&c)[PER], uint32_t want, uint32_t* s_w,
                                           uint32_t* found) {
  uint32_t sum = 0, total;
#pragma unroll
  for (int k = 0; k < PER; ++k) sum += c[k];
  uint32_t above = block_scan<WARPS>(sum, s_w, total);
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    if (above < want && want <= above + c[k]) {
      found[0] = BINS - 1 - (threadIdx.x * PER + k);
      found[1] = want - above;
      found[2] = c[k];
    }
    above += c[k];
  }
}

// ------------------------------------------------------------ selection, small

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelKeys = 8;  // keys per thread, in registers
// Up to here one block: at 8,192 Gaussians 9.4 us against 12.6 for the grid,
// whose barriers cost more than the block's longer passes (1,000: 6 us).
constexpr int kSelMax = kSelThreads * kSelKeys;

// The warps hold consecutive spans of 32 per_thread Gaussians; lane l of a
// warp its elements l, l + 32, ... Digit counts have one counter per lane:
// equal scores by the thousand (Gaussians never seen), or scores of one
// magnitude, would otherwise make a warp's 32 additions wait for one another.
__global__ void __launch_bounds__(kSelThreads) k_ev_select(const float* __restrict__ score,
                                                           const uint8_t* __restrict__ protect,
                                                           int n, int n_keep, int per_thread,
                                                           int8_t* __restrict__ decisions) {
  __shared__ uint4 s_copies[256][8];  // [digit][32 lanes]
  __shared__ __align__(16) uint32_t s_hist[256];
  __shared__ uint32_t s_equal[kSelWarps];
  __shared__ uint32_t s_found[3];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int first = warp * 32 * per_thread + lane;
  int mine = first < n ? (n - first + 31) / 32 : 0;  // elements this lane holds
  if (mine > per_thread) mine = per_thread;
  uint32_t key[kSelKeys];
#pragma unroll
  for (int k = 0; k < kSelKeys; ++k) {
    if (k >= per_thread) break;
    key[k] = k < mine ? ev_key_at(score, protect, first + 32 * k) : 0u;
  }
  (&s_copies[0][0])[threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
  (&s_copies[0][0])[threadIdx.x + kSelThreads] = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();

  uint32_t t = 0, rank = (uint32_t)n_keep, equal = 0;
  uint32_t* copies = reinterpret_cast<uint32_t*>(s_copies) + lane;
  for (int shift = 24; shift >= 0; shift -= 8) {
    const uint32_t known = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
#pragma unroll
    for (int k = 0; k < kSelKeys; ++k) {
      if (k >= per_thread) break;
      if (k < mine && ((key[k] ^ t) & known) == 0u)
        atomicAdd(&copies[((key[k] >> shift) & 255u) * 32], 1u);
    }
    __syncthreads();
    // four threads to a digit; the counters are cleared for the next one
    uint4* c = &s_copies[threadIdx.x >> 2][2 * (threadIdx.x & 3)];
    const uint4 a = c[0], b = c[1];
    c[0] = c[1] = make_uint4(0u, 0u, 0u, 0u);
    uint32_t x = a.x + a.y + a.z + a.w + b.x + b.y + b.z + b.w;
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    if ((threadIdx.x & 3) == 0) s_hist[threadIdx.x >> 2] = x;
    __syncthreads();
    // the first warp, eight digits to a lane from the highest down, finds the
    // one in which the wanted key lies
    if (warp == 0) {
      const uint4 hi = *reinterpret_cast<const uint4*>(&s_hist[252 - 8 * lane]);
      const uint4 lo = *reinterpret_cast<const uint4*>(&s_hist[248 - 8 * lane]);
      const uint32_t h[8] = {hi.w, hi.z, hi.y, hi.x, lo.w, lo.z, lo.y, lo.x};
      uint32_t sum = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) sum += h[k];
      uint32_t incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      uint32_t above = incl - sum;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (above < rank && rank <= above + h[k]) {
          s_found[0] = 255 - (8 * lane + k);
          s_found[1] = rank - above;
          s_found[2] = h[k];
        }
        above += h[k];
      }
    }
    __syncthreads();
    t |= s_found[0] << shift;
    rank = s_found[1];
    equal = s_found[2];
  }

  // equal keys before this warp's, when not all of them survive
  const bool ties = equal != rank;
  uint32_t before = 0;
  if (ties) {
    uint32_t e = 0;
#pragma unroll
    for (int k = 0; k < kSelKeys; ++k) {
      if (k >= per_thread) break;
      e += __popc(__ballot_sync(0xffffffffu, k < mine && key[k] == t));
    }
    if (lane == 0) s_equal[warp] = e;
    __syncthreads();
    before = __reduce_add_sync(0xffffffffu, lane < warp ? s_equal[lane] : 0u);
  }
  const uint32_t lt = lanemask_lt();
#pragma unroll
  for (int k = 0; k < kSelKeys; ++k) {
    if (k >= per_thread) break;
    const bool eq = k < mine && key[k] == t;
    bool keep = k < mine && key[k] >= t;
    if (ties) {
      const uint32_t bal = __ballot_sync(0xffffffffu, eq);
      keep = keep && (!eq || before + __popc(bal & lt) < rank);
      before += __popc(bal);
    }
    if (k < mine) decisions[first + 32 * k] = keep ? 1 : 0;
  }
}

// ------------------------------------------------------------ selection, large

constexpr int kGridFlight = 2;                        // 16-byte reads in flight per lane
constexpr int kWarpStep = 128 * kGridFlight;          // Gaussians a warp takes at a time
constexpr int kCopies = 4;                            // counters per digit, by lane
constexpr int kGridMin = 2 * kSelThreads;             // Gaussians per block at least: fewer
                                                      // blocks meet faster (16,000: 11.2 us
                                                      // against 12.5 with 1,024)
constexpr uint32_t kZeroKey = 0x80000000u;            // the key of a score of 0

// Digit PASS of a key, the most significant first, and the bits above it.
template <int PASS>
struct Digit {
  static constexpr int kShift = PASS == 0 ? 21 : (PASS == 1 ? 10 : 0);
  static constexpr uint32_t kBins = PASS == 2 ? 1024 : 2048;
  __device__ static bool shares(uint32_t key, uint32_t prefix) {
    constexpr int kHigh = PASS == 0 ? 31 : (PASS == 1 ? 21 : 10);
    return PASS == 0 || (key >> kHigh) == (prefix >> kHigh);
  }
  __device__ static uint32_t of(uint32_t key) { return (key >> kShift) & (kBins - 1); }
};

// Scores (bits) and protection of Gaussians i .. i + 3, by one 16-byte and one
// 4-byte read where VEC says the pointers allow it.
struct Raw4 {
  uint32_t b[4], p;
};
template <bool VEC>
__device__ __forceinline__ Raw4 ev_read4(const float* __restrict__ score,
                                         const uint8_t* __restrict__ protect, int64_t i) {
  Raw4 r;
  r.p = 0u;
  if (VEC) {
    const uint4 f = __ldg(reinterpret_cast<const uint4*>(score + i));
    r.b[0] = f.x, r.b[1] = f.y, r.b[2] = f.z, r.b[3] = f.w;
    if (protect) r.p = __ldg(reinterpret_cast<const uint32_t*>(protect + i));
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) r.b[k] = __float_as_uint(__ldg(&score[i + k]));
    if (protect) {
#pragma unroll
      for (int k = 0; k < 4; ++k) r.p |= protect[i + k] ? 0xffu << (8 * k) : 0u;
    }
  }
  return r;
}

// Their keys. Scores that are neither negative nor NaN and unprotected, as
// accumulated weights mostly are, take the short way.
__device__ __forceinline__ void ev_keys4(const Raw4& r, uint32_t (&key)[4]) {
  if (max(max(r.b[0], r.b[1]), max(r.b[2], r.b[3])) <= 0x7f800000u && r.p == 0u) {
#pragma unroll
    for (int k = 0; k < 4; ++k) key[k] = r.b[k] | 0x80000000u;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      key[k] = ev_key(__uint_as_float(r.b[k]), (r.p >> (8 * k)) & 0xffu);
  }
}

// Barrier over the grid, number `turn` of the launch (from 1): false when the
// other blocks did not arrive within the limit.
__device__ __forceinline__ bool grid_barrier(uint32_t* arrived, uint32_t turn, bool* s_ok,
                                             const WaitCfg& wc, uint32_t* status) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    // test hook: this block never arrives
    if ((int64_t)blockIdx.x != wc.stall) atomicAdd(arrived, 1u);
    const uint32_t want = turn * gridDim.x;
    const uint64_t t0 = globaltimer_ns();
    bool ok;
    while (!(ok = *reinterpret_cast<volatile uint32_t*>(arrived) >= want))
      if (globaltimer_ns() - t0 > wc.limit_ns) break;
    if (!ok) atomicOr(status, kStatusTimeout);
    __threadfence();
    *s_ok = ok;
  }
  __syncthreads();
  return *s_ok;
}

struct GridShared {
  uint4 copies[2048];
  uint32_t w[kSelWarps];
  uint32_t found[3];
  bool ok;
};

// The grid's time is latency: about 3 us for each of the three or (with ties at
// the threshold) four phases between barriers -- counting, the counters'
// additions in L2, the barrier, reading the counters back -- and above a few
// million Gaussians the keys' own instructions and reads: 60,000 in 12.5 us,
// 1.2M in 14, 10M in 45 (their 50 MB alone would take 8).
//
// A warp's contiguous part [w0, w1) of the set, taken kWarpStep Gaussians at a
// time, four consecutive ones per lane, as far as `whole`; then up to three
// single ones. HELD: the part is one step, whose keys stay in registers (1.2M
// Gaussians: 13.7 us against 15.3 when they are read again).
template <bool VEC, bool HELD>
struct WarpPart {
  const float* score;
  const uint8_t* protect;
  int64_t w0, w1, whole;
  uint32_t key[kGridFlight][4];
  uint32_t key1;  // of the lane's single one
  bool single;

  __device__ __forceinline__ int64_t at(int64_t i0, int f) const {
    return i0 + 128 * f + 4 * (threadIdx.x & 31);
  }
  __device__ __forceinline__ void read(int64_t i0) {
    Raw4 raw[kGridFlight];  // all reads before the first branch on one
#pragma unroll
    for (int f = 0; f < kGridFlight; ++f) {
      raw[f] = Raw4{{0u, 0u, 0u, 0u}, 0u};
      if (at(i0, f) < whole) raw[f] = ev_read4<VEC>(score, protect, at(i0, f));
    }
#pragma unroll
    for (int f = 0; f < kGridFlight; ++f) ev_keys4(raw[f], key[f]);
  }
  __device__ __forceinline__ void begin(const float* s, const uint8_t* p, int64_t a, int64_t b) {
    score = s, protect = p, w0 = a, w1 = b;
    whole = w0 + ((w1 - w0) & ~(int64_t)3);
    const int64_t i = whole + (threadIdx.x & 31);
    single = i < w1;
    key1 = single ? ev_key_at(score, protect, i) : 0u;
    if (HELD) read(w0);
  }
  __device__ __forceinline__ void step(int64_t i0) {
    if (!HELD) read(i0);
  }
};

// One digit of the wanted key over the block's parts, then over the grid.
// False: gave up at the barrier.
template <int PASS, bool VEC, bool HELD>
__device__ __forceinline__ bool grid_digit(GridShared& s, WarpPart<VEC, HELD>& part,
                                           EvictState* st, uint32_t& prefix, uint32_t& want,
                                           uint32_t& equal, const WaitCfg& wc, uint32_t* status) {
  using D = Digit<PASS>;
  static_assert(kCopies * sizeof(uint32_t) == sizeof(uint4), "one uint4 per digit");
  uint32_t* copies = reinterpret_cast<uint32_t*>(s.copies) + (threadIdx.x & (kCopies - 1));
  for (uint32_t d = threadIdx.x; d < D::kBins; d += kSelThreads)
    s.copies[d] = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
  // Gaussians never seen have a score of exactly 0: those are counted in
  // registers, they would queue up at one counter
  uint32_t zeros = 0;
  auto count = [&](uint32_t key) {
    if (key == kZeroKey)
      ++zeros;
    else if (D::shares(key, prefix))
      atomicAdd(&copies[D::of(key) * kCopies], 1u);
  };
  for (int64_t i0 = part.w0; i0 < part.whole; i0 += kWarpStep) {
    part.step(i0);
#pragma unroll
    for (int f = 0; f < kGridFlight; ++f) {
      if (part.at(i0, f) >= part.whole) continue;
      const uint32_t(&key)[4] = part.key[f];
      // four keys at once that all differ from the wanted one above this digit
      if (PASS > 0 && min(min(key[0] - prefix, key[1] - prefix),
                          min(key[2] - prefix, key[3] - prefix)) >= D::kBins << D::kShift)
        continue;
#pragma unroll
      for (int k = 0; k < 4; ++k) count(key[k]);
    }
  }
  if (part.single) count(part.key1);
  zeros = __reduce_add_sync(0xffffffffu, zeros);
  if ((threadIdx.x & 31) == 0 && zeros && D::shares(kZeroKey, prefix))
    atomicAdd(&copies[D::of(kZeroKey) * kCopies], zeros);
  __syncthreads();
  for (uint32_t d = threadIdx.x; d < D::kBins; d += kSelThreads) {
    const uint4 h = s.copies[d];
    const uint32_t c = h.x + h.y + h.z + h.w;
    if (c) atomicAdd(&st->hist[PASS][d], c);
  }
  if (!grid_barrier(&st->arrived, PASS + 1, &s.ok, wc, status)) return false;
  constexpr int kPer = D::kBins / kSelThreads;
  uint32_t c[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k)
    c[k] = __ldcg(&st->hist[PASS][D::kBins - 1 - (threadIdx.x * kPer + k)]);
  find_digit<kSelWarps, D::kBins, kPer>(c, want, s.w, s.found);
  __syncthreads();
  prefix |= s.found[0] << D::kShift;
  want = s.found[1];
  equal = s.found[2];
  return true;
}

template <bool VEC>
__device__ __forceinline__ void put_decisions(int8_t* d, bool a, bool b, bool c, bool e) {
  if (VEC) {
    *reinterpret_cast<uint32_t*>(d) =
        (a ? 1u : 0u) | (b ? 1u << 8 : 0u) | (c ? 1u << 16 : 0u) | (e ? 1u << 24 : 0u);
  } else {
    d[0] = a, d[1] = b, d[2] = c, d[3] = e;
  }
}

// Every block holds a contiguous share of the set, its warps contiguous parts
// of that (`part` Gaussians, a multiple of 4), so that ties need no more than
// the equal keys before each warp.
template <bool VEC, bool HELD>
__global__ void __launch_bounds__(kSelThreads) k_ev_select_grid(
    const float* __restrict__ score, const uint8_t* __restrict__ protect, int n, int n_keep,
    int64_t part_size, EvictState* st, uint32_t* counts, int8_t* __restrict__ decisions,
    WaitCfg wc, uint32_t* status) {
  __shared__ GridShared s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  WarpPart<VEC, HELD> part;
  {
    const int64_t a = ((int64_t)blockIdx.x * kSelWarps + warp) * part_size;
    part.begin(score, protect, a < n ? a : n, a + part_size < n ? a + part_size : n);
  }
  uint32_t t = 0, rank = (uint32_t)n_keep, equal = 0;
  if (!grid_digit<0>(s, part, st, t, rank, equal, wc, status) ||
      !grid_digit<1>(s, part, st, t, rank, equal, wc, status) ||
      !grid_digit<2>(s, part, st, t, rank, equal, wc, status))
    return;

  if (equal == rank) {
    for (int64_t i0 = part.w0; i0 < part.whole; i0 += kWarpStep) {
      part.step(i0);
#pragma unroll
      for (int f = 0; f < kGridFlight; ++f)
        if (part.at(i0, f) < part.whole)
          put_decisions<VEC>(decisions + part.at(i0, f), part.key[f][0] >= t,
                             part.key[f][1] >= t, part.key[f][2] >= t, part.key[f][3] >= t);
    }
    if (part.single) decisions[part.whole + lane] = part.key1 >= t ? 1 : 0;
    return;
  }

  // not all of the equal keys survive: those before this warp's
  uint32_t x = 0, total, before;
  for (int64_t i0 = part.w0; i0 < part.whole; i0 += kWarpStep) {
    part.step(i0);
#pragma unroll
    for (int f = 0; f < kGridFlight; ++f)
      if (part.at(i0, f) < part.whole) {
#pragma unroll
        for (int k = 0; k < 4; ++k) x += part.key[f][k] == t;
      }
  }
  if (part.single) x += part.key1 == t;
  x = __reduce_add_sync(0xffffffffu, x);
  const uint32_t in_block =
      __shfl_sync(0xffffffffu, block_scan<kSelWarps>(lane == 0 ? x : 0u, s.w, total), 0);
  if (threadIdx.x == 0) counts[blockIdx.x] = total;
  if (!grid_barrier(&st->arrived, 4, &s.ok, wc, status)) return;
  uint32_t y = 0;
  for (unsigned b = threadIdx.x; b < blockIdx.x; b += kSelThreads) y += __ldcg(&counts[b]);
  block_scan<kSelWarps>(y, s.w, before);
  before += in_block;
  for (int64_t i0 = part.w0; i0 < part.whole; i0 += kWarpStep) {
    part.step(i0);
#pragma unroll
    for (int f = 0; f < kGridFlight; ++f) {
      const bool in = part.at(i0, f) < part.whole;
      uint32_t eq = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) eq += in && part.key[f][k] == t;
      uint32_t incl = eq;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t z = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += z;
      }
      uint32_t e = before + incl - eq;
      before += __shfl_sync(0xffffffffu, incl, 31);
      bool keep[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        keep[k] = part.key[f][k] > t || (part.key[f][k] == t && e < rank);
        e += part.key[f][k] == t;
      }
      if (in) put_decisions<VEC>(decisions + part.at(i0, f), keep[0], keep[1], keep[2], keep[3]);
    }
  }
  const bool eq = part.single && part.key1 == t;
  const uint32_t e = before + __popc(__ballot_sync(0xffffffffu, eq) & lanemask_lt());
  if (part.single) decisions[part.whole + lane] = part.key1 > t || (eq && e < rank) ? 1 : 0;
}

// ------------------------------------------------------------ compaction

constexpr int kMoveRows = 256;     // Gaussians (and threads) per block
constexpr int kMoveGroup = 1024;   // blocks per group total
// Up to here every block reads the decisions before its own instead of counts
// from a kernel before it: at 16,000 Gaussians 4.8 us against 5.0, at 24,000
// 5.8 against 5.2 (the reads grow with the square of the set).
constexpr int kMoveDirect = 16384;

// Nonzero bytes of a word.
__device__ __forceinline__ uint32_t nonzero_bytes(uint32_t x) {
  return __popc((((x & 0x7f7f7f7fu) + 0x7f7f7f7fu) | x) & 0x80808080u);
}

// Survivors among decisions[a .. b), added up by `threads` threads of which
// this is number t (their parts, not the total).
__device__ __forceinline__ uint32_t survivors_part(const int8_t* __restrict__ decisions, int64_t a,
                                                   int64_t b, int t, int threads) {
  uint32_t x = 0;
  if ((reinterpret_cast<uintptr_t>(decisions) & 7) == 0 && (a & 7) == 0) {
    for (int64_t i = a + 8 * t; i < b; i += 8 * (int64_t)threads) {
      if (i + 7 < b) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(decisions + i));
        x += nonzero_bytes(w.x) + nonzero_bytes(w.y);
      } else {
        for (int64_t j = i; j < b; ++j) x += decisions[j] != 0;
      }
    }
  } else {
    for (int64_t i = a + t; i < b; i += threads) x += decisions[i] != 0;
  }
  return x;
}

// Eight lanes per kMoveRows Gaussians, 32 of those per block.
__global__ void __launch_bounds__(256) k_ev_count(const int8_t* __restrict__ decisions, int n,
                                                  int blocks, uint32_t* __restrict__ counts,
                                                  uint32_t* __restrict__ groups) {
  let_next_begin();
  __shared__ uint32_t s_w[8];
  const int b = blockIdx.x * 32 + (threadIdx.x >> 3), lane = threadIdx.x & 7;
  const int64_t a = (int64_t)b * kMoveRows, e = a + kMoveRows < n ? a + kMoveRows : n;
  uint32_t x = b < blocks ? survivors_part(decisions, a, e, lane, 8) : 0u, total;
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if (lane == 0 && b < blocks) counts[b] = x;
  if (!groups) return;
  block_scan<8>(lane == 0 ? x : 0u, s_w, total);
  if (threadIdx.x == 0 && total) atomicAdd(&groups[blockIdx.x * 32 / kMoveGroup], total);
}

// One array set: the fields of gs_params.
struct EvSet {
  const float4 *means, *log_scales, *quats;
  const float *logit, *sh;
  float4 *o_means, *o_log_scales, *o_quats;
  float *o_logit, *o_sh;
};
struct EvSets {
  EvSet s[3];
};

// Bound by HBM: 4M Gaussians of SH degree 3 with moments, 85 % kept, move 5.1 GB
// in 0.77 ms, 6.7 TB/s (the plain copy's rate). One array set per block keeps
// small sets on enough SMs (100,000: 20 us; all sets in blocks of 1,024
// Gaussians took 95); 256 rows let every thread fetch one row's 52 bytes of
// small fields at once, then six elements of the SH rows. Rows of PER elements
// of type E there (kNoSh: none); 27 floats go one by one (0.4 of 778,000: 23
// us, 5.3 TB/s with the sectors read in part).
constexpr int kNoSh = -1;
template <typename E, int PER>
__global__ void __launch_bounds__(kMoveRows) k_ev_move(EvSets sets,
                                                       const int8_t* __restrict__ decisions,
                                                       int n, int64_t capacity,
                                                       const uint32_t* counts,
                                                       const uint32_t* groups,
                                                       uint32_t* __restrict__ source,
                                                       int64_t* __restrict__ n_out,
                                                       uint32_t* __restrict__ status) {
  constexpr int kWarps = kMoveRows / 32;
  __shared__ uint32_t s_w[kWarps];
  __shared__ uint8_t s_row[kMoveRows];
  const int64_t first = (int64_t)blockIdx.x * kMoveRows;
  // survivors before this block
  uint32_t part = 0, before;
  const bool keep = first + threadIdx.x < n && decisions[first + threadIdx.x] != 0;
  if (counts) {
    wait_for_previous();  // the counts are there
    const unsigned g = groups ? blockIdx.x / kMoveGroup : 0u;
    for (unsigned b = threadIdx.x; b < g; b += kMoveRows) part += __ldcg(&groups[b]);
    for (unsigned b = g * kMoveGroup + threadIdx.x; b < blockIdx.x; b += kMoveRows)
      part += __ldcg(&counts[b]);
  } else {
    part = survivors_part(decisions, 0, first, threadIdx.x, kMoveRows);
  }
  block_scan<kWarps>(part, s_w, before);
  uint32_t m;
  const uint32_t o = block_scan<kWarps>(keep ? 1u : 0u, s_w, m);
  const int64_t base = before;
  if (keep) s_row[o] = (uint8_t)threadIdx.x;
  __syncthreads();
  if (blockIdx.x == gridDim.x - 1 && blockIdx.y == 0 && threadIdx.x == 0) {
    *n_out = base + m;
    if (base + m > capacity) atomicOr(status, kStatusCapacity);
  }
  // rows past the capacity are not written
  if (base + m > capacity) m = base < capacity ? (uint32_t)(capacity - base) : 0u;

  const EvSet& s = sets.s[blockIdx.y];
  if (threadIdx.x < m) {
    const int64_t i = first + s_row[threadIdx.x], j = base + threadIdx.x;
    const float4 a = __ldg(&s.means[i]), b = __ldg(&s.log_scales[i]), c = __ldg(&s.quats[i]);
    const float d = __ldg(&s.logit[i]);
    s.o_means[j] = a;
    s.o_log_scales[j] = b;
    s.o_quats[j] = c;
    s.o_logit[j] = d;
    if (source && blockIdx.y == 0) source[j] = (uint32_t)i;
  }
  if constexpr (PER > 0) {
    const E* in = reinterpret_cast<const E*>(s.sh) + first * PER;
    E* out = reinterpret_cast<E*>(s.o_sh) + base * PER;
    const uint32_t total = m * PER;
    constexpr int kFlight = 6;  // reads in flight per thread
    for (uint32_t e0 = threadIdx.x; e0 < total; e0 += kFlight * kMoveRows) {
      E v[kFlight];
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        const uint32_t e = e0 + k * kMoveRows, r = e / PER;
        if (e < total) v[k] = __ldg(in + (uint32_t)s_row[r] * PER + (e - r * PER));
      }
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        const uint32_t e = e0 + k * kMoveRows;
        if (e < total) out[e] = v[k];
      }
    }
  }
}

EvSet ev_set(const DpTensorPtrs& in, const DpTensorPtrs& out) {
  auto c4 = [](const float* p) { return reinterpret_cast<const float4*>(p); };
  auto m4 = [](float* p) { return reinterpret_cast<float4*>(p); };
  return EvSet{c4(in.means),  c4(in.log_scales),  c4(in.quats),  in.logit,  in.sh,
               m4(out.means), m4(out.log_scales), m4(out.quats), out.logit, out.sh};
}

int move_blocks(int64_t n) { return (int)((n + kMoveRows - 1) / kMoveRows); }

constexpr int kMaxSms = 1024;  // room for the counts of one block per SM

}  // namespace

int64_t evict_groups(int64_t n) { return (move_blocks(n) + kMoveGroup - 1) / kMoveGroup; }
int64_t evict_counts(int64_t n) {
  return move_blocks(n) > kMaxSms ? move_blocks(n) : kMaxSms;
}

cudaError_t launch_evict_select(const float* score, const uint8_t* protect, int n, int n_keep,
                                int8_t* decisions, const EvictScratch& w, uint32_t* status,
                                const WaitCfg& wc, cudaStream_t stream) {
  if (n == 0) return cudaSuccess;
  if (n_keep <= 0 || n_keep >= n)
    return cudaMemsetAsync(decisions, n_keep > 0 ? 1 : 0, (size_t)n, stream);
  if (n <= kSelMax) {
    k_ev_select<<<1, kSelThreads, 0, stream>>>(score, protect, n, n_keep,
                                               (n + kSelThreads - 1) / kSelThreads, decisions);
    return cudaGetLastError();
  }
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaMemsetAsync(w.state, 0, sizeof(EvictState), stream);
  if (e != cudaSuccess) return e;
  if (sms > kMaxSms) sms = kMaxSms;
  // one block per SM, or one for every kGridMin Gaussians
  const int64_t want = ((int64_t)n + kGridMin - 1) / kGridMin;
  const int blocks = want < sms ? (int)want : sms;
  const int64_t warps = (int64_t)blocks * kSelWarps;
  const int64_t part = ((int64_t)n + 4 * warps - 1) / (4 * warps) * 4;
  const bool vec = (reinterpret_cast<uintptr_t>(score) & 15) == 0 &&
                   (reinterpret_cast<uintptr_t>(protect) & 3) == 0 &&
                   (reinterpret_cast<uintptr_t>(decisions) & 3) == 0;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  attr.id = cudaLaunchAttributeCooperative;  // all blocks at once, or an error
  attr.val.cooperative = 1;
  const bool held = part <= kWarpStep;
  const auto kernel = held ? (vec ? k_ev_select_grid<true, true> : k_ev_select_grid<false, true>)
                           : (vec ? k_ev_select_grid<true, false> : k_ev_select_grid<false, false>);
  return cudaLaunchKernelEx(&cfg, kernel, score, protect, n, n_keep, part, w.state, w.counts,
                            decisions, wc, status);
}

cudaError_t launch_evict_compact(const DpTensorPtrs& p_in, const DpTensorPtrs& m_in,
                                 const DpTensorPtrs& v_in, const int8_t* decisions, int n, int k3,
                                 const DpTensorPtrs& p_out, const DpTensorPtrs& m_out,
                                 const DpTensorPtrs& v_out, int64_t capacity, uint32_t* source,
                                 int64_t* n_out, const EvictScratch& w, uint32_t* status,
                                 cudaStream_t stream) {
  if (n == 0) return cudaMemsetAsync(n_out, 0, sizeof(int64_t), stream);
  const int nb = move_blocks(n);
  uint32_t *counts = nullptr, *groups = nullptr;
  if (n > kMoveDirect) {
    counts = w.counts;
    if (nb > kMoveGroup) {
      groups = w.groups;
      const cudaError_t e =
          cudaMemsetAsync(groups, 0, (size_t)evict_groups(n) * sizeof(uint32_t), stream);
      if (e != cudaSuccess) return e;
    }
    k_ev_count<<<(nb + 31) / 32, 256, 0, stream>>>(decisions, n, nb, counts, groups);
  }
  EvSets sets{};
  sets.s[0] = ev_set(p_in, p_out);
  sets.s[1] = ev_set(m_in, m_out);
  sets.s[2] = ev_set(v_in, v_out);
  const dim3 grid(nb, m_in.means ? 3 : 1);
  const auto move = k3 == 48   ? k_ev_move<float4, 12>
                    : k3 == 27 ? k_ev_move<float, 27>
                    : k3 == 12 ? k_ev_move<float4, 3>
                    : k3 == 3  ? k_ev_move<float, 3>
                               : k_ev_move<float, kNoSh>;
  if (!counts) {
    move<<<grid, kMoveRows, 0, stream>>>(sets, decisions, n, capacity, counts, groups, source,
                                         n_out, status);
    return cudaGetLastError();
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_dependent(move, grid, dim3(kMoveRows), stream, sets, decisions, n, capacity,
                          (const uint32_t*)counts, (const uint32_t*)groups, source, n_out, status);
}

}  // namespace gsb
