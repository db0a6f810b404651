// evict.cu -- eviction under a budget: which Gaussians survive, and their
// compaction, sm_100a.
//
// Selection keeps the n_keep Gaussians with the highest scores (accumulated
// blending weights, or any score), protected ones first, equal scores by the
// lowest index. A score becomes a 32-bit key whose unsigned order is the
// score's; the threshold is the n_keep-th largest key, found digit by digit
// (11 + 11 + 10 bits) from counts alone:
//
//  k_ev_digit   counts one digit of the keys that share the digits found so
//               far; the block that finishes last finds the digit of the
//               n_keep-th key.
//  k_ev_equal   keys equal to the threshold per block (nothing to do when all
//               of them survive).
//  k_ev_write   decisions: keys above the threshold, and the first of the equal
//               ones in index order.
//
// Compaction moves the survivors' rows in index order:
//
//  k_ev_count   survivors per block.
//  k_ev_move    every block adds up the counts before it, lists its survivors
//               and copies their rows; consecutive threads write consecutive
//               elements of the output.

#include <cuda_runtime.h>

#include "gs_internal.h"

namespace gsb {
namespace {

constexpr int kEvThreads = 256;
constexpr int kEvRows = 1024;  // Gaussians per block of the index-ordered kernels
constexpr int kEvPer = kEvRows / kEvThreads;
constexpr int kEvGroup = 1024;  // blocks per group total

// Key of a score: unsigned order = score order, -0 and +0 alike, NaN the
// lowest (0), a protected Gaussian the highest (above +infinity).
__device__ __forceinline__ uint32_t ev_key(const float* score, const uint8_t* protect, int i) {
  if (protect && protect[i]) return 0xffffffffu;
  const uint32_t b = __float_as_uint(score[i]);
  if ((b & 0x7fffffffu) > 0x7f800000u) return 0u;
  if (b == 0x80000000u) return 0x80000000u;
  return (b >> 31) ? ~b : (b | 0x80000000u);
}

// Exclusive sum over the block's threads of x, and the total.
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
  uint32_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kEvThreads / 32; ++w) {
    before += w < warp ? s_w[w] : 0u;
    total += s_w[w];
  }
  return before + incl - x;
}

// Sum of the counts of the blocks before this one, by the whole block: whole
// groups of kEvGroup blocks from their group totals, the rest one by one.
__device__ __forceinline__ uint32_t counts_before(const uint32_t* counts, const uint32_t* groups,
                                                  uint32_t* s_w) {
  const unsigned g = blockIdx.x / kEvGroup;
  uint32_t s = 0, total;
  for (unsigned b = threadIdx.x; b < g; b += kEvThreads) s += groups[b];
  for (unsigned b = g * kEvGroup + threadIdx.x; b < blockIdx.x; b += kEvThreads) s += counts[b];
  block_scan(s, s_w, total);
  return total;
}

template <int PASS>
__global__ void __launch_bounds__(kEvThreads) k_ev_digit(const float* __restrict__ score,
                                                         const uint8_t* __restrict__ protect,
                                                         int n, int n_keep, EvictState* st) {
  constexpr int kShift = PASS == 0 ? 21 : (PASS == 1 ? 10 : 0);
  constexpr uint32_t kBins = PASS == 2 ? 1024 : 2048;
  __shared__ uint32_t s_hist[kBins];
  __shared__ uint32_t s_w[kEvThreads / 32];
  __shared__ bool s_last;
  for (uint32_t d = threadIdx.x; d < kBins; d += kEvThreads) s_hist[d] = 0;
  __syncthreads();
  const uint32_t prefix = PASS == 0 ? 0u : st->prefix;
  for (int64_t i = (int64_t)blockIdx.x * kEvThreads + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * kEvThreads) {
    const uint32_t key = ev_key(score, protect, (int)i);
    constexpr int kHigh = PASS == 0 ? 0 : (PASS == 1 ? 21 : 10);
    if (PASS == 0 || (key >> kHigh) == (prefix >> kHigh))
      atomicAdd(&s_hist[(key >> kShift) & (kBins - 1)], 1u);
  }
  __syncthreads();
  for (uint32_t d = threadIdx.x; d < kBins; d += kEvThreads)
    if (s_hist[d]) atomicAdd(&st->hist[PASS][d], s_hist[d]);
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) s_last = atomicAdd(&st->done[PASS], 1u) == gridDim.x - 1;
  __syncthreads();
  if (!s_last) return;
  // the last block: from the highest digit down, the one in which the wanted
  // key lies
  __threadfence();
  const uint32_t want = PASS == 0 ? (uint32_t)n_keep : st->rank;
  constexpr uint32_t kPer = kBins / kEvThreads;
  uint32_t c[kPer], sum = 0, total;
#pragma unroll
  for (uint32_t k = 0; k < kPer; ++k) {
    c[k] = __ldcg(&st->hist[PASS][kBins - 1 - (threadIdx.x * kPer + k)]);
    sum += c[k];
  }
  uint32_t above = block_scan(sum, s_w, total);
#pragma unroll
  for (uint32_t k = 0; k < kPer; ++k) {
    if (above < want && want <= above + c[k]) {
      st->prefix = prefix | ((kBins - 1 - (threadIdx.x * kPer + k)) << kShift);
      st->rank = want - above;
      if (PASS == 2) st->equal = c[k];
    }
    above += c[k];
  }
}

__global__ void __launch_bounds__(kEvThreads) k_ev_equal(const float* __restrict__ score,
                                                         const uint8_t* __restrict__ protect,
                                                         int n, const EvictState* st,
                                                         uint32_t* __restrict__ counts,
                                                         uint32_t* __restrict__ groups) {
  __shared__ uint32_t s_w[kEvThreads / 32];
  if (st->equal == st->rank) return;
  const uint32_t t = st->prefix;
  uint32_t x = 0, total;
#pragma unroll
  for (int k = 0; k < kEvPer; ++k) {
    const int64_t i = (int64_t)blockIdx.x * kEvRows + k * kEvThreads + threadIdx.x;
    if (i < n) x += ev_key(score, protect, (int)i) == t;
  }
  block_scan(x, s_w, total);
  if (threadIdx.x == 0) {
    counts[blockIdx.x] = total;
    if (total) atomicAdd(&groups[blockIdx.x / kEvGroup], total);
  }
}

__global__ void __launch_bounds__(kEvThreads) k_ev_write(const float* __restrict__ score,
                                                         const uint8_t* __restrict__ protect,
                                                         int n, const EvictState* st,
                                                         const uint32_t* __restrict__ counts,
                                                         const uint32_t* __restrict__ groups,
                                                         int8_t* __restrict__ decisions) {
  __shared__ uint32_t s_w[kEvThreads / 32];
  const uint32_t t = st->prefix, rank = st->rank;
  const bool ties = st->equal != rank;
  uint32_t before = ties ? counts_before(counts, groups, s_w) : 0u;
  for (int k = 0; k < kEvPer; ++k) {
    const int64_t i = (int64_t)blockIdx.x * kEvRows + k * kEvThreads + threadIdx.x;
    const uint32_t key = i < n ? ev_key(score, protect, (int)i) : 0u;
    bool keep = key > t || (key == t && !ties);
    if (ties) {
      uint32_t total;
      const bool eq = i < n && key == t;
      const uint32_t e = before + block_scan(eq, s_w, total);
      keep = keep || (eq && e < rank);
      before += total;
    }
    if (i < n) decisions[i] = keep ? 1 : 0;
  }
}

__global__ void __launch_bounds__(kEvThreads) k_ev_count(const int8_t* __restrict__ decisions,
                                                         int n, uint32_t* __restrict__ counts,
                                                         uint32_t* __restrict__ groups) {
  __shared__ uint32_t s_w[kEvThreads / 32];
  uint32_t x = 0, total;
#pragma unroll
  for (int k = 0; k < kEvPer; ++k) {
    const int64_t i = (int64_t)blockIdx.x * kEvRows + k * kEvThreads + threadIdx.x;
    if (i < n) x += decisions[i] != 0;
  }
  block_scan(x, s_w, total);
  if (threadIdx.x == 0) {
    counts[blockIdx.x] = total;
    if (total) atomicAdd(&groups[blockIdx.x / kEvGroup], total);
  }
}

struct EvArray {
  const void* in;
  void* out;
  int per;   // elements per row
  int wide;  // 16-byte elements (else 4-byte)
};
struct EvArrays {
  EvArray a[15];
  int n;
};

template <typename E>
__device__ __forceinline__ void move_rows(const EvArray& a, const uint16_t* s_row, int64_t first,
                                          int64_t base, uint32_t m) {
  const E* in = static_cast<const E*>(a.in) + first * a.per;
  E* out = static_cast<E*>(a.out) + base * a.per;
  const uint32_t total = m * a.per;
#pragma unroll 4
  for (uint32_t e = threadIdx.x; e < total; e += kEvThreads) {
    const uint32_t r = e / a.per, q = e - r * a.per;
    out[e] = __ldg(in + (uint32_t)s_row[r] * a.per + q);
  }
}

__global__ void __launch_bounds__(kEvThreads) k_ev_move(EvArrays arrays,
                                                        const int8_t* __restrict__ decisions,
                                                        int n, int64_t capacity,
                                                        const uint32_t* __restrict__ counts,
                                                        const uint32_t* __restrict__ groups,
                                                        uint32_t* __restrict__ source,
                                                        int64_t* __restrict__ n_out,
                                                        uint32_t* __restrict__ status) {
  __shared__ uint32_t s_w[kEvThreads / 32];
  __shared__ uint16_t s_row[kEvRows];
  const int64_t base = counts_before(counts, groups, s_w);
  const int64_t first = (int64_t)blockIdx.x * kEvRows;
  uint32_t m = 0;
  for (int k = 0; k < kEvPer; ++k) {
    const int r = k * kEvThreads + threadIdx.x;
    const bool keep = first + r < n && decisions[first + r] != 0;
    uint32_t total;
    const uint32_t o = m + block_scan(keep, s_w, total);
    if (keep) s_row[o] = (uint16_t)r;
    m += total;
  }
  __syncthreads();
  if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) {
    *n_out = base + m;
    if (base + m > capacity) atomicOr(status, kStatusCapacity);
  }
  // rows past the capacity are not written
  if (base + m > capacity) m = base < capacity ? (uint32_t)(capacity - base) : 0u;
  if (source)
    for (uint32_t r = threadIdx.x; r < m; r += kEvThreads)
      source[base + r] = (uint32_t)(first + s_row[r]);
  for (int k = 0; k < arrays.n; ++k) {
    if (arrays.a[k].wide)
      move_rows<float4>(arrays.a[k], s_row, first, base, m);
    else
      move_rows<float>(arrays.a[k], s_row, first, base, m);
  }
}

void add_arrays(EvArrays& v, const DpTensorPtrs& in, const DpTensorPtrs& out, int k3) {
  if (!in.means) return;
  v.a[v.n++] = EvArray{in.means, out.means, 1, 1};
  v.a[v.n++] = EvArray{in.log_scales, out.log_scales, 1, 1};
  v.a[v.n++] = EvArray{in.quats, out.quats, 1, 1};
  v.a[v.n++] = EvArray{in.logit, out.logit, 1, 0};
  if (k3 > 0) {
    const bool wide = k3 % 4 == 0;
    v.a[v.n++] = EvArray{in.sh, out.sh, wide ? k3 / 4 : k3, wide};
  }
}

}  // namespace

int64_t evict_blocks(int64_t n) { return (n + kEvRows - 1) / kEvRows; }
int64_t evict_groups(int64_t n) { return (evict_blocks(n) + kEvGroup - 1) / kEvGroup; }

cudaError_t launch_evict_select(const float* score, const uint8_t* protect, int n, int n_keep,
                                int8_t* decisions, const EvictScratch& w, cudaStream_t stream) {
  if (n == 0) return cudaSuccess;
  if (n_keep <= 0 || n_keep >= n)
    return cudaMemsetAsync(decisions, n_keep > 0 ? 1 : 0, (size_t)n, stream);
  // the group totals follow the state
  const cudaError_t e =
      cudaMemsetAsync(w.state, 0, sizeof(EvictState) + (size_t)evict_groups(n) * 4, stream);
  if (e != cudaSuccess) return e;
  const int nb = (int)evict_blocks(n);
  const int db = nb < 592 ? nb : 592;
  k_ev_digit<0><<<db, kEvThreads, 0, stream>>>(score, protect, n, n_keep, w.state);
  k_ev_digit<1><<<db, kEvThreads, 0, stream>>>(score, protect, n, n_keep, w.state);
  k_ev_digit<2><<<db, kEvThreads, 0, stream>>>(score, protect, n, n_keep, w.state);
  k_ev_equal<<<nb, kEvThreads, 0, stream>>>(score, protect, n, w.state, w.counts, w.groups);
  k_ev_write<<<nb, kEvThreads, 0, stream>>>(score, protect, n, w.state, w.counts, w.groups,
                                            decisions);
  return cudaGetLastError();
}

cudaError_t launch_evict_compact(const DpTensorPtrs& p_in, const DpTensorPtrs& m_in,
                                 const DpTensorPtrs& v_in, const int8_t* decisions, int n, int k3,
                                 const DpTensorPtrs& p_out, const DpTensorPtrs& m_out,
                                 const DpTensorPtrs& v_out, int64_t capacity, uint32_t* source,
                                 int64_t* n_out, const EvictScratch& w, uint32_t* status,
                                 cudaStream_t stream) {
  if (n == 0) return cudaMemsetAsync(n_out, 0, sizeof(int64_t), stream);
  EvArrays v{};
  add_arrays(v, p_in, p_out, k3);
  add_arrays(v, m_in, m_out, k3);
  add_arrays(v, v_in, v_out, k3);
  const cudaError_t e = cudaMemsetAsync(w.groups, 0, (size_t)evict_groups(n) * 4, stream);
  if (e != cudaSuccess) return e;
  const int nb = (int)evict_blocks(n);
  k_ev_count<<<nb, kEvThreads, 0, stream>>>(decisions, n, w.counts, w.groups);
  k_ev_move<<<nb, kEvThreads, 0, stream>>>(v, decisions, n, capacity, w.counts, w.groups, source,
                                           n_out, status);
  return cudaGetLastError();
}

}  // namespace gsb
