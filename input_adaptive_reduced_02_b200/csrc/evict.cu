// Eviction from a cache by accumulated weight: per (sequence, head) the rows
// of the first `sink` and last `recent` tokens and, of the tokens between, the
// ones of greatest weight stay, `budget` rows in all, moved together in their
// order. It is the selection of the reduced P·V ("Estratégia de Seleção" on
// the gist.science summary of "Reduced Matrix Multiplication: Input-Adaptive
// Matrix-Product Reduction for LLM Inference": keep the highest-scoring keys,
// ties to the lower index), with the score summed over the queries so far.
//
// Two launches. The selection runs one CTA per (sequence, head); the move
// copies the kept rows of every plane through the indices and is bound by HBM:
// 4·n bytes of weights and 2·row_bytes per kept row and plane.
#include <algorithm>

#include "rmm_device.cuh"
#include "rmm_internal.h"

namespace rmm {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kDigitBits = 11;
constexpr int kBins = 1 << kDigitBits;
constexpr int kBinsPerThread = kBins / kSelThreads;

// Order-preserving map from f32 to u32 (larger weight, larger key; -0 equals +0).
__device__ __forceinline__ uint32_t order_key(float x) {
  uint32_t u = __float_as_uint(x);
  if ((u & 0x7FFFFFFFu) == 0) u = 0;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// idx[item][0, m) = the kept tokens ascending, idx[item][m, budget) = -1, with
// m = min(n, budget). A radix select over the middle tokens' keys, 11 bits a
// pass from the top, finds the threshold key and how many equal to it are
// kept; a warp then owns a contiguous run of the tokens, counts its keys above
// and equal to the threshold, and after one scan over the warps writes its
// kept tokens in order. Integer work: the result depends only on the order of
// the weights. Keys are re-read from global memory (L2) in every sweep, so any
// capacity works.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t wtot[kSelWarps], weq[kSelWarps];
  __shared__ uint32_t sh_bin, sh_above;
  pdl_trigger();
  pdl_wait();
  const int64_t item = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t n = int32_t(min(max(int64_t(a.lens[item / a.heads]), int64_t(0)), a.cap));
  const int32_t budget = int32_t(a.budget);
  int32_t* out = a.idx + item * a.budget;
  const float* w = a.w + item * a.cap;
  const int32_t m = min(n, budget);
  if (tid == 0) a.counts[item] = m;
  for (int32_t t = m + tid; t < budget; t += kSelThreads) out[t] = -1;
  if (n <= budget) {
    for (int32_t t = tid; t < n; t += kSelThreads) out[t] = t;
    return;
  }
  const int32_t lo = int32_t(a.sink), hi = n - int32_t(a.recent);  // middle tokens [lo, hi)
  const uint32_t want = uint32_t(budget - lo - int32_t(a.recent));  // of them, < hi - lo since n > budget

  uint32_t prefix = 0, mask = 0, remaining = want;
  bool bad = false;
  if (want > 0) {
    int shift = 32 - kDigitBits;  // 21, 10, then the low 10 bits
    for (int pass = 0; pass < 3; ++pass) {
      const uint32_t dmask = pass < 2 ? kBins - 1u : (1u << 10) - 1u;
      for (int b = tid; b < kBins; b += kSelThreads) hist[b] = 0;
      __syncthreads();
      for (int32_t t = lo + tid; t < hi; t += kSelThreads) {
        const float x = w[t];
        if (pass == 0) bad |= !isfinite(x);
        const uint32_t k = order_key(x);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & dmask], 1u);
      }
      __syncthreads();
      // thread t owns bins kBins-1-4t .. kBins-4-4t, highest first
      uint32_t cnt[kBinsPerThread], c = 0;
#pragma unroll
      for (int q = 0; q < kBinsPerThread; ++q) {
        cnt[q] = hist[kBins - 1 - kBinsPerThread * tid - q];
        c += cnt[q];
      }
      uint32_t incl = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) wtot[warp] = incl;
      __syncthreads();
      uint32_t before = incl - c;
      for (int v = 0; v < warp; ++v) before += wtot[v];
      if (before < remaining && remaining <= before + c) {
#pragma unroll
        for (int q = 0; q < kBinsPerThread; ++q) {
          if (before + cnt[q] >= remaining) {
            sh_bin = uint32_t(kBins - 1 - kBinsPerThread * tid - q);
            sh_above = before;
            break;
          }
          before += cnt[q];
        }
      }
      __syncthreads();
      prefix |= sh_bin << shift;
      mask |= dmask << shift;
      remaining -= sh_above;
      shift = pass == 0 ? 10 : 0;
    }
    if (__syncthreads_or(bad) && tid == 0) status_or(a.status, RMM_NONFINITE_BIT);
  }

  // prefix is now the threshold key (want > 0): keys above it stay, and the
  // first `remaining` keys equal to it
  const int32_t run = ((n + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int32_t r0 = min(n, warp * run), r1 = min(n, r0 + run);
  uint32_t above = 0, equal = 0;
  for (int32_t t = r0 + lane; t - lane < r1; t += 32) {
    const bool in = t < r1;
    const bool always = in && (t < lo || t >= hi);
    const uint32_t k = in && !always && want > 0 ? order_key(w[t]) : 0u;
    const bool mid = in && !always && want > 0;
    above += __popc(__ballot_sync(0xffffffffu, always || (mid && k > prefix)));
    equal += __popc(__ballot_sync(0xffffffffu, mid && k == prefix));
  }
  if (lane == 0) {
    wtot[warp] = above;
    weq[warp] = equal;
  }
  __syncthreads();
  uint32_t eq_before = 0, pos = 0;
  for (int v = 0; v < warp; ++v) {
    pos += wtot[v] + (eq_before < remaining ? min(weq[v], remaining - eq_before) : 0u);
    eq_before += weq[v];
  }
  for (int32_t t = r0 + lane; t - lane < r1; t += 32) {
    const bool in = t < r1;
    const bool always = in && (t < lo || t >= hi);
    const bool mid = in && !always && want > 0;
    const uint32_t k = mid ? order_key(w[t]) : 0u;
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t eq = __ballot_sync(0xffffffffu, mid && k == prefix);
    const bool keep = always || (mid && (k > prefix || (k == prefix && eq_before + __popc(eq & below) < remaining)));
    const uint32_t kept = __ballot_sync(0xffffffffu, keep);
    if (keep) out[pos + __popc(kept & below)] = t;
    pos += __popc(kept);
    eq_before += __popc(eq);
  }
}

// dst row t of plane p = src row idx[t]. One CTA per (row block, plane and
// column slice, item). A plane that is moved in place (src == dst) is given
// to one CTA per column slice, which walks the rows in order: a block of rows
// is read into registers, and after a barrier written. Kept tokens ascend, so
// idx[t] >= t: a block's writes stay below every later block's reads.
constexpr int kMoveThreads = 256;
constexpr int kMoveVecs = 4;  // vectors in flight per thread

template <typename VecT>
__device__ __forceinline__ void move_rows(const EvictArgs& a, const EvictPlane& pl, int64_t item, int32_t m,
                                          int32_t row0, int32_t rows, int col0, int cols) {
  const int64_t nv = pl.row_bytes / int64_t(sizeof(VecT));
  const VecT* src = static_cast<const VecT*>(pl.src) + item * a.cap * nv;
  VecT* dst = static_cast<VecT*>(pl.dst) + item * a.cap_out * nv;
  const int32_t* idx = a.idx + item * a.budget;
  const bool in_place = pl.src == pl.dst;
  const int32_t end = min(m, row0 + rows);
  const int per = kMoveThreads / cols;            // rows a pass of the block's threads covers
  const int r_in = threadIdx.x / cols, c = col0 + threadIdx.x % cols;
  const bool live = r_in < per;
  for (int32_t base = row0; base < end; base += per * kMoveVecs) {
    VecT v[kMoveVecs];
    int32_t t[kMoveVecs];
#pragma unroll
    for (int u = 0; u < kMoveVecs; ++u) {
      t[u] = base + u * per + r_in;
      if (live && t[u] < end) v[u] = src[int64_t(idx[t[u]]) * nv + c];
    }
    if (in_place) __syncthreads();
#pragma unroll
    for (int u = 0; u < kMoveVecs; ++u)
      if (live && t[u] < end) dst[int64_t(t[u]) * nv + c] = v[u];
  }
}

struct MoveUnit {
  int16_t plane;
  int16_t vec;         // bytes per vector
  int32_t col0, cols;  // vectors
};
constexpr int kSlices = 8;  // column slices per plane at most
struct MovePlan {
  MoveUnit unit[kMaxPlanes * kSlices];
  int32_t rows;  // rows per CTA for planes that are not moved in place
};

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a, const MovePlan plan) {
  pdl_trigger();
  pdl_wait();
  const int64_t item = blockIdx.x;
  const int32_t m = a.counts[item];
  // lens is read here for the last time, and only by the thread that writes lens_out, which may be lens
  if (blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0 && item % a.heads == 0) a.lens_out[item / a.heads] = m;
  if (a.n_planes == 0) return;
  const MoveUnit u = plan.unit[blockIdx.y];
  const EvictPlane pl = a.plane[u.plane];
  const bool in_place = pl.src == pl.dst;
  // in place with the last kept row at its own index: every row is where it belongs
  if (m == 0 || (in_place && (blockIdx.z > 0 || a.idx[item * a.budget + m - 1] == m - 1))) return;
  const int32_t row0 = in_place ? 0 : int32_t(blockIdx.z) * plan.rows;
  const int32_t rows = in_place ? m : plan.rows;
  if (row0 >= m) return;
  if (u.vec == 16)
    move_rows<uint4>(a, pl, item, m, row0, rows, u.col0, u.cols);
  else
    move_rows<uint32_t>(a, pl, item, m, row0, rows, u.col0, u.cols);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st) {
  const int64_t items = a.batch * a.heads;
  cudaError_t e = launch_pdl(evict_select_kernel, dim3(unsigned(items)), dim3(kSelThreads), 0, st, dim3(0, 0, 0), a);
  if (e != cudaSuccess) return e;
  MovePlan plan;
  int units = 0;
  bool all_in_place = true;
  for (int p = 0; p < a.n_planes; ++p) {
    const EvictPlane& pl = a.plane[p];
    const bool vec16 = pl.row_bytes % 16 == 0 && ((reinterpret_cast<uintptr_t>(pl.src) |
                                                   reinterpret_cast<uintptr_t>(pl.dst)) & 15u) == 0;
    const int vec = vec16 ? 16 : 4;
    const int64_t nv = pl.row_bytes / vec;  // at most kSlices * kMoveThreads
    const bool in_place = pl.src == pl.dst;
    all_in_place &= in_place;
    // in place: narrow slices, so that more CTAs share the plane
    const int64_t slice = in_place ? std::max<int64_t>((nv + kSlices - 1) / kSlices, vec16 ? 4 : 16) : kMoveThreads;
    for (int64_t c = 0; c < nv; c += slice)
      plan.unit[units++] = MoveUnit{int16_t(p), int16_t(vec), int32_t(c), int32_t(std::min(slice, nv - c))};
  }
  plan.rows = 128;
  const unsigned bz = all_in_place ? 1u : unsigned((a.budget + plan.rows - 1) / plan.rows);
  return launch_pdl(evict_move_kernel, dim3(unsigned(items), unsigned(std::max(units, 1)), bz), dim3(kMoveThreads), 0,
                    st, dim3(0, 0, 0), a, plan);
}

}  // namespace rmm
