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

constexpr int32_t kBadBit = 1 << 30;  // of an item's count: one of its weights was NaN or infinite

// idx[item][0, m) = the kept tokens ascending, idx[item][m, budget) = -1, with
// m = min(n, budget). A radix select over the middle tokens' keys finds the
// threshold and how many equal to it are kept; a warp owns a contiguous run of
// the tokens, counts its keys above and equal to the threshold, and after one
// scan over the warps writes its kept tokens in order. Digits are taken of key
// - smallest key, 11 bits a pass from the highest bit that varies, which
// spreads weights of a few binades over all the bins; it ends early where a
// bin is kept whole. Integer work: the result depends only on the order of the
// weights. With KPT > 0 a thread's KPT keys stay in registers between the
// sweeps (n <= KPT·512); with KPT = 0 they are read again from L2.
template <int KPT>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t wtot[kSelWarps], weq[kSelWarps], wmin[kSelWarps], wmax[kSelWarps];
  __shared__ uint32_t sh_bin, sh_above, sh_count;
  pdl_trigger();
  pdl_wait();
  const int64_t item = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t n = int32_t(min(max(int64_t(a.lens[item / a.heads]), int64_t(0)), a.cap));
  const int32_t budget = int32_t(a.budget);
  int32_t* out = a.idx + item * a.budget;
  const float* w = a.w + item * a.cap;
  const int32_t m = min(n, budget);
  for (int32_t t = m + tid; t < budget; t += kSelThreads) out[t] = -1;
  if (n <= budget) {
    if (tid == 0) a.counts[item] = m;
    for (int32_t t = tid; t < n; t += kSelThreads) out[t] = t;
    return;
  }
  const int32_t lo = int32_t(a.sink), hi = n - int32_t(a.recent);  // middle tokens [lo, hi)
  const uint32_t want = uint32_t(budget - lo - int32_t(a.recent));  // of them, < hi - lo since n > budget
  const int32_t run = ((n + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int32_t r0 = min(n, warp * run), r1 = min(n, r0 + run);

  uint32_t keys[KPT > 0 ? KPT : 1];
  auto raw = [&](int32_t t) { return t >= lo && t < hi ? w[t] : 0.f; };
  if constexpr (KPT > 0) {
    float x[KPT];
#pragma unroll
    for (int i = 0; i < KPT; ++i) x[i] = raw(r0 + 32 * i + lane < r1 ? r0 + 32 * i + lane : -1);
#pragma unroll
    for (int i = 0; i < KPT; ++i) keys[i] = __float_as_uint(x[i]);
  }
  // f(t, key, whether t is a middle token) for the warp's tokens, 32 at a time, in order
  auto sweep = [&](auto&& f) {
    if constexpr (KPT > 0) {
#pragma unroll
      for (int i = 0; i < KPT; ++i) {
        const int32_t t = r0 + 32 * i + lane;
        f(t, keys[i], t < r1 && t >= lo && t < hi);
      }
    } else {
      for (int32_t t = r0 + lane; t - lane < r1; t += 32) {
        const bool mid = t < r1 && t >= lo && t < hi;
        f(t, order_key(raw(mid ? t : -1)), mid);
      }
    }
  };

  uint32_t base = 0, prefix = 0, mask = 0, remaining = want;
  if (want > 0) {
    bool bad = false;
    uint32_t least = 0xFFFFFFFFu, most = 0u;
    if constexpr (KPT > 0) {
#pragma unroll
      for (int i = 0; i < KPT; ++i) {
        bad |= !isfinite(__uint_as_float(keys[i]));
        keys[i] = order_key(__uint_as_float(keys[i]));
      }
    }
    sweep([&](int32_t, uint32_t k, bool mid) {
      if (KPT == 0) bad |= mid && (k <= 0x007FFFFFu || k >= 0xFF800000u);  // the keys of -inf, inf and NaN
      least = min(least, mid ? k : 0xFFFFFFFFu);
      most = max(most, mid ? k : 0u);
    });
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) {
      wmin[warp] = least;
      wmax[warp] = most;
    }
    bad = __syncthreads_or(bad);
    if (tid == 0) a.counts[item] = m | (bad ? kBadBit : 0);
    least = __reduce_min_sync(0xffffffffu, wmin[lane % kSelWarps]);
    most = __reduce_max_sync(0xffffffffu, wmax[lane % kSelWarps]);
    base = least;
    int bits = 32 - __clz(most - least);  // bits not looked at yet
    while (bits > 0) {
      const int digit = min(bits, kDigitBits);
      const int shift = bits - digit;
      const uint32_t dmask = (1u << digit) - 1u;
      for (int b = tid; b < kBins; b += kSelThreads) hist[b] = 0;
      __syncthreads();
      sweep([&](int32_t, uint32_t k, bool mid) {
        const uint32_t d = k - base;
        if (mid && (d & mask) == prefix) atomicAdd(&hist[(d >> shift) & dmask], 1u);
      });
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
#pragma unroll
      for (int v = 0; v < kSelWarps; ++v)
        if (v < warp) before += wtot[v];
      if (before < remaining && remaining <= before + c) {
#pragma unroll
        for (int q = 0; q < kBinsPerThread; ++q) {
          if (before + cnt[q] >= remaining) {
            sh_bin = uint32_t(kBins - 1 - kBinsPerThread * tid - q);
            sh_above = before;
            sh_count = cnt[q];
            break;
          }
          before += cnt[q];
        }
      }
      __syncthreads();
      prefix |= sh_bin << shift;
      mask |= dmask << shift;
      remaining -= sh_above;
      bits = shift;
      if (sh_count == remaining) break;  // the whole bin stays
    }
  } else if (tid == 0) {
    a.counts[item] = m;
  }

  // Of the middle tokens those with (key - base) & mask above prefix stay, and
  // the first `remaining` equal to it (mask = 0: every key is the same).
  uint32_t above = 0, equal = 0;
  sweep([&](int32_t t, uint32_t k, bool mid) {
    const bool always = t < r1 && !mid;
    const uint32_t d = (k - base) & mask;
    above += __popc(__ballot_sync(0xffffffffu, always || (mid && want > 0 && d > prefix)));
    equal += __popc(__ballot_sync(0xffffffffu, mid && want > 0 && d == prefix));
  });
  if (lane == 0) {
    wtot[warp] = above;
    weq[warp] = equal;
  }
  __syncthreads();
  uint32_t eq_before = 0, pos = 0;
#pragma unroll
  for (int v = 0; v < kSelWarps; ++v)
    if (v < warp) {
      pos += wtot[v] + (eq_before < remaining ? min(weq[v], remaining - eq_before) : 0u);
      eq_before += weq[v];
    }
  const uint32_t below = (1u << lane) - 1u;
  sweep([&](int32_t t, uint32_t k, bool mid) {
    const bool always = t < r1 && !mid;
    const uint32_t d = (k - base) & mask;
    const uint32_t eq = __ballot_sync(0xffffffffu, mid && want > 0 && d == prefix);
    const bool keep = always || (mid && want > 0 &&
                                 (d > prefix || (d == prefix && eq_before + __popc(eq & below) < remaining)));
    const uint32_t kept = __ballot_sync(0xffffffffu, keep);
    if (keep) out[pos + __popc(kept & below)] = t;
    pos += __popc(kept);
    eq_before += __popc(eq);
  });
}

// dst row t of plane p = src row idx[t]. blockIdx.y below copy_blocks: a block
// of rows, all planes that are copied. The rest: a plane moved in place (src ==
// dst), one CTA per column slice, which walks the rows in order: a block of
// rows is read into registers, and after a barrier written. Kept tokens
// ascend, so idx[t] >= t: a block's writes stay below every later block's
// reads, and the next block can be on its way meanwhile.
constexpr int kMoveThreads = 256;
constexpr int kMoveVecs = 4;  // vectors in flight per thread
constexpr int kMoveRows = 256;

struct MoveUnit {
  int16_t plane;
  int16_t vec;         // bytes per vector
  int32_t col0, cols;  // vectors
};
constexpr int kSlices = 8;  // column slices per plane at most
struct MovePlan {
  MoveUnit unit[kMaxPlanes * kSlices];  // planes moved in place
  int16_t copy[kMaxPlanes];             // planes copied
  int32_t n_copy;
  int32_t rows, copy_blocks;            // rows per CTA (at most kMoveRows), CTAs of an item's rows
};

template <typename VecT>
__device__ __forceinline__ void copy_rows(const EvictArgs& a, const EvictPlane& pl, int64_t item, int32_t row0,
                                          int32_t rows, const int32_t* from) {
  const int32_t nv = int32_t(pl.row_bytes / int64_t(sizeof(VecT)));
  const VecT* src = static_cast<const VecT*>(pl.src) + item * a.cap * nv;
  VecT* dst = static_cast<VecT*>(pl.dst) + (item * a.cap_out + row0) * nv;
  const int32_t total = rows * nv;  // at most 256 x 2048
  const bool pow2 = (nv & (nv - 1)) == 0;
  const int sh = 31 - __clz(nv);
  for (int32_t i0 = threadIdx.x; i0 < total; i0 += kMoveVecs * kMoveThreads) {
    VecT v[kMoveVecs];
#pragma unroll
    for (int u = 0; u < kMoveVecs; ++u) {
      const int32_t i = i0 + u * kMoveThreads;
      if (i < total) {
        const int32_t r = pow2 ? i >> sh : i / nv;
        v[u] = src[int64_t(from[r]) * nv + (i - r * nv)];
      }
    }
#pragma unroll
    for (int u = 0; u < kMoveVecs; ++u) {
      const int32_t i = i0 + u * kMoveThreads;
      if (i < total) dst[i] = v[u];
    }
  }
}

template <typename VecT>
__device__ __forceinline__ void move_rows(const EvictArgs& a, const EvictPlane& pl, int64_t item, int32_t m, int col0,
                                          int cols) {
  const int64_t nv = pl.row_bytes / int64_t(sizeof(VecT));
  VecT* plane = static_cast<VecT*>(pl.dst) + item * a.cap * nv;
  const int32_t* idx = a.idx + item * a.budget;
  const int per = kMoveThreads / cols;  // rows a pass of the block's threads covers
  const int r_in = threadIdx.x / cols, c = col0 + threadIdx.x % cols;
  VecT v[2][kMoveVecs];
  auto load = [&](VecT (&x)[kMoveVecs], int32_t base) {
#pragma unroll
    for (int u = 0; u < kMoveVecs; ++u) {
      const int32_t t = base + u * per + r_in;
      if (r_in < per && t < m) x[u] = plane[int64_t(idx[t]) * nv + c];
    }
  };
  auto store = [&](const VecT (&x)[kMoveVecs], int32_t base) {
#pragma unroll
    for (int u = 0; u < kMoveVecs; ++u) {
      const int32_t t = base + u * per + r_in;
      if (r_in < per && t < m) plane[int64_t(t) * nv + c] = x[u];
    }
  };
  const int32_t step = per * kMoveVecs;
  load(v[0], 0);
  for (int32_t base = 0; base < m; base += 2 * step) {
    load(v[1], base + step);
    __syncthreads();
    store(v[0], base);
    load(v[0], base + 2 * step);
    __syncthreads();
    store(v[1], base + step);
  }
}

// IN_PLACE: some plane is. Without that path six blocks fit an SM, which moves
// 290 MB of 4-bit rows in 52 us instead of 57 us.
template <bool IN_PLACE>
__global__ void __launch_bounds__(kMoveThreads, IN_PLACE ? 3 : 6)
evict_move_kernel(const EvictArgs a, const MovePlan plan) {
  __shared__ int32_t from[kMoveRows];
  pdl_trigger();
  pdl_wait();
  const int64_t item = blockIdx.x;
  const int tid = threadIdx.x;
  const int32_t m = a.counts[item] & (kBadBit - 1);
  if (blockIdx.y == 0) {
    // nothing reads lens any more, which lens_out may be
    if (tid == 0 && item % a.heads == 0) a.lens_out[item / a.heads] = m;
    if (item == 0) {
      int bad = 0;
      for (int64_t i = tid; i < a.batch * a.heads; i += kMoveThreads) bad |= a.counts[i] & kBadBit;
      bad = __syncthreads_or(bad);
      if (tid == 0) *a.status = bad ? RMM_NONFINITE_BIT : 0u;
    }
  }
  if (int32_t(blockIdx.y) < plan.copy_blocks) {
    const int32_t row0 = int32_t(blockIdx.y) * plan.rows;
    const int32_t rows = min(plan.rows, m - row0);
    if (rows <= 0) return;
    for (int32_t i = tid; i < rows; i += kMoveThreads) from[i] = a.idx[item * a.budget + row0 + i];
    __syncthreads();
    for (int p = 0; p < plan.n_copy; ++p) {
      const EvictPlane pl = a.plane[plan.copy[p]];
      const bool vec16 =
          ((pl.row_bytes | int64_t(reinterpret_cast<uintptr_t>(pl.src) | reinterpret_cast<uintptr_t>(pl.dst))) & 15) == 0;
      if (vec16)
        copy_rows<uint4>(a, pl, item, row0, rows, from);
      else
        copy_rows<uint32_t>(a, pl, item, row0, rows, from);
    }
    return;
  }
  if constexpr (!IN_PLACE) return;
  const int unit = int32_t(blockIdx.y) - plan.copy_blocks;
  // the last kept row at its own index: every row is where it belongs
  if (a.n_planes == plan.n_copy || m == 0 || a.idx[item * a.budget + m - 1] == m - 1) return;
  const MoveUnit u = plan.unit[unit];
  if (u.vec == 16)
    move_rows<uint4>(a, a.plane[u.plane], item, m, u.col0, u.cols);
  else
    move_rows<uint32_t>(a, a.plane[u.plane], item, m, u.col0, u.cols);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st) {
  const int64_t items = a.batch * a.heads;
  const dim3 grid(static_cast<unsigned>(items)), block(kSelThreads);
  cudaError_t e;
  if (a.cap <= 4 * kSelThreads)
    e = launch_pdl(evict_select_kernel<4>, grid, block, 0, st, dim3(0, 0, 0), a);
  else if (a.cap <= 16 * kSelThreads)
    e = launch_pdl(evict_select_kernel<16>, grid, block, 0, st, dim3(0, 0, 0), a);
  else
    e = launch_pdl(evict_select_kernel<0>, grid, block, 0, st, dim3(0, 0, 0), a);
  if (e != cudaSuccess) return e;
  MovePlan plan;
  plan.n_copy = 0;
  int units = 0;
  for (int p = 0; p < a.n_planes; ++p) {
    const EvictPlane& pl = a.plane[p];
    if (pl.src != pl.dst) {
      plan.copy[plan.n_copy++] = int16_t(p);
      continue;
    }
    const bool vec16 = pl.row_bytes % 16 == 0 && (reinterpret_cast<uintptr_t>(pl.dst) & 15u) == 0;
    const int vec = vec16 ? 16 : 4;
    const int64_t nv = pl.row_bytes / vec;  // at most kSlices * kMoveThreads
    // narrow slices, so that more CTAs share the plane
    const int64_t slice = std::max<int64_t>((nv + kSlices - 1) / kSlices, vec16 ? 4 : 16);
    for (int64_t c = 0; c < nv; c += slice)
      plan.unit[units++] = MoveUnit{int16_t(p), int16_t(vec), int32_t(c), int32_t(std::min(slice, nv - c))};
  }
  // as many rows per CTA as leave four CTAs per SM
  plan.rows = kMoveRows;
  while (plan.rows > 32 && items * ((a.budget + plan.rows - 1) / plan.rows) < 4 * 148) plan.rows /= 2;
  plan.copy_blocks = plan.n_copy > 0 ? int32_t((a.budget + plan.rows - 1) / plan.rows) : 0;
  const dim3 grid2(unsigned(items), unsigned(std::max(plan.copy_blocks + units, 1)));
  if (units > 0)
    return launch_pdl(evict_move_kernel<true>, grid2, dim3(kMoveThreads), 0, st, dim3(0, 0, 0), a, plan);
  return launch_pdl(evict_move_kernel<false>, grid2, dim3(kMoveThreads), 0, st, dim3(0, 0, 0), a, plan);
}

}  // namespace rmm
