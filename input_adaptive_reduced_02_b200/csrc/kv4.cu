// A cache of keys and values held in 4 bits: writing tokens into it, and one
// decode step's attention over it (P·V and Q·Kᵀ of one query token, "Escopo de
// Aplicação" on the gist.science summary of "Reduced Matrix Multiplication:
// Input-Adaptive Matrix-Product Reduction for LLM Inference"; the pages name
// no cache format, the one here is this library's).
//
// A row of d channels is cut into groups of 32. A group holds a bf16 minimum
// m, a bf16 step s = bf16((max - min) / 15) and per channel a 4-bit code
// c = clamp(rint((x - m) / s), 0, 15), 0 where s is 0; it stands for m + s·c.
#include <algorithm>

#include "rmm_device.cuh"
#include "rmm_internal.h"

namespace rmm {
namespace {

// The last i in [0, n) with cu[i] <= t (cu[0] <= t; repeated boundaries are
// empty sequences, which the last one passes over).
__device__ __forceinline__ int64_t find_seq(const int32_t* cu, int64_t n, int64_t t) {
  int64_t lo = 0, hi = n - 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) >> 1;
    if (int64_t(cu[mid]) <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// ---------------------------------------------------------------- store
// A thread quantises 8 channels, four neighbouring lanes a group.
template <typename T>
__global__ void __launch_bounds__(256) kv4_store_kernel(const Kv4StoreArgs a) {
  pdl_trigger();
  pdl_wait();
  const int32_t ng = int32_t(a.d / kKv4Group);
  const int32_t per_row = 4 * ng;
  const int64_t total = a.T * a.h_kv * 2 * per_row;
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t ic = i < total ? i : total - 1;  // surplus threads repeat the last unit and store nothing
  const int32_t u = int32_t(ic % per_row);
  int64_t r = ic / per_row;
  const int kv = int(r & 1);
  r >>= 1;
  const int64_t h = r % a.h_kv, t = r / a.h_kv;
  int64_t b = t, in_seq = 0;
  bool live = i < total;
  if (a.cu) {
    b = find_seq(a.cu, a.n_seq, t);
    in_seq = t - a.cu[b];
    live = live && in_seq >= 0 && t < a.cu[b + 1];
  }
  const int64_t slot = int64_t(a.start[b]) + in_seq;
  const bool in_cache = slot >= 0 && slot < a.cap;
  const int w = u >> 2, j = u & 3;  // group, quarter of the group
  const TokView& x = kv ? a.v : a.k;
  const T* src = static_cast<const T*>(x.ptr) + t * x.ts + h * x.hs + 8 * u;
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = elem_to_f32(src[e]);
  float lo = f[0], hi = f[0];
  bool bad = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    lo = fminf(lo, f[e]);
    hi = fmaxf(hi, f[e]);
    bad |= !isfinite(f[e]);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  // (step, minimum) as stored; IEEE divisions, so that the codes depend on nothing but the values
  const uint32_t sm = pack_bf16x2(__fdiv_rn(hi - lo, 15.0f), lo);
  const float step = __uint_as_float(sm << 16), mn = __uint_as_float(sm & 0xFFFF0000u);
  uint32_t codes = 0;  // nibble e: channel 8u + e
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float q = step > 0.f ? rintf(__fdiv_rn(f[e] - mn, step)) : 0.f;
    codes |= uint32_t(fminf(fmaxf(q, 0.f), 15.f)) << (4 * e);
  }
  // the values' half-words need one nibble from each of the group's four lanes
  uint32_t half[2] = {0u, 0u};  // half-words r = 2j, 2j + 1 of group w
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const uint32_t c = __shfl_sync(0xffffffffu, codes, (threadIdx.x & 28) | s);
    half[0] |= ((c >> (8 * j)) & 15u) << (4 * s);
    half[1] |= ((c >> (8 * j + 4)) & 15u) << (4 * s);
  }
  if (!live) return;
  if (bad) status_or(a.status, RMM_NONFINITE_BIT);
  if (!in_cache) {
    status_or(a.status, RMM_RANGE_BIT);
    return;
  }
  const int64_t row = (b * a.h_kv + h) * a.cap + slot;
  uint32_t* scales = reinterpret_cast<uint32_t*>(kv ? a.c.vs : a.c.ks);
  if (j == 0) scales[row * ng + w] = sm;
  if (!kv) {
    reinterpret_cast<uint32_t*>(a.c.kc)[row * per_row + j * ng + w] = codes;
    if (u == 0 && a.w) a.w[row] = a.w_new ? a.w_new[h * a.T + t] : 0.f;
  } else {
    uint16_t* v = reinterpret_cast<uint16_t*>(a.c.vc) + row * (2 * per_row);
    v[(2 * j) * ng + w] = uint16_t(half[0]);
    v[(2 * j + 1) * ng + w] = uint16_t(half[1]);
  }
}

// ---------------------------------------------------------------- attention
struct Kv4Dev {
  Kv4AttnArgs a;
  float* ml;      // [batch][h_q][max_splits][2] (maximum in log2 units, sum)
  float* po;      // [batch][h_q][max_splits][d] unnormalised
  float* scores;  // [batch][h_q][cap] log2 units, or null
  int32_t split_len, max_splits;
};

__device__ __forceinline__ int32_t seq_len(const Kv4AttnArgs& a, int64_t b) {
  return int32_t(min(max(int64_t(a.lens[b]), int64_t(0)), a.cap));
}

constexpr int kSimpleThreads = 128;

// One CTA per (split, query head, sequence): a thread a token for the scores,
// then a thread a channel for the sums.
__global__ void __launch_bounds__(kSimpleThreads) kv4_attn_split_kernel(const Kv4Dev p) {
  __shared__ float q[kKv4MaxD];
  __shared__ float pr[kSimpleThreads];
  __shared__ float red[4];
  pdl_trigger();
  pdl_wait();
  const Kv4AttnArgs& a = p.a;
  const int split = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t hq = blockIdx.y, b = blockIdx.z;
  const int64_t h = hq / (a.h_q / a.h_kv);
  const int32_t d = int32_t(a.d), ng = d / 32;
  if (split == 0 && hq == 0 && b == 0 && tid == 0) *static_cast<uint32_t*>(a.workspace) = 0u;
  const int32_t len = seq_len(a, b);
  const int32_t t0 = split * p.split_len, t1 = min(len, t0 + p.split_len);
  if (t0 >= t1) return;
  if (tid < d)
    q[tid] = bf16_to_f32(static_cast<const uint16_t*>(a.q)[b * a.q_ss + hq * a.q_hs + tid]) *
             (a.scale * 1.4426950408889634f);
  __syncthreads();
  const int64_t row0 = (b * a.h_kv + h) * a.cap;
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (int32_t base = t0; base < t1; base += kSimpleThreads) {
    const int32_t t = base + tid;
    float x = -INFINITY;
    if (t < t1) {
      x = 0.f;
      const uint32_t* kc = reinterpret_cast<const uint32_t*>(a.c.kc) + (row0 + t) * (4 * ng);
      const uint32_t* ks = reinterpret_cast<const uint32_t*>(a.c.ks) + (row0 + t) * ng;
      for (int w = 0; w < ng; ++w) {
        const float s = __uint_as_float(ks[w] << 16), mn = __uint_as_float(ks[w] & 0xFFFF0000u);
        for (int j = 0; j < 4; ++j) {
          const uint32_t c = kc[j * ng + w];
          for (int e = 0; e < 8; ++e) x += q[32 * w + 8 * j + e] * fmaf(s, float((c >> (4 * e)) & 15u), mn);
        }
      }
      if (p.scores) p.scores[(b * a.h_q + hq) * a.cap + t] = x;
    }
    float mx = x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (lane == 0) red[warp] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float m2 = fmaxf(m, mx);
    const float corr = exp2f(m - m2);
    pr[tid] = t < t1 ? exp2f(x - m2) : 0.f;
    __syncthreads();
    m = m2;
    l *= corr;
    acc *= corr;
    const int32_t cnt = min(kSimpleThreads, t1 - base);
    const int w = tid / 32, i = tid % 32 / 8, r = tid % 8;
    for (int k = 0; k < cnt; ++k) {
      l += pr[k];
      if (tid < d) {
        const int64_t row = row0 + base + k;
        const uint32_t c = reinterpret_cast<const uint16_t*>(a.c.vc)[row * (8 * ng) + r * ng + w];
        const uint32_t sm = reinterpret_cast<const uint32_t*>(a.c.vs)[row * ng + w];
        acc += pr[k] * fmaf(__uint_as_float(sm << 16), float((c >> (4 * i)) & 15u), __uint_as_float(sm & 0xFFFF0000u));
      }
    }
    __syncthreads();
  }
  const int64_t part = (b * a.h_q + hq) * p.max_splits + split;
  if (tid == 0) {
    p.ml[2 * part] = m;
    p.ml[2 * part + 1] = l;
  }
  if (tid < d) p.po[part * d + tid] = acc;
}

// Joins the splits. Blocks [0, batch·h_q): O and the log-sum-exp of one head.
// The rest, w_out = w_in + the group's probabilities, 512 tokens each.
constexpr int kJoinThreads = 128;
constexpr int kJoinTokens = 512;

// max and sum over the splits of one head (log2 units): every thread gets both
__device__ __forceinline__ float2 join_ml(const float* ml, int32_t splits, int lane) {
  float m = -INFINITY;
  for (int s = lane; s < splits; s += 32) m = fmaxf(m, ml[2 * s]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float l = 0.f;
  for (int s = lane; s < splits; s += 32) l += ml[2 * s + 1] * exp2f(ml[2 * s] - m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  return make_float2(m, l);
}

__global__ void __launch_bounds__(kJoinThreads) kv4_attn_join_kernel(const Kv4Dev p, int64_t o_blocks) {
  extern __shared__ float lse2[];  // [h_q / h_kv]
  pdl_trigger();
  pdl_wait();
  const Kv4AttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (int64_t(blockIdx.x) < o_blocks) {
    const int64_t b = blockIdx.x / a.h_q, hq = blockIdx.x % a.h_q;
    const int32_t len = seq_len(a, b);
    const int32_t splits = (len + p.split_len - 1) / p.split_len;
    const int64_t part = (b * a.h_q + hq) * p.max_splits;
    const float2 g = join_ml(p.ml + 2 * part, splits, lane);
    if (tid == 0) {
      if (len > 0 && !(g.y > 0.f && g.y < INFINITY && isfinite(g.x)))
        status_or(static_cast<uint32_t*>(a.workspace), RMM_NONFINITE_BIT);
      if (a.lse) a.lse[b * a.h_q + hq] = len > 0 ? (g.x + log2f(g.y)) * 0.6931471805599453f : -INFINITY;
    }
    if (tid < a.d) {
      float o = 0.f;
      for (int s = 0; s < splits; ++s) o += p.po[(part + s) * a.d + tid] * exp2f(p.ml[2 * (part + s)] - g.x);
      o = len > 0 ? o / g.y : 0.f;
      const int64_t at = b * a.o_ss + hq * a.o_hs + tid;
      if (a.out == kBF16)
        static_cast<uint16_t*>(a.o)[at] = uint16_t(pack_bf16x2(o, 0.f));
      else
        static_cast<float*>(a.o)[at] = o;
    }
    return;
  }
  const int64_t i = blockIdx.x - o_blocks;
  const int64_t chunks = (a.cap + kJoinTokens - 1) / kJoinTokens;
  const int64_t item = i / chunks;
  const int64_t b = item / a.h_kv, h = item % a.h_kv;
  const int32_t len = seq_len(a, b);
  const int32_t t0 = int32_t(i % chunks) * kJoinTokens;
  if (t0 >= len) return;
  const int32_t gq = int32_t(a.h_q / a.h_kv);
  const int32_t splits = (len + p.split_len - 1) / p.split_len;
  const int64_t head0 = b * a.h_q + h * gq;
  for (int g = warp; g < gq; g += kJoinThreads / 32) {
    const float2 ml = join_ml(p.ml + 2 * (head0 + g) * p.max_splits, splits, lane);
    if (lane == 0) lse2[g] = ml.x + log2f(ml.y);
  }
  __syncthreads();
  const int32_t t1 = min(len, t0 + kJoinTokens);
  for (int32_t t = t0 + tid; t < t1; t += kJoinThreads) {
    float s = 0.f;
    for (int g = 0; g < gq; ++g) s += exp2f(p.scores[(head0 + g) * a.cap + t] - lse2[g]);
    const int64_t at = item * a.cap + t;
    a.w_out[at] = a.w_in ? a.w_in[at] + s : s;
  }
}

}  // namespace

cudaError_t launch_kv4_store(const Kv4StoreArgs& a, cudaStream_t st) {
  const int64_t total = a.T * a.h_kv * 2 * (a.d / 8);
  const dim3 grid(unsigned((total + 255) / 256));
  if (a.in == kBF16) return launch_pdl(kv4_store_kernel<uint16_t>, grid, dim3(256), 0, st, dim3(0, 0, 0), a);
  return launch_pdl(kv4_store_kernel<uint32_t>, grid, dim3(256), 0, st, dim3(0, 0, 0), a);
}

Kv4Ws kv4_ws(int64_t batch, int64_t h_q, int64_t h_kv, int64_t d, int64_t cap, bool weights) {
  Kv4Ws w;
  const int64_t want = batch * h_kv * cap / (148 * 4);
  w.split_len = std::min<int64_t>(std::max<int64_t>((want + 63) / 64 * 64, 128), 1024);
  w.max_splits = (cap + w.split_len - 1) / w.split_len;
  auto al = [](int64_t x) { return (x + 1023) / 1024 * 1024; };
  int64_t off = 1024;
  w.ml = size_t(off);
  off += al(batch * h_q * w.max_splits * 8);
  w.o = size_t(off);
  off += al(batch * h_q * w.max_splits * d * 4);
  w.scores = size_t(off);
  if (weights) off += al(batch * h_q * cap * 4);
  w.bytes = size_t(off);
  return w;
}

cudaError_t launch_kv4_attn(const Kv4AttnArgs& a, cudaStream_t st) {
  const Kv4Ws w = kv4_ws(a.batch, a.h_q, a.h_kv, a.d, a.cap, a.w_out != nullptr);
  char* base = static_cast<char*>(a.workspace);
  Kv4Dev p;
  p.a = a;
  p.ml = reinterpret_cast<float*>(base + w.ml);
  p.po = reinterpret_cast<float*>(base + w.o);
  p.scores = a.w_out ? reinterpret_cast<float*>(base + w.scores) : nullptr;
  p.split_len = int32_t(w.split_len);
  p.max_splits = int32_t(w.max_splits);
  cudaError_t e = launch_pdl(kv4_attn_split_kernel, dim3(unsigned(w.max_splits), unsigned(a.h_q), unsigned(a.batch)),
                             dim3(kSimpleThreads), 0, st, dim3(0, 0, 0), p);
  if (e != cudaSuccess) return e;
  const int64_t o_blocks = a.batch * a.h_q;
  const int64_t w_blocks = a.w_out ? a.batch * a.h_kv * ((a.cap + kJoinTokens - 1) / kJoinTokens) : 0;
  return launch_pdl(kv4_attn_join_kernel, dim3(unsigned(o_blocks + w_blocks)), dim3(kJoinThreads),
                    size_t(a.h_q / a.h_kv) * 4, st, dim3(0, 0, 0), p, o_blocks);
}

}  // namespace rmm
