// Attention of packed prompts (softmax(scale·Q·Kᵀ)·V per head, causal or not,
// grouped heads) and the weight each key received: the attention sites of
// "Escopo de Aplicação" on the gist.science summary of "Reduced Matrix
// Multiplication: Input-Adaptive Matrix-Product Reduction for LLM Inference"
// without P in memory.
#include <algorithm>

#include "rmm_device.cuh"
#include "rmm_internal.h"

namespace rmm {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct SeqSpan {
  int32_t q0, q1, k0, k1;
};

// Boundaries of sequence i, clamped so that no boundary list can point outside the tokens.
__device__ __forceinline__ SeqSpan seq_span(const AttnArgs& a, int64_t i) {
  SeqSpan s;
  auto clamp = [](int64_t x, int64_t lo, int64_t hi) { return int32_t(x < lo ? lo : (x > hi ? hi : x)); };
  s.q0 = a.cu_q ? clamp(a.cu_q[i], 0, a.T_q) : 0;
  s.q1 = a.cu_q ? clamp(a.cu_q[i + 1], s.q0, a.T_q) : int32_t(a.T_q);
  s.k0 = a.cu_k ? clamp(a.cu_k[i], 0, a.T_k) : 0;
  s.k1 = a.cu_k ? clamp(a.cu_k[i + 1], s.k0, a.T_k) : int32_t(a.T_k);
  return s;
}

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

constexpr int kMaxD = 128;

__device__ __forceinline__ float dot_row(const uint16_t* k, const float* q, int d) {
  float x = 0.f;
  for (int c = 0; c < d; c += 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(k + c);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x = fmaf(q[c + 2 * e], __uint_as_float(w[e] << 16), x);
      x = fmaf(q[c + 2 * e + 1], __uint_as_float(w[e] & 0xFFFF0000u), x);
    }
  }
  return x;
}

// A warp per (query token, head): lanes take 32 keys at a time for the scores, then 4 channels each for the sums.
__global__ void __launch_bounds__(128) attn_prompt_kernel(const AttnArgs a) {
  __shared__ float qs[4][kMaxD];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = int64_t(blockIdx.x) * 4 + warp;
  const int64_t hq = blockIdx.y, h = hq / (a.h_q / a.h_kv);
  if (t >= a.T_q) return;
  const int64_t i = a.cu_q ? find_seq(a.cu_q, a.n_seq, t) : 0;
  const SeqSpan s = seq_span(a, i);
  if (t < s.q0 || t >= s.q1) return;
  const int d = int(a.d);
  const uint16_t* q = static_cast<const uint16_t*>(a.q.ptr) + t * a.q.ts + hq * a.q.hs;
  for (int c = lane; c < d; c += 32) qs[warp][c] = bf16_to_f32(q[c]) * (a.scale * kLog2e);
  __syncwarp();
  int64_t end = s.k1;
  if (a.causal) end = min(end, int64_t(s.k0) + (t - s.q0) + (s.k1 - s.k0) - (s.q1 - s.q0) + 1);
  const uint16_t* K = static_cast<const uint16_t*>(a.k.ptr) + h * a.k.hs;
  const uint16_t* V = static_cast<const uint16_t*>(a.v.ptr) + h * a.v.hs;
  float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int64_t k0 = s.k0; k0 < end; k0 += 32) {
    const int64_t k = k0 + lane;
    const float x = k < end ? dot_row(K + k * a.k.ts, qs[warp], d) : -INFINITY;
    float mx = x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float m2 = fmaxf(m, mx), corr = exp2f(m - m2);
    const float p = exp2f(x - m2);
    m = m2;
    l = l * corr + p;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] *= corr;
    const int cnt = int(min(int64_t(32), end - k0));
    for (int j = 0; j < cnt; ++j) {
      const float pj = __shfl_sync(0xffffffffu, p, j);
      const uint16_t* v = V + (k0 + j) * a.v.ts;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (4 * lane + e < d) acc[e] = fmaf(pj, bf16_to_f32(v[4 * lane + e]), acc[e]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const bool any = end > s.k0;
  if (lane == 0) {
    if (any && !(l > 0.f && l < INFINITY)) status_or(a.status, RMM_NONFINITE_BIT);
    if (a.lse) a.lse[hq * a.T_q + t] = any ? (m + log2f(l)) * kLn2 : -INFINITY;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int c = 4 * lane + e;
    if (c >= d) continue;
    const float o = any ? acc[e] / l : 0.f;
    const int64_t at = t * a.o_ts + hq * a.o_hs + c;
    if (a.out == kBF16)
      static_cast<uint16_t*>(a.o)[at] = uint16_t(pack_bf16x2(o, 0.f));
    else
      static_cast<float*>(a.o)[at] = o;
  }
}

// A thread per key of one head; the queries go by in order.
__global__ void __launch_bounds__(128) attn_key_weights_kernel(const AttnArgs a) {
  __shared__ float qs[kMaxD];
  pdl_trigger();
  pdl_wait();
  const int64_t h = blockIdx.y;
  const int64_t i = blockIdx.z;
  const SeqSpan s = seq_span(a, i);
  const int d = int(a.d), g = int(a.h_q / a.h_kv);
  const int64_t kb = int64_t(s.k0) + int64_t(blockIdx.x) * 128;
  if (kb >= s.k1) return;
  const int64_t k = kb + threadIdx.x;
  const int64_t off = int64_t(s.k1 - s.k0) - (s.q1 - s.q0);
  const uint16_t* kr = static_cast<const uint16_t*>(a.k.ptr) + h * a.k.hs + min(k, int64_t(s.k1) - 1) * a.k.ts;
  float w = 0.f;
  for (int64_t t = s.q0; t < s.q1; ++t) {
    const int64_t end = a.causal ? min(int64_t(s.k1), int64_t(s.k0) + (t - s.q0) + off + 1) : int64_t(s.k1);
    if (end <= kb) continue;
    float part = 0.f;
    for (int e = 0; e < g; ++e) {
      const int64_t hq = h * g + e;
      __syncthreads();
      if (int(threadIdx.x) < d)
        qs[threadIdx.x] =
            bf16_to_f32((static_cast<const uint16_t*>(a.q.ptr) + t * a.q.ts + hq * a.q.hs)[threadIdx.x]) * a.scale;
      __syncthreads();
      if (k < end) part += expf(dot_row(kr, qs, d) - a.lse[hq * a.T_q + t]);
    }
    w += part;
  }
  if (k < s.k1) {
    if (!isfinite(w)) status_or(a.status, RMM_NONFINITE_BIT);
    const int64_t at = h * a.T_k + k;
    a.w_out[at] = a.w_in ? a.w_in[at] + w : w;
  }
}

}  // namespace

cudaError_t launch_attn_prompt(const AttnArgs& a, cudaStream_t st, const char**) {
  return launch_pdl(attn_prompt_kernel, dim3(unsigned((a.T_q + 3) / 4), unsigned(a.h_q)), dim3(128), 0, st,
                    dim3(0, 0, 0), a);
}

cudaError_t launch_attn_key_weights(const AttnArgs& a, cudaStream_t st, const char**) {
  return launch_pdl(attn_key_weights_kernel, dim3(unsigned((a.T_k + 127) / 128), unsigned(a.h_kv), unsigned(a.n_seq)),
                    dim3(128), 0, st, dim3(0, 0, 0), a);
}

}  // namespace rmm
