// Attention of packed prompts (softmax(scale·Q·Kᵀ)·V per head, causal or not,
// grouped heads) and the weight each key received: the attention sites of
// "Escopo de Aplicação" on the gist.science summary of "Reduced Matrix
// Multiplication: Input-Adaptive Matrix-Product Reduction for LLM Inference"
// without P in memory.
//
// A tile is 128 rows of (query, head) pairs, the g = h_q / h_kv heads of one
// key head side by side: 128 / g queries, head fastest (rows past (128/g)·g are
// idle). So the g heads read their keys and values once, and a causal tile
// spans few queries.
//
// Attention, per CTA two such tiles and one key head:
//   warps 0-3, 4-7  one row per thread: S from TMEM, running maximum and sum
//                   in log2 units, P as bf16 back to TMEM over S
//   warp 8          one lane issues tcgen05.mma: S_t = Q_t·Kᵀ (both operands
//                   in shared memory) and O_t += P_t·V (P in TMEM); while one
//                   tile's softmax runs, the other tile's products do
//   warp 9          TMA: Q once, then K and V tiles of 128 keys through one ring
// TMEM: S_0, S_1, O_0, O_1 of 128 columns each. O is rescaled in TMEM by the
// softmax warps themselves, and only when a row's maximum grew by more than
// 2^8 in the exponential's argument: P then stays below 256, which bf16 and
// the f32 sums hold as well as values below 1. The barrier that hands S_t(j)
// over tracks every product issued before it, P_t·V of tile j-1 among them,
// so O needs no barrier of its own.
// Every wait is bounded (rmm_set_wait_limit_ns) as in gemm_tc.cu.
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "rmm_device.cuh"
#include "rmm_internal.h"

namespace rmm {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kRows = 128;  // rows of a tile, keys of a key tile
constexpr int kThreads = 320;
constexpr float kRescale = 8.0f;  // log2 of the growth of P that is let through unscaled

struct TcArgs {
  AttnArgs a;
  int32_t g, nq_tile;  // heads per key head, queries per tile
  int32_t row_bytes;   // bytes of one tile's Q box: nq_tile·g·128
};

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

struct Work {
  SeqSpan s;
  int32_t tile;  // tile (of `span` tokens) within the sequence; -1: none left
};

// The sequence and tile of block `b` when sequence i has ceil(n_i / span)
// tiles (n_i its queries, or its keys), the warp taking 32 sequences at a
// time. Boundaries that are no ascending list can only make the sum of tiles
// larger than the grid, which leaves tiles out but reads nothing outside.
template <bool KEYS>
__device__ __forceinline__ Work find_work(const AttnArgs& a, int64_t b, int32_t span, int lane) {
  Work w;
  w.tile = -1;
  for (int64_t i0 = 0; i0 < a.n_seq; i0 += 32) {
    int32_t tiles = 0;
    SeqSpan s = {0, 0, 0, 0};
    if (i0 + lane < a.n_seq) {
      s = seq_span(a, i0 + lane);
      const int32_t n = KEYS ? s.k1 - s.k0 : s.q1 - s.q0;
      tiles = (n + span - 1) / span;
    }
    int32_t incl = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const uint32_t after = __ballot_sync(0xffffffffu, int64_t(incl) > b);
    if (after) {
      const int src = __ffs(after) - 1;
      w.s.q0 = __shfl_sync(0xffffffffu, s.q0, src);
      w.s.q1 = __shfl_sync(0xffffffffu, s.q1, src);
      w.s.k0 = __shfl_sync(0xffffffffu, s.k0, src);
      w.s.k1 = __shfl_sync(0xffffffffu, s.k1, src);
      const int32_t n = __shfl_sync(0xffffffffu, tiles, src);
      const int32_t before = __shfl_sync(0xffffffffu, incl, src) - n;
      const int32_t t = int32_t(b - before);
      w.tile = KEYS ? t : n - 1 - t;  // the longest rows (most queries) first
      return w;
    }
    b -= __shfl_sync(0xffffffffu, incl, 31);
  }
  return w;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void raise_abort(volatile int* abort_flag, uint32_t* status) {
  *abort_flag = 1;
  status_or(status, RMM_TIMEOUT_BIT);
}

// All lanes wait (each needs the acquire); the warp goes on together or not at all.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint64_t limit, const volatile int* abort) {
  const bool ok = mbar_wait_bounded(bar, parity, limit, abort);
  return __all_sync(0xffffffffu, ok);
}

template <int DP>
struct PromptCfg {
  static constexpr int BOXES = DP / 64;
  static constexpr uint32_t BOX = kRows * 128;       // 128 rows x 64 bf16
  static constexpr uint32_t TILE = BOXES * BOX;      // one Q, K or V tile
  static constexpr int STAGES = DP == 128 ? 5 : 8;   // K and V tiles in flight
  static constexpr size_t SMEM = 1024 + size_t(2 + STAGES) * TILE + 256;
  static_assert(SMEM <= 232448, "shared memory budget");
};

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
attn_prompt_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const TcArgs p) {
  using Cfg = PromptCfg<DP>;
  constexpr int STAGES = Cfg::STAGES;
  extern __shared__ uint8_t attn_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(attn_smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                   // two tiles
  uint8_t* sKV = sQ + 2 * Cfg::TILE;    // ring
  uint64_t* full = reinterpret_cast<uint64_t*>(sKV + STAGES * Cfg::TILE);
  uint64_t* empty = full + STAGES;
  uint64_t* q_full = empty + STAGES;    // [2]
  uint64_t* s_full = q_full + 2;        // [2] S_t ready (and O_t up to the previous key tile)
  uint64_t* p_full = s_full + 2;        // [2] P_t written, O_t rescaled
  uint64_t* o_full = p_full + 2;        // [2] O_t complete
  uint64_t* drain = o_full + 2;
  uint32_t* tmem_base_sh = reinterpret_cast<uint32_t*>(drain + 1);
  int* abort_sh = reinterpret_cast<int*>(tmem_base_sh + 1);
  int* never_sh = abort_sh + 1;  // stays 0: waits that must not be cut short

  const AttnArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 1);
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 4);
      mbar_init(&o_full[t], 1);
    }
    mbar_init(drain, 1);
    *abort_sh = 0;
    *never_sh = 0;
    fence_mbar_init();
  }
  if (warp == 9 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 8) {
    tmem_alloc<1>(tmem_base_sh, 512);
    tmem_relinquish<1>();
  }
  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_base_sh;
  pdl_wait();
  volatile int* abort_v = abort_sh;
  const volatile int* never_v = never_sh;
  const uint64_t limit = a.wait_limit_ns;

  const int32_t span = 2 * p.nq_tile;
  const Work w = find_work<false>(a, blockIdx.x / uint32_t(a.h_kv), span, lane);
  const int32_t h = int32_t(blockIdx.x % uint32_t(a.h_kv));
  if (w.tile >= 0) {
    const int32_t S_q = w.s.q1 - w.s.q0, S_k = w.s.k1 - w.s.k0;
    // keys visible to query q: [0, q + off + 1) of the sequence when causal
    const int32_t off = S_k - S_q;
    int32_t qt[2], nk[2];  // first query of each tile; its key tiles
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      qt[t] = w.tile * span + t * p.nq_tile;
      const int32_t last = min(S_q, qt[t] + p.nq_tile) - 1;
      const int32_t lim = last < qt[t] ? 0 : (a.causal ? min(S_k, last + off + 1) : S_k);
      nk[t] = lim > 0 ? (lim + kRows - 1) / kRows : 0;
    }
    const int32_t n = max(nk[0], nk[1]);

    if (warp == 9) {
      // ---------------------------------------------------------- TMA (one lane)
      if (lane == 0) {
        bool ok = true;
        uint32_t issued = 0, issued_par = 0;
        for (int t = 0; t < 2; ++t) {
          if (nk[t] == 0) continue;
          mbar_arrive_expect_tx(&q_full[t], uint32_t(Cfg::BOXES * p.row_bytes));
#pragma unroll
          for (int x = 0; x < Cfg::BOXES; ++x)
            tma_load_3d(sQ + t * Cfg::TILE + x * Cfg::BOX, &tmQ, &q_full[t], x * 64, h * p.g, w.s.q0 + qt[t]);
        }
        uint32_t stage = 0, phase = 0;
        for (int32_t i = 0; ok && i < 2 * n; ++i) {  // K_0, V_0, K_1, V_1, ...
          if (!mbar_wait_bounded(&empty[stage], phase ^ 1u, limit, abort_v)) {
            ok = false;
            break;
          }
          const CUtensorMap* m = (i & 1) ? &tmV : &tmK;
          mbar_arrive_expect_tx(&full[stage], Cfg::TILE);
#pragma unroll
          for (int x = 0; x < Cfg::BOXES; ++x)
            tma_load_3d(sKV + stage * Cfg::TILE + x * Cfg::BOX, m, &full[stage], x * 64, h,
                        w.s.k0 + (i >> 1) * kRows);
          issued |= 1u << stage;
          issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) raise_abort(abort_v, a.status);
        // no load may still be writing shared memory when the CTA exits
        for (int t = 0; t < 2; ++t)
          if (nk[t] > 0) mbar_wait_bounded(&q_full[t], 0, limit, never_v);
        for (int s = 0; s < STAGES; ++s)
          if (issued & (1u << s)) mbar_wait_bounded(&full[s], (issued_par >> s) & 1u, limit, never_v);
      }
      __syncwarp();
    } else if (warp == 8) {
      // ---------------------------------------------------------- MMA
      // The whole warp waits (it also zeroes the value rows past the
      // sequence's end, whose probabilities are 0 but whose memory may hold
      // NaN); lane 0 issues.
      const uint32_t dn = uint32_t((a.d + 15) / 16 * 16);
      const uint32_t id_s = umma_idesc_bf16_f32(kRows, kRows, false);
      const uint32_t id_o = umma_idesc_bf16_f32(kRows, dn, true);
      const int ksteps = int(dn / 16);
      bool ok = true;
      uint32_t p_par[2] = {0u, 0u};
      auto ring = [&](int32_t i, uint32_t& stage, uint32_t& par) {
        stage = uint32_t(i) % STAGES;
        par = (uint32_t(i) / STAGES) & 1u;
      };
      auto issue_s = [&](int t, uint32_t stage) {
        if (lane == 0) {
          const uint32_t q = smem_addr(sQ + t * Cfg::TILE), k = smem_addr(sKV + stage * Cfg::TILE);
          for (int kk = 0; kk < ksteps; ++kk) {
            const uint32_t o = uint32_t(kk >> 2) * Cfg::BOX + uint32_t(kk & 3) * 32;
            umma_bf16<1>(tmem + t * 128, umma_desc_k_sw128(q + o), umma_desc_k_sw128(k + o), id_s, kk != 0);
          }
          umma_commit<1>(smem_addr(&s_full[t]));
        }
      };
      auto issue_o = [&](int t, uint32_t stage, int32_t j) {
        if (lane == 0) {
          const uint32_t v = smem_addr(sKV + stage * Cfg::TILE);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_bf16_ts(tmem + 256 + t * 128, tmem + t * 128 + kk * 8, umma_desc_mn_sw128(v + kk * 2048, Cfg::BOX),
                         id_o, j != 0 || kk != 0);
          if (j == nk[t] - 1) umma_commit<1>(smem_addr(&o_full[t]));
        }
      };
      uint32_t st, par;
      if (n > 0) {
        ring(0, st, par);
        ok = warp_wait(&full[st], par, limit, abort_v);
        for (int t = 0; ok && t < 2; ++t) {
          if (nk[t] == 0) continue;
          ok = warp_wait(&q_full[t], 0, limit, abort_v);
          if (ok) {
            tc_fence_after();
            issue_s(t, st);
          }
        }
        if (ok && lane == 0) umma_commit<1>(smem_addr(&empty[st]));
      }
      for (int32_t j = 0; ok && j < n; ++j) {
        uint32_t vst, vpar, kst = 0, kpar = 0;
        ring(2 * j + 1, vst, vpar);
        ok = warp_wait(&full[vst], vpar, limit, abort_v);
        if (!ok) break;
        const int32_t past = (j + 1) * kRows - S_k;  // rows of this tile past the sequence
        if (past > 0) {
          for (int32_t r = kRows - past; r < kRows; ++r)
            for (int c = lane; c < Cfg::BOXES * 8; c += 32)
              *reinterpret_cast<uint4*>(sKV + vst * Cfg::TILE + (c >> 3) * Cfg::BOX + r * 128 + (c & 7) * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          __syncwarp();
        }
        const bool more = j + 1 < n;
        for (int t = 0; ok && t < 2; ++t) {
          if (j < nk[t]) {
            ok = warp_wait(&p_full[t], p_par[t], limit, abort_v);
            if (!ok) break;
            p_par[t] ^= 1u;
            tc_fence_after();
            issue_o(t, vst, j);
          }
          if (t == 0 && more) {
            ring(2 * j + 2, kst, kpar);
            ok = warp_wait(&full[kst], kpar, limit, abort_v);
            if (!ok) break;
            tc_fence_after();
          }
          if (t == 1 && lane == 0) umma_commit<1>(smem_addr(&empty[vst]));
          if (j + 1 < nk[t]) issue_s(t, kst);
          if (t == 1 && more && lane == 0) umma_commit<1>(smem_addr(&empty[kst]));
        }
      }
      if (lane == 0) {
        if (!ok) raise_abort(abort_v, a.status);
        umma_commit<1>(smem_addr(drain));  // every product done before tensor memory is freed
        mbar_wait_bounded(drain, 0, limit, never_v);
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------- softmax, one row per thread
      const int t = warp >> 2;
      const int r = (warp & 3) * 32 + lane;
      const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
      const uint32_t tS = tmem + lane_base + t * 128, tO = tS + 256;
      const int32_t q = qt[t] + r / p.g;  // query within the sequence
      const bool row_ok = r < p.nq_tile * p.g && q < S_q;
      const int32_t lim = row_ok ? (a.causal ? min(S_k, q + off + 1) : S_k) : S_k;  // idle rows: anything
      const float c = a.scale * kLog2e;
      float m = -INFINITY, nm = 0.f, l = 0.f;  // maximum of s; -(maximum·c) (0 while there is none); sum
      bool ok = true;
      for (int32_t j = 0; j < nk[t]; ++j) {
        if (!warp_wait(&s_full[t], uint32_t(j) & 1u, limit, abort_v)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int x = 0; x < 4; ++x) tmem_ld_32x32b_x32(tS + 32 * x, s[x]);
        tmem_ld_wait();
        const int32_t left = lim - j * kRows;  // visible keys of this tile
        if (__any_sync(0xffffffffu, left < kRows)) {
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (32 * x + e >= left) s[x][e] = 0xff800000u;
        }
        float mx[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          mx[x] = __uint_as_float(s[x][0]);
#pragma unroll
          for (int e = 1; e < 32; ++e) mx[x] = fmaxf(mx[x], __uint_as_float(s[x][e]));
        }
        const float m2 = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(fmaxf(mx[2], mx[3]), m));
        // (m2 - m)·c, a first maximum counting as growth
        if (__any_sync(0xffffffffu, m2 > m && !(fmaf(m2, c, nm) <= kRescale && m > -INFINITY))) {
          const float nm2 = m2 > -INFINITY ? -m2 * c : 0.f;
          if (j > 0) {
            const float f = m > -INFINITY ? ex2(nm2 - nm) : 1.f;
            l *= f;
#pragma unroll
            for (int x = 0; x < DP / 32; ++x) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(tO + 32 * x, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st_32x32b_x32(tO + 32 * x, o);
            }
          }
          m = m2;
          nm = nm2;
        }
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float p0 = ex2(fmaf(__uint_as_float(s[x][2 * e]), c, nm));
            const float p1 = ex2(fmaf(__uint_as_float(s[x][2 * e + 1]), c, nm));
            sum[e & 3] += p0 + p1;
            pk[e] = pack_bf16x2(p0, p1);
          }
          tmem_st_32x32b_x16(tS + 16 * x, pk);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t]);
      }
      if (ok && nk[t] > 0) ok = warp_wait(&o_full[t], 0, limit, abort_v);
      if (!ok) {
        if (lane == 0) raise_abort(abort_v, a.status);
      } else {
        tc_fence_after();
        const int64_t tok = int64_t(w.s.q0) + q, hq = int64_t(h) * p.g + r % p.g;
        const bool any = lim > 0 && nk[t] > 0;
        if (row_ok) {
          if (any && !(l > 0.f && l < INFINITY)) status_or(a.status, RMM_NONFINITE_BIT);
          if (a.lse) a.lse[hq * a.T_q + tok] = any ? (log2f(l) - nm) * kLn2 : -INFINITY;
        }
        const float inv = any ? 1.0f / l : 0.f;
#pragma unroll
        for (int x = 0; x < DP / 32; ++x) {
          uint32_t o[32];
          __syncwarp();
          if (nk[t] > 0) {
            tmem_ld_32x32b_x32(tO + 32 * x, o);
            tmem_ld_wait();
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = any ? __float_as_uint(__uint_as_float(o[e]) * inv) : 0u;
          if (!row_ok) continue;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int col = 32 * x + 8 * v;
            if (col >= a.d) break;
            const uint32_t* e = o + 8 * v;
            const int64_t at = tok * a.o_ts + hq * a.o_hs + col;
            if (a.out == kBF16) {
              auto two = [&](int i) { return pack_bf16x2(__uint_as_float(e[i]), __uint_as_float(e[i + 1])); };
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + at) = make_uint4(two(0), two(2), two(4), two(6));
            } else {
              uint4* dst = reinterpret_cast<uint4*>(static_cast<float*>(a.o) + at);
              dst[0] = make_uint4(e[0], e[1], e[2], e[3]);
              dst[1] = make_uint4(e[4], e[5], e[6], e[7]);
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc<1>(tmem, 512);
}

// A thread per key of one head; the queries go by in order.
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

// ------------------------------------------------------------------ host side
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// [tokens][heads][d] read in boxes of box_t tokens x box_h heads x 64 channels
// (128-byte rows, 128-byte swizzle), zeros past d and past the last token.
bool encode_tokens(CUtensorMap* m, const TokView& v, int64_t tokens, int64_t heads, int64_t d, uint32_t box_t,
                   uint32_t box_h) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  // the stride of a dimension of extent 1 is never used, but must be a valid one
  const uint64_t hs = heads > 1 ? uint64_t(v.hs) * 2 : 256, ts = tokens > 1 ? uint64_t(v.ts) * 2 : 256;
  cuuint64_t dims[3] = {uint64_t(d), uint64_t(heads), uint64_t(tokens)};
  cuuint64_t strides[2] = {hs, ts};
  cuuint32_t box[3] = {64, box_h, box_t};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(v.ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t device_ok(const char** why) {
  int dev = 0, major = 0, minor = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (e != cudaSuccess) return e;
  if (major == 10 && minor == 0) return cudaSuccess;
  *why = "the attention kernels are built for sm_100a (B200) only";
  return cudaErrorNoKernelImageForDevice;
}

template <int DP>
cudaError_t launch_prompt(const TcArgs& p, cudaStream_t st, const char** why) {
  using Cfg = PromptCfg<DP>;
  const AttnArgs& a = p.a;
  CUtensorMap tmQ, tmK, tmV;
  bool ok = encode_tokens(&tmQ, a.q, a.T_q, a.h_q, a.d, uint32_t(p.nq_tile), uint32_t(p.g));
  if (a.T_k > 0) {
    ok = ok && encode_tokens(&tmK, a.k, a.T_k, a.h_kv, a.d, kRows, 1) &&
         encode_tokens(&tmV, a.v, a.T_k, a.h_kv, a.d, kRows, 1);
  } else {
    tmK = tmV = tmQ;  // no key is ever loaded
  }
  if (!ok) {
    *why = "cuTensorMapEncodeTiled failed for Q, K or V";
    return cudaErrorInvalidValue;
  }
  cudaError_t e = cudaFuncSetAttribute(attn_prompt_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       int(Cfg::SMEM));
  if (e != cudaSuccess) return e;
  const int64_t span = 2 * p.nq_tile;
  const int64_t tiles = a.n_seq == 1 ? (a.T_q + span - 1) / span : a.T_q / span + a.n_seq;
  return launch_pdl(attn_prompt_kernel<DP>, dim3(unsigned(tiles * a.h_kv)), dim3(kThreads), Cfg::SMEM, st,
                    dim3(0, 0, 0), tmQ, tmK, tmV, p);
}

TcArgs tc_args(const AttnArgs& a) {
  TcArgs p;
  p.a = a;
  p.g = int32_t(a.h_q / a.h_kv);
  p.nq_tile = kRows / p.g;
  p.row_bytes = p.nq_tile * p.g * 128;
  return p;
}

}  // namespace

cudaError_t launch_attn_prompt(const AttnArgs& a, cudaStream_t st, const char** why) {
  cudaError_t e = device_ok(why);
  if (e != cudaSuccess) return e;
  const TcArgs p = tc_args(a);
  return a.d <= 64 ? launch_prompt<64>(p, st, why) : launch_prompt<128>(p, st, why);
}

cudaError_t launch_attn_key_weights(const AttnArgs& a, cudaStream_t st, const char**) {
  return launch_pdl(attn_key_weights_kernel, dim3(unsigned((a.T_k + 127) / 128), unsigned(a.h_kv), unsigned(a.n_seq)),
                    dim3(128), 0, st, dim3(0, 0, 0), a);
}

}  // namespace rmm
