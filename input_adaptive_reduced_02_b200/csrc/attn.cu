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
// Attention, per CTA two such tiles t and one key head:
//   warps 0-3, 4-7  one row per thread: S from TMEM, running maximum and sum
//                   in log2 units, P as bf16 back to TMEM over S
//   warps 8, 9      tile 0 and 1: tcgen05.mma, S_t = Q_t·Kᵀ (both operands in
//                   shared memory) and O_t += P_t·V (P in TMEM); while one
//                   tile's softmax runs, the other tile's products do
//   warp 10         TMA: Q once, then K and V tiles of 128 keys through one
//                   ring; zeroes the value rows past the sequence's end
// TMEM: S_0, S_1, O_0, O_1 of 128 columns each. O is rescaled in TMEM by the
// softmax warps themselves, and only when a row's maximum grew by more than
// 2^8 in the exponential's argument: P then stays below 256, which bf16 and
// the f32 sums hold as well as values below 1. The barrier that hands S_t(j)
// over tracks every product issued before it, P_t·V of tile j-1 among them, so O
// needs no barrier of its own.
// A tile's softmax and its products take turns, and that chain bounds the
// kernel: per 128 keys about 2000 cycles of softmax (16 exponentials a cycle
// per SM: 1024 for 128 x 128) and 1400 of P·V (512), S (800: both operands
// from shared memory come at 82 of 128 bytes a cycle) and handovers.
// Every wait is bounded (rmm_set_wait_limit_ns) as in gemm_tc.cu.
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "rmm_device.cuh"
#include "rmm_internal.h"

namespace rmm {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kRows = 128;  // rows of a tile, keys of a key tile
constexpr int kThreads = 384;
// Registers per thread: 168 at launch (64512 for 384 threads); the eight softmax
// warps, with a row of S and their row's state, take what the other four give back.
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(8 * kSoftmaxRegs + 4 * kOtherRegs <= 12 * 168, "registers of the block");
constexpr float kRescale = 8.0f;  // log2 of the growth of P that is let through unscaled

struct TcArgs {
  AttnArgs a;
  int32_t g, nq_tile;  // heads per key head, queries per tile
  int32_t row_bytes;   // bytes of one tile's Q box: nq_tile·g·128
  uint32_t split;      // key weights: CTAs of a cluster that share the queries
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

template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
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

// D = A·Bᵀ over d: A's rows 128 by 64-channel boxes of 128 rows, B's of BROWS
// rows, both as TMA wrote them. ksteps: 16 channels each, up to DP / 16.
template <int DP, int BROWS>
__device__ __forceinline__ void issue_product(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, int ksteps) {
#pragma unroll
  for (int kk = 0; kk < DP / 16; ++kk)
    if (kk < ksteps)
      umma_bf16_warp(d_tmem, a_lo + (kk >> 2) * (kRows * 128 >> 4) + (kk & 3) * 2,
                     b_lo + (kk >> 2) * (BROWS * 128 >> 4) + (kk & 3) * 2, idesc, kk != 0);
}

template <int DP>
struct PromptCfg {
  static constexpr int BOXES = DP / 64;
  static constexpr uint32_t BOX = kRows * 128;       // 128 rows x 64 bf16
  static constexpr uint32_t TILE = BOXES * BOX;      // one Q, K or V tile
  static constexpr int STAGES = DP == 128 ? 4 : 8;   // K and V tiles in flight
  static constexpr uint32_t STAGING = 8 * 32 * 128;  // 128 bytes of each output row
  static constexpr size_t SMEM = 1024 + size_t(2 + STAGES) * TILE + STAGING + 256;
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
  uint8_t* staging = sKV + STAGES * Cfg::TILE;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + Cfg::STAGING);
  uint64_t* empty = full + STAGES;
  uint64_t* q_full = empty + STAGES;    // [2]
  uint64_t* s_full = q_full + 2;        // [2] S_t ready (and O_t up to the previous key tile)
  uint64_t* p_full = s_full + 2;        // [2] P_t written, O_t rescaled
  uint64_t* o_full = p_full + 2;        // [2] O_t complete
  uint64_t* v_zeroed = o_full + 2;
  uint64_t* drain = v_zeroed + 1;       // [2]
  uint32_t* tmem_base_sh = reinterpret_cast<uint32_t*>(drain + 2);
  int* abort_sh = reinterpret_cast<int*>(tmem_base_sh + 1);
  int* never_sh = abort_sh + 1;  // stays 0: waits that must not be cut short
  static_assert((2 * STAGES + 11) * 8 + 3 * 4 <= 256, "barrier area");

  const AttnArgs& a = p.a;
  const int warp = warp_index(), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 1);
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 4);
      mbar_init(&o_full[t], 1);
      mbar_init(&drain[t], 1);
    }
    mbar_init(v_zeroed, 1);
    *abort_sh = 0;
    *never_sh = 0;
    fence_mbar_init();
  }
  if (warp == 10 && lane == 0) {
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

    if (warp >= 8) {
    fewer_registers<kOtherRegs>();
    if (warp == 10) {
      // ---------------------------------------------------------- TMA (one lane)
      bool ok = true;
      uint32_t issued = 0, issued_par = 0;
      if (lane == 0) {
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
      }
      // Value rows past the sequence's end: their probabilities are 0, but their memory may hold NaN.
      ok = __shfl_sync(0xffffffffu, int(ok), 0);
      if (ok && n > 0 && n * kRows > S_k) {
        const uint32_t st = uint32_t(2 * n - 1) % STAGES, par = (uint32_t(2 * n - 1) / STAGES) & 1u;
        if (warp_wait(&full[st], par, limit, abort_v)) {
          for (int32_t r = S_k - (n - 1) * kRows; r < kRows; ++r)
            for (int c = lane; c < Cfg::BOXES * 8; c += 32)
              *reinterpret_cast<uint4*>(sKV + st * Cfg::TILE + (c >> 3) * Cfg::BOX + r * 128 + (c & 7) * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(v_zeroed);
        } else if (lane == 0) {
          raise_abort(abort_v, a.status);
        }
      }
      if (lane == 0) {
        // no load may still be writing shared memory when the CTA exits
        for (int t = 0; t < 2; ++t)
          if (nk[t] > 0) mbar_wait_bounded(&q_full[t], 0, limit, never_v);
        for (int s = 0; s < STAGES; ++s)
          if (issued & (1u << s)) mbar_wait_bounded(&full[s], (issued_par >> s) & 1u, limit, never_v);
      }
      __syncwarp();
    } else if (warp < 10) {
      // ---------------------------------------------------------- MMA of tile t
      const int t = warp - 8;
      const int32_t nt = t == 0 ? nk[0] : nk[1];
      const uint32_t dn = uint32_t((a.d + 15) / 16 * 16);
      const uint32_t id_s = umma_idesc_bf16_f32(kRows, kRows, false);
      const uint32_t id_o = umma_idesc_bf16_f32(kRows, dn, true);
      const int ksteps = int(dn / 16);
      const uint32_t desc_q = umma_desc_lo(smem_addr(sQ)) + t * (Cfg::TILE >> 4);
      const uint32_t desc_k = umma_desc_lo(smem_addr(sKV));
      const uint32_t desc_v = umma_desc_lo(smem_addr(sKV), Cfg::BOX);  // channels contiguous, 64 to a box
      const uint32_t tS = tmem + t * 128, tO = tS + 256;
      bool ok = true;
      uint32_t ring = 0, phase = 0;  // of the next K or V tile
      auto next = [&] {
        if (++ring == STAGES) {
          ring = 0;
          phase ^= 1u;
        }
      };
      auto issue_s = [&](uint32_t stage) {
        issue_product<DP, kRows>(tS, desc_q, desc_k + stage * (Cfg::TILE >> 4), id_s, ksteps);
        umma_commit_warp(&s_full[t]);
      };
      if (n > 0) {
        ok = (nt == 0 || warp_wait(&q_full[t], 0, limit, abort_v)) && warp_wait(&full[0], 0, limit, abort_v);
        if (ok) {
          tc_fence_after();
          if (nt > 0) issue_s(0);
          umma_commit_warp(&empty[0]);
          next();
        }
      }
      for (int32_t j = 0; ok && j < n; ++j) {
        // what the products need besides P, which comes last
        const uint32_t vst = ring;
        ok = warp_wait(&full[ring], phase, limit, abort_v);
        if (ok && j == n - 1 && n * kRows > S_k) ok = warp_wait(v_zeroed, 0, limit, abort_v);
        next();
        const uint32_t kst = ring;
        const bool more = j + 1 < n;
        if (ok && more) ok = warp_wait(&full[ring], phase, limit, abort_v);
        if (ok && j < nt) ok = warp_wait(&p_full[t], uint32_t(j) & 1u, limit, abort_v);
        if (!ok) break;
        if (j < nt) {
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_bf16_ts_warp(tO, tS + kk * 8, desc_v + vst * (Cfg::TILE >> 4) + kk * (2048 >> 4), id_o,
                              kk != 0 ? 1u : uint32_t(j));
          if (j + 1 < nt)
            issue_s(kst);
          else
            umma_commit_warp(&o_full[t]);
        }
        umma_commit_warp(&empty[vst]);
        if (more) {
          umma_commit_warp(&empty[kst]);
          next();
        }
      }
      if (!ok && lane == 0) raise_abort(abort_v, a.status);
      umma_commit_warp(&drain[t]);  // every product done before tensor memory is freed
      mbar_wait_bounded(&drain[t], 0, limit, never_v);
      __syncwarp();
    }
    } else {
      more_registers<kSoftmaxRegs>();
      // ---------------------------------------------------------- softmax, one row per thread
      const int t = warp >> 2;
      const int r = (warp & 3) * 32 + lane;
      const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
      const uint32_t tS = tmem + lane_base + t * 128, tO = tS + 256;
      const int32_t q = qt[t] + r / p.g;  // query within the sequence
      const bool row_ok = r < p.nq_tile * p.g && q < S_q;
      const int32_t lim = row_ok ? (a.causal ? min(S_k, q + off + 1) : S_k) : S_k;  // idle rows: anything
      const float c = a.scale * kLog2e;
      // Maximum of s; -(maximum·c) (0 while there is none); sum. An idle row holds whatever shared memory
      // or the next sequence's queries do: above every score, it never votes for a rescaling, which
      // would round the live rows' P under another maximum.
      float m = row_ok ? -INFINITY : INFINITY, nm = 0.f, l = 0.f;
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
        tmem_ld_wait(s[0]);
#pragma unroll
        for (int x = 1; x < 4; ++x) tmem_ld_waited(s[x]);
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
          mx[x] = fmaxf(__uint_as_float(s[x][0]), __uint_as_float(s[x][1]));
#pragma unroll
          for (int e = 2; e < 32; e += 2) mx[x] = max3(mx[x], __uint_as_float(s[x][e]), __uint_as_float(s[x][e + 1]));
        }
        const float m2 = fmaxf(max3(mx[0], mx[1], mx[2]), fmaxf(mx[3], m));
        // (m2 - m)·c, a first maximum counting as growth
        if (__any_sync(0xffffffffu, m2 > m && !(fmaf(m2, c, nm) <= kRescale && m > -INFINITY))) {
          const float nm2 = m2 > -INFINITY ? -m2 * c : 0.f;
          if (j > 0) {
            const float f = m > -INFINITY ? ex2(nm2 - nm) : 1.f;
            l *= f;
#pragma unroll
            for (int x = 0; x < DP / 16; ++x) {  // few columns at a time: S is in registers too
              uint32_t o[16];
              tmem_ld_32x32b_x16(tO + 16 * x, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st_32x32b_x16(tO + 16 * x, o);
            }
          }
          m = m2;
          nm = nm2;
        }
        const float2 c2 = make_float2(c, c), nm2 = make_float2(nm, nm);
        float2 sum[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) sum[x] = make_float2(0.f, 0.f);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 y = fma2(make_float2(__uint_as_float(s[x][2 * e]), __uint_as_float(s[x][2 * e + 1])), c2, nm2);
            const float2 pe = make_float2(ex2(y.x), ex2(y.y));
            sum[e & 3] = add2(sum[e & 3], pe);
            pk[e] = pack_bf16x2(pe.x, pe.y);
          }
          tmem_st_32x32b_x16(tS + 16 * x, pk);
        }
        const float2 sums = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
        l += sums.x + sums.y;
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
        // Rows leave through shared memory, so that a store instruction covers whole
        // 128-byte pieces of four of them (a thread's own row lies 16 bytes to each).
        uint8_t* mine = staging + warp * (32 * 128);
        const int64_t row_at = row_ok ? tok * a.o_ts + hq * a.o_hs : -1;
        auto leave = [&](int col0, int per) {  // per: channels of 16 bytes
          __syncwarp();
          const int col = col0 + (lane & 7) * per;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int row = 4 * i + (lane >> 3);
            const int64_t at = __shfl_sync(0xffffffffu, row_at, row) + col;
            const uint4 v = *reinterpret_cast<const uint4*>(mine + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
            if (at < col || col >= a.d) continue;
            if (a.out == kBF16)
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + at) = v;
            else
              *reinterpret_cast<uint4*>(static_cast<float*>(a.o) + at) = v;
          }
          __syncwarp();
        };
#pragma unroll
        for (int x = 0; x < DP / 32; ++x) {
          uint32_t o[32];
          if (nk[t] > 0) {
            tmem_ld_32x32b_x32(tO + 32 * x, o);
            tmem_ld_wait(o);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = any ? __float_as_uint(__uint_as_float(o[e]) * inv) : 0u;
          if (a.out == kBF16) {
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              auto two = [&](int i) { return pack_bf16x2(__uint_as_float(o[8 * v + i]), __uint_as_float(o[8 * v + i + 1])); };
              *reinterpret_cast<uint4*>(mine + lane * 128 + (((4 * (x & 1) + v) ^ (lane & 7)) << 4)) =
                  make_uint4(two(0), two(2), two(4), two(6));
            }
            if (x & 1) leave(32 * (x - 1), 8);
          } else {
#pragma unroll
            for (int v = 0; v < 8; ++v)
              *reinterpret_cast<uint4*>(mine + lane * 128 + ((v ^ (lane & 7)) << 4)) =
                  make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
            leave(32 * x, 4);
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

// ---------------------------------------------------------------- key weights
// Per CTA two tiles of 128 keys of one head: S_tᵀ = K_t·Qᵀ against tiles of 128
// (query, head) pairs, so that a thread owns a key and sums its row of S_tᵀ
// without leaving its registers:
//   warps 8t .. 8t+7  one key of tile t and half of the columns per thread: sum
//                     of 2^(s·c - lse·log2 e) over the tile's pairs, added to the
//                     thread's total with compensation
//   warp 16           issues tcgen05.mma; S_t is double buffered, so a tile's
//                     products run while the sums of the one before do
//   warp 17           TMA: both K tiles once, then Q tiles through a ring
//   warp 18           -lse·log2 e of a Q tile's pairs, through a ring of its own
// A lone warp of a scheduler issues one of these instructions every three
// cycles or so: with four (two per tile, on half of the columns) the sums of one
// prompt of 8192 tokens take 363 us, with two per scheduler 394 us.
// The CTAs of a cluster share the queries of the same keys, tile i going to
// CTA i mod C, and add their sums through distributed shared memory in rank
// order: no atomics, no workspace, one result whatever the schedule.
constexpr int kWtMma = 16, kWtTma = 17, kWtLse = 18;  // warps
constexpr int kWtThreads = 32 * (kWtLse + 1);
constexpr int kLseRing = 4;

template <int DP>
struct WeightCfg {
  static constexpr int BOXES = DP / 64;
  static constexpr uint32_t BOX = kRows * 128;
  static constexpr uint32_t TILE = BOXES * BOX;
  static constexpr int STAGES = 4;
  static constexpr uint32_t LSE = kLseRing * kRows * 4;
  static constexpr uint32_t SUMS = 4 * kRows * 4;  // [column half][tile][key]
  static constexpr size_t SMEM = 1024 + size_t(2 + STAGES) * TILE + LSE + SUMS + 256;
  static_assert(SMEM <= 232448, "shared memory budget");
};

__device__ __forceinline__ float ld_cluster_f32(uint32_t cluster_addr) {
  float x;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(cluster_addr) : "memory");
  return x;
}

template <int DP>
__global__ void __launch_bounds__(kWtThreads, 1)
attn_key_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const TcArgs p) {
  using Cfg = WeightCfg<DP>;
  constexpr int STAGES = Cfg::STAGES;
  extern __shared__ uint8_t attn_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(attn_smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem;                 // two tiles
  uint8_t* sQ = sK + 2 * Cfg::TILE;   // ring
  float* lse_sh = reinterpret_cast<float*>(sQ + STAGES * Cfg::TILE);
  float* sum_sh = lse_sh + kLseRing * kRows;
  uint64_t* full = reinterpret_cast<uint64_t*>(sum_sh + 4 * kRows);
  uint64_t* empty = full + STAGES;
  uint64_t* l_full = empty + STAGES;
  uint64_t* l_empty = l_full + kLseRing;
  uint64_t* k_full = l_empty + kLseRing;  // [2]
  uint64_t* s_full = k_full + 2;          // [2][2] tile, buffer
  uint64_t* s_empty = s_full + 4;         // [2][2]
  uint64_t* drain = s_empty + 4;
  uint32_t* tmem_base_sh = reinterpret_cast<uint32_t*>(drain + 1);
  int* abort_sh = reinterpret_cast<int*>(tmem_base_sh + 1);
  int* never_sh = abort_sh + 1;
  static_assert((2 * STAGES + 2 * kLseRing + 11) * 8 + 12 <= 256, "barrier area");

  const AttnArgs& a = p.a;
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const uint32_t rank = blockIdx.x % p.split;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kLseRing; ++s) {
      mbar_init(&l_full[s], 1);
      mbar_init(&l_empty[s], 16);
    }
    for (int t = 0; t < 2; ++t) mbar_init(&k_full[t], 1);
    for (int t = 0; t < 4; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&s_empty[t], 8);
    }
    mbar_init(drain, 1);
    *abort_sh = 0;
    *never_sh = 0;
    fence_mbar_init();
  }
  if (warp == kWtTma && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
  }
  if (warp == kWtMma) {
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

  const uint32_t unit = blockIdx.x / p.split;
  const Work w = find_work<true>(a, unit / uint32_t(a.h_kv), 2 * kRows, lane);
  const int32_t h = int32_t(unit % uint32_t(a.h_kv));
  float total = 0.f;
  if (w.tile >= 0) {
    const int32_t S_q = w.s.q1 - w.s.q0, S_k = w.s.k1 - w.s.k0;
    const int32_t off = S_k - S_q;
    const int32_t n_qt = (S_q + p.nq_tile - 1) / p.nq_tile;
    // key tile t: its first query tile of this CTA (n_qt on: none), and of the CTA
    int32_t i0[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int32_t k = w.tile * 2 * kRows + t * kRows;
      int32_t first = n_qt;
      if (k < S_k) first = a.causal ? min(max(k - off, 0) / p.nq_tile, n_qt) : 0;
      i0[t] = first + int32_t((rank + p.split - uint32_t(first) % p.split) % p.split);  // next one of this rank
    }
    const int32_t begin = min(i0[0], i0[1]), step = int32_t(p.split);

    if (warp == kWtTma) {
      if (lane == 0 && begin < n_qt) {
        bool ok = true;
        uint32_t issued = 0, issued_par = 0;
        for (int t = 0; t < 2; ++t) {
          if (i0[t] >= n_qt) continue;
          mbar_arrive_expect_tx(&k_full[t], Cfg::TILE);
#pragma unroll
          for (int x = 0; x < Cfg::BOXES; ++x)
            tma_load_3d(sK + t * Cfg::TILE + x * Cfg::BOX, &tmK, &k_full[t], x * 64, h,
                        w.s.k0 + w.tile * 2 * kRows + t * kRows);
        }
        uint32_t stage = 0, phase = 0;
        for (int32_t i = begin; i < n_qt; i += step) {
          if (!mbar_wait_bounded(&empty[stage], phase ^ 1u, limit, abort_v)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[stage], uint32_t(Cfg::BOXES * p.row_bytes));
#pragma unroll
          for (int x = 0; x < Cfg::BOXES; ++x)
            tma_load_3d(sQ + stage * Cfg::TILE + x * Cfg::BOX, &tmQ, &full[stage], x * 64, h * p.g,
                        w.s.q0 + i * p.nq_tile);
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
          if (i0[t] < n_qt) mbar_wait_bounded(&k_full[t], 0, limit, never_v);
        for (int s = 0; s < STAGES; ++s)
          if (issued & (1u << s)) mbar_wait_bounded(&full[s], (issued_par >> s) & 1u, limit, never_v);
      }
      __syncwarp();
    } else if (warp == kWtMma) {
      const uint32_t id_s = umma_idesc_bf16_f32(kRows, kRows, false);
      const int ksteps = int((a.d + 15) / 16);
      const uint32_t desc_k = umma_desc_lo(smem_addr(sK)), desc_q = umma_desc_lo(smem_addr(sQ));
      bool ok = true;
      uint32_t stage = 0, phase = 0, par[2] = {0u, 0u}, seen[2] = {0u, 0u};
      for (int32_t i = begin; ok && i < n_qt; i += step) {
        ok = warp_wait(&full[stage], phase, limit, abort_v);
        for (int t = 0; ok && t < 2; ++t) {
          if (i < i0[t]) continue;
          if (!seen[t]) {
            ok = warp_wait(&k_full[t], 0, limit, abort_v);
            if (!ok) break;
          }
          const uint32_t buf = seen[t]++ & 1u;
          // a buffer's first use needs no wait
          if (seen[t] > 2) {
            ok = warp_wait(&s_empty[t * 2 + buf], (par[t] >> buf) & 1u, limit, abort_v);
            if (!ok) break;
            par[t] ^= 1u << buf;
          }
          tc_fence_after();
          issue_product<DP, kRows>(tmem + (t * 2 + buf) * 128, desc_k + t * (Cfg::TILE >> 4),
                                   desc_q + stage * (Cfg::TILE >> 4), id_s, ksteps);
          umma_commit_warp(&s_full[t * 2 + buf]);
        }
        if (!ok) break;
        umma_commit_warp(&empty[stage]);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok && lane == 0) raise_abort(abort_v, a.status);
      umma_commit_warp(drain);
      mbar_wait_bounded(drain, 0, limit, never_v);
      __syncwarp();
    } else if (warp == kWtLse) {
      // a tile's values are read before the one before it is handed over
      constexpr int N = 4;
      const float* src[N];
      float v[N];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int32_t c = 32 * e + lane;
        src[e] = a.lse + int64_t(h * p.g + c % p.g) * a.T_q + w.s.q0 + c / p.g;
      }
      auto read = [&](int32_t i) {
        const int32_t q0 = i * p.nq_tile, live = min(p.nq_tile, S_q - q0) * p.g;
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = 32 * e + lane < live ? src[e][q0] : 0.f;
      };
      read(begin);
      bool ok = true;
      uint32_t r = 0, phase = 0;
      for (int32_t i = begin; i < n_qt; i += step) {
        float nl[N];
#pragma unroll
        for (int e = 0; e < N; ++e) nl[e] = -v[e] * kLog2e;
        read(i + step);
        if (!warp_wait(&l_empty[r], phase ^ 1u, limit, abort_v)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int e = 0; e < N; ++e) lse_sh[r * kRows + 32 * e + lane] = nl[e];
        __syncwarp();
        if (lane == 0) mbar_arrive(&l_full[r]);
        if (++r == kLseRing) {
          r = 0;
          phase ^= 1u;
        }
      }
      if (!ok && lane == 0) raise_abort(abort_v, a.status);
    } else {
      const int t = warp >> 3, half = (warp >> 2) & 1;
      const int r = (warp & 3) * 32 + lane;
      const uint32_t tS = tmem + (uint32_t((warp & 3) * 32) << 16) + t * 256 + half * 64;
      const int32_t k = w.tile * 2 * kRows + t * kRows + r;
      const float2 c2 = make_float2(a.scale * kLog2e, a.scale * kLog2e);
      float comp = 0.f;
      bool ok = true;
      uint32_t ring = 0, l_phase = 0, n = 0;
      for (int32_t i = begin; i < n_qt; i += step) {
        if (!warp_wait(&l_full[ring], l_phase, limit, abort_v)) {
          ok = false;
          break;
        }
        if (i >= (t == 0 ? i0[0] : i0[1])) {
          const uint32_t buf = n & 1u, s_phase = (n >> 1) & 1u;
          ++n;
          if (!warp_wait(&s_full[t * 2 + buf], s_phase, limit, abort_v)) {
            ok = false;
            break;
          }
          tc_fence_after();
          // pairs [lo, hi) of this half of the tile count: queries that see this key, and that exist
          // (cut at 0 first: a key long before the queries lies 2^31 pairs before them)
          const int32_t lo = a.causal ? max(k - off - i * p.nq_tile, 0) * p.g - 64 * half : 0;
          const int32_t hi = min(p.nq_tile, S_q - i * p.nq_tile) * p.g - 64 * half;
          const bool masked = __any_sync(0xffffffffu, lo > 0) || hi < 64;
          const float* nl = lse_sh + ring * kRows + 64 * half;
          float2 part[4];
#pragma unroll
          for (int v = 0; v < 4; ++v) part[v] = make_float2(0.f, 0.f);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t s[32];
            tmem_ld_32x32b_x32(tS + buf * 128 + 32 * x, s);
            tmem_ld_wait(s);
            if (x == 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&s_empty[t * 2 + buf]);
            }
            auto add_up = [&](auto mask) {
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 l4 = *reinterpret_cast<const float4*>(nl + 32 * x + e);
                const uint32_t* v = &s[e];
                float2 y[2] = {fma2(make_float2(__uint_as_float(v[0]), __uint_as_float(v[1])), c2,
                                    make_float2(l4.x, l4.y)),
                               fma2(make_float2(__uint_as_float(v[2]), __uint_as_float(v[3])), c2,
                                    make_float2(l4.z, l4.w))};
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  if constexpr (decltype(mask)::value) {  // whatever the product or its lse is
                    const int col = 32 * x + e + 2 * z;
                    if (col < lo || col >= hi) y[z].x = -INFINITY;
                    if (col + 1 < lo || col + 1 >= hi) y[z].y = -INFINITY;
                  }
                  float2& sum = part[((e >> 1) + z) & 3];
                  sum = add2(sum, make_float2(ex2(y[z].x), ex2(y[z].y)));
                }
              }
            };
            if (masked)
              add_up(std::true_type());
            else
              add_up(std::false_type());
          }
          const float2 p2 = add2(add2(part[0], part[1]), add2(part[2], part[3]));
          // total + comp: the sum with the rounding of each addition carried along
          const float y = __fsub_rn(__fadd_rn(p2.x, p2.y), comp);
          const float z = __fadd_rn(total, y);
          comp = __fsub_rn(__fsub_rn(z, total), y);
          total = z;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&l_empty[ring]);
        if (++ring == kLseRing) {
          ring = 0;
          l_phase ^= 1u;
        }
      }
      if (!ok && lane == 0) raise_abort(abort_v, a.status);
      sum_sh[(half * 2 + t) * kRows + r] = total;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWtMma) tmem_dealloc<1>(tmem, 512);
  if (p.split > 1) cluster_sync_all();
  if (w.tile >= 0) {
    const int32_t per = 2 * kRows / int32_t(p.split);
    const int32_t k = w.tile * 2 * kRows + int32_t(rank) * per + int32_t(threadIdx.x);
    if (int32_t(threadIdx.x) < per && k < w.s.k1 - w.s.k0) {
      const int32_t i = int32_t(rank) * per + int32_t(threadIdx.x);
      float x = 0.f;
      for (uint32_t r = 0; r < p.split; ++r) {
        const uint32_t at = p.split == 1 ? 0u : mapa_shared(smem_addr(sum_sh + i), r);
        x += p.split == 1 ? sum_sh[i] + sum_sh[2 * kRows + i]
                          : ld_cluster_f32(at) + ld_cluster_f32(at + 2 * kRows * 4);
      }
      if (!isfinite(x)) status_or(a.status, RMM_NONFINITE_BIT);
      const int64_t at = int64_t(h) * a.T_k + w.s.k0 + k;
      a.w_out[at] = a.w_in ? a.w_in[at] + x : x;
    }
  }
  if (p.split > 1) cluster_sync_all();  // no CTA leaves while another reads its sums
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

template <int DP>
cudaError_t launch_weights(TcArgs p, cudaStream_t st, const char** why) {
  using Cfg = WeightCfg<DP>;
  const AttnArgs& a = p.a;
  CUtensorMap tmQ, tmK;
  bool ok = encode_tokens(&tmK, a.k, a.T_k, a.h_kv, a.d, kRows, 1);
  if (a.T_q > 0)
    ok = ok && encode_tokens(&tmQ, a.q, a.T_q, a.h_q, a.d, uint32_t(p.nq_tile), uint32_t(p.g));
  else
    tmQ = tmK;  // no query is ever loaded
  if (!ok) {
    *why = "cuTensorMapEncodeTiled failed for Q or K";
    return cudaErrorInvalidValue;
  }
  cudaError_t e = cudaFuncSetAttribute(attn_key_weights_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       int(Cfg::SMEM));
  if (e != cudaSuccess) return e;
  const int64_t span = 2 * kRows;
  const int64_t units = (a.n_seq == 1 ? (a.T_k + span - 1) / span : a.T_k / span + a.n_seq) * a.h_kv;
  // Enough CTAs to even out the units' different lengths over 148 SMs, but at
  // least 4 query tiles each on average. The CTAs of a cluster need that many
  // free SMs of one GPC at once, so larger clusters pay only while all CTAs
  // find room: eight while they fit the SMs, four up to about two per SM, pairs
  // beyond (us alone, in pairs, fours, eights; d = 128):
  //   16 units, 6 heads on one key head, 4096 tokens    307  160   90   51
  //   32 units, 1024 tokens                              51   33   23   33
  //   64 units, 2048 tokens                              96   57   45   66
  //  128 units, 4096 tokens                             186  102  123  164
  //  256 units, 8192 tokens                             363  346  404  506
  //  312 units, a packed batch                          184  148  191  281
  //  512 units, 16384 tokens                           1278 1255 1454 1761
  // (d = 64: 128 units 33, 29, 43, 78; 256 units 57, 72, 102, 172.)
  // The lengths are on the device, so the number of query tiles is an average.
  // Batches of short prompts lose by clusters (16 x 256 tokens, 256 units: 25,
  // 35; 64 x 32 tokens, 576 units: 29, 59); one long prompt among 31 short ones,
  // which the average takes for short, would gain (184, 127).
  const int64_t q_tiles = (a.T_q / std::max<int64_t>(a.n_seq, 1)) / p.nq_tile;
  p.split = 1;
  if (units < 400 && q_tiles >= 8) p.split = 2;
  if (units * 4 <= 320 && q_tiles >= 16) p.split = 4;
  if (units * 8 <= 148 && q_tiles >= 32) p.split = 8;
  return launch_pdl(attn_key_weights_kernel<DP>, dim3(unsigned(units * p.split)), dim3(kWtThreads), Cfg::SMEM, st,
                    p.split > 1 ? dim3(p.split, 1, 1) : dim3(0, 0, 0), tmQ, tmK, p);
}

TcArgs tc_args(const AttnArgs& a) {
  TcArgs p;
  p.a = a;
  p.g = int32_t(a.h_q / a.h_kv);
  p.nq_tile = kRows / p.g;
  p.row_bytes = p.nq_tile * p.g * 128;
  p.split = 1;
  return p;
}

}  // namespace

cudaError_t launch_attn_prompt(const AttnArgs& a, cudaStream_t st, const char** why) {
  cudaError_t e = device_ok(why);
  if (e != cudaSuccess) return e;
  const TcArgs p = tc_args(a);
  return a.d <= 64 ? launch_prompt<64>(p, st, why) : launch_prompt<128>(p, st, why);
}

cudaError_t launch_attn_key_weights(const AttnArgs& a, cudaStream_t st, const char** why) {
  cudaError_t e = device_ok(why);
  if (e != cudaSuccess) return e;
  const TcArgs p = tc_args(a);
  return a.d <= 64 ? launch_weights<64>(p, st, why) : launch_weights<128>(p, st, why);
}

}  // namespace rmm
