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
#include <type_traits>

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
// A thread quantises 8 channels of a token's keys and of its values, four
// neighbouring lanes a group, 4·NG a row; a block takes rows of one head.
// Bound by HBM for whole prompts: 2·d values read, 2·(d/2 + d/8) bytes written.
constexpr int kStoreThreads = 256;

template <typename T>
__device__ __forceinline__ void load8(float (&f)[8], const T* p, bool vec) {
  if (vec) {
    if constexpr (sizeof(T) == 2) {
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[2 * e] = __uint_as_float(w[e] << 16);
        f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 u = reinterpret_cast<const float4*>(p)[h];
        f[4 * h] = u.x, f[4 * h + 1] = u.y, f[4 * h + 2] = u.z, f[4 * h + 3] = u.w;
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = elem_to_f32(p[e]);
  }
}

// bf16(range / 15), the quotient IEEE's. The product with 1/15 is off by at most
// two units in its last place, which matters next to the middle of two bf16
// numbers only (and below the normal range).
__device__ __forceinline__ float fifteenth(float range) {
  const float q = range * (1.0f / 15.0f);
  const uint32_t low = (__float_as_uint(q) & 0xFFFFu) - 0x7FFCu;
  return low <= 8u || q < 0x1p-100f ? __fdiv_rn(range, 15.0f) : q;
}

// The 8 codes of x (channel pairs), nibble e for channel e: rint((x - mn) / step)
// within 0 .. 15. The product with the approximate reciprocal is within 2^-17 of
// the quotient (about -1 to 17), so only where one lands next to a half, or
// where the reciprocal is no normal number, are the divisions made.
__device__ __forceinline__ uint32_t codes_of(const float2 (&x)[4], float step, float mn) {
  if (!(step > 0.f)) return 0;
  auto both = [](float v) { return make_float2(v, v); };
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(step));
  float2 r[4];
  float far = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    // the nearest integer, by an addition that leaves no bits below 1 (exact for quotients below 2^22)
    const float2 q = mul2(add2(x[e], both(-mn)), both(inv));
    r[e] = add2(add2(q, both(12582912.f)), both(-12582912.f));
    const float2 off = fma2(r[e], both(-1.f), q);
    far = max3(far, fabsf(off.x), fabsf(off.y));
  }
  if (!(far < 0.5f - 0x1p-15f && step > 0x1p-120f && step < 0x1p120f)) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      r[e] = make_float2(rintf(__fdiv_rn(x[e].x - mn, step)), rintf(__fdiv_rn(x[e].y - mn, step)));
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    r[e] = make_float2(fminf(fmaxf(r[e].x, 0.f), 15.f), fminf(fmaxf(r[e].y, 0.f), 15.f));
  // four codes as one number below 2^16
  const float2 lo = fma2(r[1], both(256.f), r[0]), hi = fma2(r[3], both(256.f), r[2]);
  return uint32_t(fmaf(lo.y, 16.f, lo.x)) | uint32_t(fmaf(hi.y, 16.f, hi.x)) << 16;
}

template <typename T, int NG>
__global__ void __launch_bounds__(kStoreThreads) kv4_store_kernel(const Kv4StoreArgs a, bool vec) {
  constexpr int LANES = 4 * NG, ROWS = kStoreThreads / LANES;
  pdl_trigger();
  pdl_wait();
  const int row = threadIdx.x / LANES, u = threadIdx.x % LANES;
  const int64_t h = blockIdx.y;
  const int w = u >> 2, j = u & 3;  // group, quarter of the group
  const int64_t t = int64_t(blockIdx.x) * ROWS + row;
  bool live = row < ROWS && t < a.T;
  const int64_t tc = min(t, a.T - 1);  // surplus threads repeat the last token and store nothing
  float x[2][8];
  load8(x[0], static_cast<const T*>(a.k.ptr) + tc * a.k.ts + h * a.k.hs + 8 * u, vec);
  load8(x[1], static_cast<const T*>(a.v.ptr) + tc * a.v.ts + h * a.v.hs + 8 * u, vec);
  int64_t b = tc, first = tc;
  if (a.cu) {
    b = find_seq(a.cu, a.n_seq, tc);
    first = a.cu[b];
    live = live && tc >= first && tc < a.cu[b + 1];
  }
  const int64_t slot = int64_t(a.start[b]) + (tc - first);
  const bool in_cache = slot >= 0 && slot < a.cap;
  const int64_t at = (b * a.h_kv + h) * a.cap + slot;
  bool odd = false;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    float2 p[4], zero = make_float2(0.f, 0.f);  // zero: NaN where an element, the step or the minimum is not finite
    float lo = x[kv][0], hi = lo;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      p[e] = make_float2(x[kv][2 * e], x[kv][2 * e + 1]);
      lo = min3(lo, p[e].x, p[e].y);
      hi = max3(hi, p[e].x, p[e].y);
      zero = fma2(p[e], make_float2(0.f, 0.f), zero);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    // (step, minimum) as stored; the IEEE quotient, so that it depends on nothing but the values
    const uint32_t sm = pack_bf16x2(fifteenth(hi - lo), lo);
    const float step = __uint_as_float(sm << 16), mn = __uint_as_float(sm & 0xFFFF0000u);
    zero = fma2(make_float2(step, mn), make_float2(0.f, 0.f), zero);
    odd |= zero.x + zero.y != 0.f;
    const uint32_t codes = codes_of(p, step, mn);
    // the values' half-words need one nibble from each of the group's four lanes
    uint32_t half[2] = {0u, 0u};  // half-words r = 2j, 2j + 1 of group w
    if (kv == 1) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const uint32_t c = __shfl_sync(0xffffffffu, codes, (threadIdx.x & 28) | s) >> (8 * j);
        half[0] |= (c & 15u) << (4 * s);
        half[1] |= ((c >> 4) & 15u) << (4 * s);
      }
    }
    if (!live || !in_cache) continue;
    if (j == 0) reinterpret_cast<uint32_t*>(kv ? a.c.vs : a.c.ks)[at * NG + w] = sm;
    if (kv == 0) {
      reinterpret_cast<uint32_t*>(a.c.kc)[at * LANES + j * NG + w] = codes;
    } else {
      uint16_t* v = reinterpret_cast<uint16_t*>(a.c.vc) + at * (2 * LANES);
      v[(2 * j) * NG + w] = uint16_t(half[0]);
      v[(2 * j + 1) * NG + w] = uint16_t(half[1]);
    }
  }
  if (!live) return;
  if (odd) status_or(a.status, RMM_NONFINITE_BIT);
  if (!in_cache)
    status_or(a.status, RMM_RANGE_BIT);
  else if (u == 0 && a.w)
    a.w[at] = a.w_new ? a.w_new[h * a.T + t] : 0.f;
}
// ---------------------------------------------------------------- attention
// The work is the tiles of 16 or 32 tokens of every item (sequence, key head, chunk
// of its query heads) with tokens, one item after the other; CTA c takes tiles
// [c·per, (c+1)·per) of the line, whichever items they are of, so ragged
// lengths leave no SM idle. A part of an item that one CTA works on is one
// partial result, in slot c + item: both only grow along the line, so no two
// share one.
struct Kv4Dev {
  Kv4AttnArgs a;
  float* ml;      // [slots][heads of a chunk][2] (maximum in log2 units, sum)
  float* po;      // [slots][heads of a chunk][d] unnormalised
  float* scores;  // [batch][h_kv][cap][h_q / h_kv] log2 units, or null
  int64_t* line;  // [batch + 1] first tile of each sequence, then all tiles; [batch + 1] tiles per CTA
  int32_t chunks, chunk_heads;  // per key head; query heads of a chunk
  int32_t tile;                 // tokens of a tile
};

__device__ __forceinline__ int32_t seq_len(const Kv4AttnArgs& a, int64_t b) {
  return int32_t(min(max(int64_t(a.lens[b]), int64_t(0)), a.cap));
}

// A CTA's warps take the tiles of a part in turn, each with a running maximum,
// sum and output of its own, joined at the part's end.
//
// Both products run on mma.sync (16 x 8 x 16; a step has a few query rows per
// key head, an eighth of the smallest tcgen05 tile), transposed so that the
// tokens or channels are the 16 rows and the heads the 8 columns, which lets
// the codes go from their bytes to operand registers with shifts and masks:
//   Sᵀ  A = codes of 16 tokens as f16 subnormals c·2^-24 (nibbles 0, 2 of a
//       half-word) or 16c·2^-24 (1, 3), B = q as f16. The head's queries are
//       scaled by a power of two to have their largest below 2^15, so bf16's 8
//       bits fit f16 exactly over 28 binades below it. One accumulator per
//       group of 32 channels, then S += step·acc in f32; min·(sum of q) of all
//       groups is one more product, the sums cut into three bf16 parts.
//   Oᵀ  A = codes of 16 channels, the same f16 subnormals, B = p·step of the
//       group in f16, transposed by movmatrix; p·min adds up in f32. A power of
//       two per head keeps the largest p·step so far near 2^12, and its tile's
//       below 2^15, lowered (and O with it) as larger ones come and raised again
//       as the running maximum leaves them behind: 11 bits where bf16 would keep
//       8, which matters since a value is the small difference of its min and
//       step·code (bf16: twice the error of the result). It follows p·step, not
//       the step, since a token of large values may have next to no weight; that
//       costs 1 % (batch of 32 x 8192: 81.4 us, one power of two from the steps
//       80.2). What lies 2^-26 below the head's largest p·step loses bits, and
//       below 2^-37 fades out.
// So a word of 8 codes costs one shift and four masks. What bounds the kernel
// is the rate of such instructions, then HBM.
// With up to 4 query heads per key head a tile has two halves of 16 tokens: the
// second half's scores and outputs take columns 4-7 of the same accumulators (B
// is zero in the other half's columns), so that no lane's scaling, exponentials
// and scales are spent on columns without a head (batch of 32 x 8192, 4 heads:
// 91 us without, 86 with).
// A tile's bytes come by cp.async through a ring per warp, STAGES - 1 tiles
// ahead; rows past the length arrive as zeros.
constexpr int kKvWarps = 8;
constexpr float kKvRescale = 8.0f;  // log2 of the growth of p that is let through unscaled

template <int NG, int HALVES>
struct KvTile {
  static constexpr int TOKENS = 16 * HALVES;
  static constexpr int CODES = TOKENS * 16 * NG;  // bytes of the rows of codes
  static constexpr int SCALES = TOKENS * 4 * NG;
  static constexpr int BYTES = 2 * (CODES + SCALES);
  static constexpr int STAGES = 4 / HALVES;
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
               " {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
               " {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float step_of(uint32_t sm) { return __uint_as_float(sm << 16); }
// the largest magnitude of a row's steps
template <int NG>
__device__ __forceinline__ float top_step(const uint32_t (&sm)[NG]) {
  uint32_t m = sm[0] & 0x7FFFu;
#pragma unroll
  for (int g = 1; g < NG; ++g) m = max(m, sm[g] & 0x7FFFu);
  return __uint_as_float(m << 16);
}
__device__ __forceinline__ float min_of(uint32_t sm) { return __uint_as_float(sm & 0xFFFF0000u); }

// NW consecutive 32-bit words from shared memory, 4·NW-byte aligned (NW 1, 2, 4) or 4-byte (3)
template <int NW>
__device__ __forceinline__ void lds_words(uint32_t (&w)[NW], const void* p) {
  if constexpr (NW == 4) {
    const uint4 v = *static_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (NW == 2) {
    const uint2 v = *static_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < NW; ++i) w[i] = static_cast<const uint32_t*>(p)[i];
  }
}

// half-word g of row a in the low half, of row b in the high half, g = 0 .. NG-1
template <int NG>
__device__ __forceinline__ void pair_halves(uint32_t (&w)[NG], const uint8_t* a, const uint8_t* b) {
  if constexpr (NG % 2 == 0) {
    uint32_t x[NG / 2], y[NG / 2];
    lds_words<NG / 2>(x, a);
    lds_words<NG / 2>(y, b);
#pragma unroll
    for (int g = 0; g < NG; ++g) w[g] = __byte_perm(x[g / 2], y[g / 2], g % 2 ? 0x7632 : 0x5410);
  } else {
#pragma unroll
    for (int g = 0; g < NG; ++g)
      w[g] = uint32_t(reinterpret_cast<const uint16_t*>(a)[g]) | uint32_t(reinterpret_cast<const uint16_t*>(b)[g]) << 16;
  }
}

// Tiles of the line before sequence b0 + i for each thread i's first sequence, and all tiles.
struct LinePos {
  int64_t before, all;
};
__device__ __forceinline__ LinePos line_scan(int64_t mine, int64_t* warp_sums, int tid) {
  const int lane = tid & 31, warp = tid >> 5;
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  LinePos r = {incl - mine, 0};
  for (int w = 0; w < kKvWarps; ++w) {
    if (w < warp) r.before += warp_sums[w];
    r.all += warp_sums[w];
  }
  return r;
}

// ceil(x / y), without the long 64-bit division wherever 32 bits do
__device__ __forceinline__ int64_t div_up(int64_t x, int64_t y) {
  if (((x + y) | y) >> 32 == 0) return (uint32_t(x) + uint32_t(y) - 1u) / uint32_t(y);
  return (x + y - 1) / y;
}

template <int NG, int NT, int HALVES>
__global__ void __launch_bounds__(kKvWarps * 32, NT == 1 ? 2 : 1) kv4_attn_split_kernel(const Kv4Dev p) {
  using Tile = KvTile<NG, HALVES>;
  constexpr int D = 32 * NG, HEADS = 8 * NT, STAGES = Tile::STAGES, TT = Tile::TOKENS;
  constexpr int SETS = NT * HALVES;  // operands of Sᵀ: of 8 heads each, or of the heads in one half's columns
  static_assert(NT == 1 || HALVES == 1, "halves share one tile of columns");
  extern __shared__ __align__(16) uint8_t kv_smem[];  // [warps][stages][tile], then the outputs
  __shared__ float m_sh[kKvWarps][HEADS], l_sh[kKvWarps][HEADS];
  __shared__ int64_t sums_sh[kKvWarps], b_sh, before_sh;
  __shared__ uint4 q_sh[SETS][SETS == 1 ? 1 : NG][SETS == 1 ? 1 : 32];  // the warps' common operand of Sᵀ
  static_assert(STAGES * Tile::BYTES >= HEADS * D * 4, "a warp's ring holds its outputs at the end");
  pdl_trigger();
  pdl_wait();
  const Kv4AttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, j = lane & 3;
  const int32_t gq = int32_t(a.h_q / a.h_kv);
  if (blockIdx.x == 0 && tid == 0) *static_cast<uint32_t*>(a.workspace) = 0u;

  // ---- this CTA's stretch of the line: a thread adds up the tiles of consecutive sequences
  const int32_t seq_items = int32_t(a.h_kv) * p.chunks;
  int64_t pos, end;
  {
    const int64_t each = (a.batch + kKvWarps * 32 - 1) / (kKvWarps * 32);
    const int64_t s0 = min(tid * each, a.batch), s1 = min(s0 + each, a.batch);
    int64_t mine = 0;
    for (int64_t i = s0; i < s1; ++i) mine += int64_t((seq_len(a, i) + TT - 1) / TT) * seq_items;
    const LinePos at = line_scan(mine, sums_sh, tid);
    // at least as many tiles as an item has on average, up to one per warp: fewer partial results to join
    const int64_t per = max(max(div_up(at.all, gridDim.x), int64_t(1)),
                            min(int64_t(kKvWarps), div_up(at.all, a.batch * seq_items)));
    pos = blockIdx.x * per;
    end = min(pos + per, at.all);
    int64_t before = at.before;
    for (int64_t i = s0; i < s1; ++i) {
      const int64_t n = int64_t((seq_len(a, i) + TT - 1) / TT) * seq_items;
      if (before <= pos && pos < before + n) {
        b_sh = i;
        before_sh = before;
      }
      if (blockIdx.x == 0) p.line[i] = before;
      before += n;
    }
    if (blockIdx.x == 0 && tid == 0) {
      p.line[a.batch] = at.all;
      p.line[a.batch + 1] = per;
    }
  }
  if (pos >= end) return;
  __syncthreads();
  int64_t b = b_sh;
  int32_t len = seq_len(a, b), item_tiles = (len + TT - 1) / TT;
  int32_t in_seq = int32_t(div_up(pos - before_sh + 1, item_tiles)) - 1;  // item of the sequence: (key head, chunk)
  int32_t first = int32_t(pos - before_sh - int64_t(in_seq) * item_tiles);
  uint8_t* ring = kv_smem + warp * (STAGES * Tile::BYTES);

  for (;;) {  // a part: tiles [first, first + tiles) of an item
  const int32_t tiles = int32_t(min(int64_t(item_tiles - first), end - pos));
  const int64_t item = b * a.h_kv + in_seq / p.chunks;
  const int32_t head0 = int32_t(in_seq % p.chunks) * HEADS;  // first of the chunk's heads within the group
  const int64_t hq0 = (item - b * a.h_kv) * gq + head0;
  const int32_t heads = min(HEADS, gq - head0);
  const int32_t t0 = TT * first, t1 = min(len, t0 + TT * tiles);
  const int64_t slot = blockIdx.x + b * seq_items + in_seq;

  const int64_t row0 = item * a.cap + t0;
  const int32_t rows = t1 - t0;
  constexpr int SB = NG == 4 ? 16 : 4;  // bytes of a piece of the scales: rows of 16 bytes are copied whole
  // one plane's rows of a tile, in pieces of SIZE bytes; rows past the length become zeros
  auto copy = [&](auto size, auto total, uint8_t* dst, const uint8_t* src, int32_t live_bytes) {
    constexpr int SIZE = decltype(size)::value, PIECES = decltype(total)::value / SIZE;
#pragma unroll
    for (int i = 0; i < (PIECES + 31) / 32; ++i) {
      const int off = (lane + 32 * i) * SIZE;
      if (PIECES % 32 != 0 && lane + 32 * i >= PIECES) continue;
      const bool in = off < live_bytes;
      if constexpr (SIZE == 16)
        cp_async16(dst + off, in ? src + off : src, in ? 16 : 0);
      else
        cp_async4(dst + off, in ? src + off : src, in ? 4 : 0);
    }
  };
  const uint8_t *k_src = a.c.kc + row0 * (16 * NG), *v_src = a.c.vc + row0 * (16 * NG);
  const uint8_t* ks_src = reinterpret_cast<const uint8_t*>(a.c.ks) + row0 * (4 * NG);
  const uint8_t* vs_src = reinterpret_cast<const uint8_t*>(a.c.vs) + row0 * (4 * NG);
  auto load = [&](int32_t tile, uint8_t* dst) {
    using Codes = std::integral_constant<int, Tile::CODES>;
    using Scales = std::integral_constant<int, Tile::SCALES>;
    const int64_t off = int64_t(tile) * Tile::CODES, soff = int64_t(tile) * Tile::SCALES;
    const int32_t live = rows - TT * tile;
    auto all = [&](int32_t code_bytes, int32_t scale_bytes) {
      copy(std::integral_constant<int, 16>(), Codes(), dst, k_src + off, code_bytes);
      copy(std::integral_constant<int, 16>(), Codes(), dst + Tile::CODES, v_src + off, code_bytes);
      copy(std::integral_constant<int, SB>(), Scales(), dst + 2 * Tile::CODES, ks_src + soff, scale_bytes);
      copy(std::integral_constant<int, SB>(), Scales(), dst + 2 * Tile::CODES + Tile::SCALES, vs_src + soff, scale_bytes);
    };
    if (live >= TT)
      all(Tile::CODES, Tile::SCALES);
    else
      all(live * (16 * NG), live * (4 * NG));
  };
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) {
    const int32_t tile = warp + s * kKvWarps;
    if (tile < tiles) load(tile, ring + s * Tile::BYTES);
    cp_async_commit();
  }

  // Queries of the head of column r (of each n tile), channels 32g + 8j .. + 7:
  // the operand of Sᵀ. Then of columns 2j, 2j+1, what their scores are made of.
  const int lh = HALVES == 2 ? j >> 1 : 0;  // half of the tile that columns 2j, 2j+1 are of
  auto head_of = [](int col) { return HALVES == 2 ? col & 3 : col; };
  // One operand stays in registers; two are read again from shared memory.
  uint32_t qsum[SETS][2];  // head r's sum of q over group j as three bf16 parts
  uint4 q_reg[SETS == 1 ? NG : 1];
  float fh[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int head = 8 * n + head_of(r);
    const bool live = head < heads;
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + b * a.q_ss + (hq0 + (live ? head : 0)) * a.q_hs;
    uint32_t w[NG][4];
    uint32_t top = 0;  // largest magnitude, as its bf16 bits
    float sum[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const uint4 u = live ? *reinterpret_cast<const uint4*>(q + 32 * g + 8 * j) : make_uint4(0u, 0u, 0u, 0u);
      w[g][0] = u.x, w[g][1] = u.y, w[g][2] = u.z, w[g][3] = u.w;
      sum[g] = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        top = max(top, max(w[g][e] & 0x7FFFu, (w[g][e] >> 16) & 0x7FFFu));
        sum[g] += __uint_as_float(w[g][e] << 16) + __uint_as_float(w[g][e] & 0xFFFF0000u);
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
      for (int g = 0; g < NG; ++g) sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], o);
    }
    // the power of two: largest query below 2^15 (a head of zeros, or of next to nothing, by 2^114)
    const int32_t e = top ? max(int32_t(top >> 7) - 127 - 14, -114) : 0;
    const float mul = __uint_as_float(uint32_t(127 - e) << 23);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float f[8];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        f[2 * c] = __uint_as_float(w[g][c] << 16) * mul;
        f[2 * c + 1] = __uint_as_float(w[g][c] & 0xFFFF0000u) * mul;
      }
      // nibbles (c, c + 4) share a register; odd ones arrive 16 times too large
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float k = c % 2 ? 0.0625f : 1.0f;
        f[c] = __uint_as_float(pack_f16x2(f[c] * k, f[c + 4] * k));
      }
      {
        const uint4 u = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                   __float_as_uint(f[3]));
        if constexpr (SETS == 1) {
          q_reg[g] = u;
        } else if (warp == 0) {
#pragma unroll
          for (int h = 0; h < HALVES; ++h)
            q_sh[n + h][g][lane] = HALVES == 1 || r >> 2 == h ? u : make_uint4(0u, 0u, 0u, 0u);
        }
      }
    }
    float qs = sum[0];
#pragma unroll
    for (int g = 1; g < NG; ++g)
      if (j == g) qs = sum[g];
    qs = j < NG ? qs * mul * 0x1p-24f : 0.f;
    const uint32_t hi = pack_bf16x2(qs, 0.f) << 16;
    const float rest = qs - __uint_as_float(hi);
    const uint32_t parts = pack_bf16x2(qs, rest);
    const uint32_t last = pack_bf16x2(rest - __uint_as_float(parts & 0xFFFF0000u), 0.f);
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
      const bool mine = HALVES == 1 || r >> 2 == h;
      qsum[n + h][0] = mine ? parts : 0u;
      qsum[n + h][1] = mine ? last : 0u;
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int32_t eh = __shfl_sync(0xffffffffu, e, 4 * (2 * j + x));  // a lane that holds column 2j + x
      fh[n][x] = a.scale * 1.4426950408889634f * 0x1p24f * __uint_as_float(uint32_t(127 + eh) << 23);
    }
  }

  float o[NT][2 * NG][4], om[NT][NG][2], nm[NT][2], l[NT][2];
  float up[NT][2], lim[NT][2];  // the power of two; 4 times the largest p·step it was chosen for (0: none yet)
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      nm[n][x] = INFINITY;  // minus the maximum: none yet
      l[n][x] = lim[n][x] = 0.f;
      up[n][x] = 1.f;
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      om[n][g][0] = om[n][g][1] = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) o[n][2 * g][c] = o[n][2 * g + 1][c] = 0.f;
    }
  }

  if constexpr (SETS > 1) __syncthreads();  // q_sh is written
  int stage = 0;
  for (int32_t tile = warp; tile < tiles; tile += kKvWarps) {
    {
      const int32_t ahead = tile + (STAGES - 1) * kKvWarps;
      const int s = stage == 0 ? STAGES - 1 : stage - 1;
      if (ahead < tiles) load(ahead, ring + s * Tile::BYTES);
      cp_async_commit();
    }
    cp_async_wait<STAGES - 1>();
    __syncwarp();
    const uint8_t* buf = ring + stage * Tile::BYTES;
    const uint8_t *kc = buf, *vc = buf + Tile::CODES, *ks = buf + 2 * Tile::CODES, *vs = ks + Tile::SCALES;
    const int32_t tok = t0 + TT * tile + 16 * lh + r;  // tokens tok and tok + 8

    // ---- scores
    float t[NT][4];
    {
      uint32_t w0[HALVES][NG], w1[HALVES][NG], s0[NG], s1[NG];
      lds_words<NG>(s0, ks + (16 * lh + r) * (4 * NG));
      lds_words<NG>(s1, ks + (16 * lh + r + 8) * (4 * NG));
      const int jg = NG == 4 ? j : min(j, NG - 1);
#pragma unroll
      for (int n = 0; n < NT; ++n) t[n][0] = t[n][1] = t[n][2] = t[n][3] = 0.f;
#pragma unroll
      for (int h = 0; h < HALVES; ++h) {
        const uint8_t *k0 = kc + (16 * h + r) * (16 * NG) + j * (4 * NG), *m = ks + (16 * h + r) * (4 * NG) + 4 * jg;
        lds_words<NG>(w0[h], k0);
        lds_words<NG>(w1[h], k0 + 8 * (16 * NG));
        const uint32_t m0 = __byte_perm(*reinterpret_cast<const uint32_t*>(m), 0, 0x3232);
        const uint32_t m1 = __byte_perm(*reinterpret_cast<const uint32_t*>(m + 8 * (4 * NG)), 0, 0x3232);
        const uint32_t mins[4] = {m0, m1, m0, m1};
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_bf16(t[n], mins, qsum[n + h][0], qsum[n + h][1]);
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const float st0 = step_of(s0[g]), st1 = step_of(s1[g]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int h = 0; h < HALVES; ++h) {
            const uint32_t x0 = w0[h][g], x1 = w1[h][g], h0 = x0 >> 8, h1 = x1 >> 8;
            const uint32_t lo[4] = {x0 & 0x000F000Fu, x1 & 0x000F000Fu, x0 & 0x00F000F0u, x1 & 0x00F000F0u};
            const uint32_t hi[4] = {h0 & 0x000F000Fu, h1 & 0x000F000Fu, h0 & 0x00F000F0u, h1 & 0x00F000F0u};
            const uint4 q = SETS == 1 ? q_reg[SETS == 1 ? g : 0] : q_sh[n + h][g][lane];
            mma_f16(c, lo, q.x, q.y);
            mma_f16(c, hi, q.z, q.w);
          }
          t[n][0] = fmaf(c[0], st0, t[n][0]);
          t[n][1] = fmaf(c[1], st0, t[n][1]);
          t[n][2] = fmaf(c[2], st1, t[n][2]);
          t[n][3] = fmaf(c[3], st1, t[n][3]);
        }
      }
    }
    const bool in0 = tok < t1, in1 = tok + 8 < t1;  // false in a part's last tile only
    if (p.scores) {
      float* dst = p.scores + (item * a.cap + tok) * gq + head0;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int head = 8 * n + head_of(2 * j + x);
          if (head >= heads) continue;
          if (in0) dst[head] = t[n][x] * fh[n][x];
          if (in1) dst[8 * gq + head] = t[n][2 + x] * fh[n][x];
        }
    }
    // ---- softmax: p = 2^(t·fh - maximum), the maximum one the whole warp uses
    uint32_t s0[NG], s1[NG];  // the values' steps and minima
    lds_words<NG>(s0, vs + (16 * lh + r) * (4 * NG));
    lds_words<NG>(s1, vs + (16 * lh + r + 8) * (4 * NG));
    const float step0 = top_step<NG>(s0), step1 = top_step<NG>(s1);
    float pr[NT][4], big[NT][4];  // p, p·up
    float top = -INFINITY, over = 0.f;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float y0 = fmaf(t[n][x], fh[n][x], nm[n][x]), y1 = fmaf(t[n][2 + x], fh[n][x], nm[n][x]);
        top = max3(top, y0, y1);
        pr[n][x] = ex2f(y0), pr[n][2 + x] = ex2f(y1);
        big[n][x] = pr[n][x] * up[n][x], big[n][2 + x] = pr[n][2 + x] * up[n][x];
        over = max3(over, big[n][x] * step0, big[n][2 + x] * step1);
      }
    const bool tail = TT * tile + TT > rows;
    if (__any_sync(0xffffffffu, tail || top > kKvRescale || over > 0x1p15f)) {
      if (tail) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (!(c < 2 ? in0 : in1)) t[n][c] = -INFINITY;
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          // fh is positive. A column of the second half may have no token yet: its maximum stays -inf.
          float mx = fmaxf(t[n][x], t[n][2 + x]) * fh[n][x];
#pragma unroll
          for (int s = 4; s < 32; s <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
          const float nm2 = fminf(nm[n][x], -mx);
          const float f = nm2 == nm[n][x] ? 1.f : ex2f(nm2 - nm[n][x]);  // 0 the first time
          nm[n][x] = nm2;
          pr[n][x] = t[n][x] == -INFINITY ? 0.f : ex2f(fmaf(t[n][x], fh[n][x], nm2));
          pr[n][2 + x] = t[n][2 + x] == -INFINITY ? 0.f : ex2f(fmaf(t[n][2 + x], fh[n][x], nm2));
          float ps = fmaxf(pr[n][x] * step0, pr[n][2 + x] * step1);
#pragma unroll
          for (int s = 4; s < 32; s <<= 1) ps = fmaxf(ps, __shfl_xor_sync(0xffffffffu, ps, s));
          // 4 times the largest p·step becomes 2^14 to 2^15. At most 2^119: p up to 2^8 times it is finite.
          lim[n][x] = fmaxf(lim[n][x] * f, 4.f * ps);
          const int32_t e = min(max(268 - int32_t(__float_as_uint(lim[n][x]) >> 23), 1), 246);
          const int32_t de = e - int32_t(__float_as_uint(up[n][x]) >> 23);
          const float fv = f * __uint_as_float(uint32_t(min(max(127 + de, 0), 254)) << 23);
          up[n][x] = __uint_as_float(uint32_t(e) << 23);
          big[n][x] = pr[n][x] * up[n][x], big[n][2 + x] = pr[n][2 + x] * up[n][x];
          l[n][x] *= f;
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            om[n][g][x] *= f;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              o[n][2 * g + u][x] *= fv;
              o[n][2 * g + u][2 + x] *= fv;
            }
          }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      l[n][0] += pr[n][0] + pr[n][2];
      l[n][1] += pr[n][1] + pr[n][3];
    }
    // ---- values
    uint32_t wl[HALVES][NG], wh[HALVES][NG];
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
      const uint8_t* v0 = vc + (16 * h + 2 * j) * (16 * NG) + r * (2 * NG);
      pair_halves<NG>(wl[h], v0, v0 + 16 * NG);
      pair_halves<NG>(wh[h], v0 + 8 * (16 * NG), v0 + 9 * (16 * NG));
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const float st0 = step_of(s0[g]), mn0 = min_of(s0[g]), st1 = step_of(s1[g]), mn1 = min_of(s1[g]);
      uint32_t b0[NT], b1[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        b0[n] = movmatrix_trans(pack_f16x2(big[n][0] * st0, big[n][1] * st0));
        b1[n] = movmatrix_trans(pack_f16x2(big[n][2] * st1, big[n][3] * st1));
        om[n][g][0] = fmaf(pr[n][0], mn0, fmaf(pr[n][2], mn1, om[n][g][0]));
        om[n][g][1] = fmaf(pr[n][1], mn0, fmaf(pr[n][3], mn1, om[n][g][1]));
      }
#pragma unroll
      for (int h = 0; h < HALVES; ++h) {
        const uint32_t x0 = wl[h][g], x1 = wh[h][g], h0 = x0 >> 8, h1 = x1 >> 8;
        const uint32_t av[2][4] = {{x0 & 0x000F000Fu, x0 & 0x00F000F0u, x1 & 0x000F000Fu, x1 & 0x00F000F0u},
                                   {h0 & 0x000F000Fu, h0 & 0x00F000F0u, h1 & 0x000F000Fu, h1 & 0x00F000F0u}};
        const uint32_t cols = HALVES == 1 || r >> 2 == h ? 0xFFFFFFFFu : 0u;  // column r's half
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_f16(o[n][2 * g], av[0], b0[n] & cols, b1[n] & cols);
          mma_f16(o[n][2 * g + 1], av[1], b0[n] & cols, b1[n] & cols);
        }
      }
    }
    stage = stage + 1 == STAGES ? 0 : stage + 1;
    __syncwarp();  // the stage is free for the next load
  }
  cp_async_wait<0>();
  __syncwarp();

  // ---- join the warps. A warp without a tile has maximum -inf, sum and outputs 0.
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
      for (int s = 4; s < 32; s <<= 1) {
        l[n][x] += __shfl_xor_sync(0xffffffffu, l[n][x], s);
#pragma unroll
        for (int g = 0; g < NG; ++g) om[n][g][x] += __shfl_xor_sync(0xffffffffu, om[n][g][x], s);
      }
      if (r == 0) {
        m_sh[warp][8 * n + 2 * j + x] = -nm[n][x];
        l_sh[warp][8 * n + 2 * j + x] = l[n][x];
      }
    }
  float* mine = reinterpret_cast<float*>(ring);  // [HEADS][D]
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float down[2] = {1.f / up[n][0], 1.f / up[n][1]};
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          mine[(8 * n + 2 * j + (c & 1)) * D + 32 * g + 16 * u + 8 * (c >> 1) + r] =
              fmaf(o[n][2 * g + u][c] * (c < 2 ? 0x1p24f : 0x1p20f), down[c & 1], om[n][g][c & 1]);
  }
  __syncthreads();
  if (tid < heads) {  // m_sh becomes the warps' factors (a head's second column: of the second half)
    float m = m_sh[0][tid];  // the first warp has a tile
#pragma unroll
    for (int w = 0; w < kKvWarps; ++w)
#pragma unroll
      for (int h = 0; h < HALVES; ++h) m = fmaxf(m, m_sh[w][tid + 4 * h]);
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kKvWarps; ++w)
#pragma unroll
      for (int h = 0; h < HALVES; ++h) {
        const float f = ex2f(m_sh[w][tid + 4 * h] - m);
        sum += l_sh[w][tid + 4 * h] * f;
        m_sh[w][tid + 4 * h] = f;
      }
    *reinterpret_cast<float2*>(p.ml + 2 * (slot * HEADS + tid)) = make_float2(m, sum);
  }
  __syncthreads();
  for (int i = 4 * tid; i < heads * D; i += 4 * kKvWarps * 32) {
    float4 out = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kKvWarps; ++w)
#pragma unroll
      for (int h = 0; h < HALVES; ++h) {
        const float f = m_sh[w][i / D + 4 * h];
        const float4 x =
            *reinterpret_cast<const float4*>(kv_smem + w * (STAGES * Tile::BYTES) + 4 * (i + 4 * h * D));
        out.x = fmaf(x.x, f, out.x), out.y = fmaf(x.y, f, out.y);
        out.z = fmaf(x.z, f, out.z), out.w = fmaf(x.w, f, out.w);
      }
    *reinterpret_cast<float4*>(p.po + slot * (HEADS * D) + i) = out;
  }
  pos += tiles;
  if (pos >= end) return;
  first = 0;
  if (++in_seq == seq_items) {
    in_seq = 0;
    do {
      len = seq_len(a, ++b);  // pos < end: a sequence with tokens follows
    } while (len == 0);
    item_tiles = (len + TT - 1) / TT;
  }
  __syncthreads();  // the outputs in shared memory are read
  }
}

// Joins the parts of each item. Blocks [0, batch·h_q): O and the log-sum-exp of
// one head. The rest, w_out = w_in + the group's probabilities, kJoinTokens
// each; their scores are on the way while the parts' sums are joined.
constexpr int kJoinThreads = 128;
constexpr int kJoinEach = 8;  // tokens of a thread
constexpr int kJoinTokens = kJoinThreads * kJoinEach;
constexpr int kJoinParts = 8;  // parts of an item on the way at once

// The slots of an item's parts: [first, last].
struct Parts {
  int64_t first, last;
};
__device__ __forceinline__ Parts item_parts(const Kv4Dev& p, int64_t b, int32_t in_seq, int32_t len) {
  const int64_t per = p.line[p.a.batch + 1], item = b * p.a.h_kv * p.chunks + in_seq;
  const int64_t tiles = (len + p.tile - 1) / p.tile, start = p.line[b] + in_seq * tiles;
  return Parts{item + div_up(start + 1, per) - 1, item + div_up(start + tiles, per) - 1};
}

// maximum and sum over the parts of one head (log2 units): every lane gets both
__device__ __forceinline__ float2 join_ml(const Kv4Dev& p, Parts s, int32_t head, int lane) {
  float m = -INFINITY;
  for (int64_t i = s.first + lane; i <= s.last; i += 32) m = fmaxf(m, p.ml[2 * (i * p.chunk_heads + head)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float l = 0.f;
  for (int64_t i = s.first + lane; i <= s.last; i += 32) {
    const float2 x = reinterpret_cast<const float2*>(p.ml)[i * p.chunk_heads + head];
    l += x.y * ex2f(x.x - m);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  return make_float2(m, l);
}

// GV: query heads per key head where that is 1, 2, 4 or 8; else 0, and the scores are read when they are needed.
template <int GV>
__global__ void __launch_bounds__(kJoinThreads) kv4_attn_join_kernel(const Kv4Dev p, int64_t o_blocks) {
  extern __shared__ float lse2[];  // [h_q / h_kv]
  pdl_trigger();
  pdl_wait();
  const Kv4AttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t gq = int32_t(a.h_q / a.h_kv);
  if (int64_t(blockIdx.x) < o_blocks) {
    const int64_t b = blockIdx.x / a.h_q, hq = blockIdx.x % a.h_q;
    const int32_t len = seq_len(a, b);
    const int32_t hg = int32_t(hq % gq), head = hg % p.chunk_heads;
    const Parts parts =
        len > 0 ? item_parts(p, b, int32_t(hq / gq) * p.chunks + hg / p.chunk_heads, len) : Parts{0, -1};
    // a thread per channel; all of them add up the parts' sums
    if (tid >= a.d) return;
    float m = -INFINITY, l = 0.f, o = 0.f;
    for (int64_t i = parts.first; len > 0 && i <= parts.last; i += kJoinParts) {
      float2 x[kJoinParts];
      float v[kJoinParts];
#pragma unroll
      for (int u = 0; u < kJoinParts; ++u) {
        const int64_t at = min(i + u, parts.last) * p.chunk_heads + head;
        x[u] = reinterpret_cast<const float2*>(p.ml)[at];
        v[u] = p.po[at * a.d + tid];
      }
      float mx = m;
#pragma unroll
      for (int u = 0; u < kJoinParts; ++u) mx = fmaxf(mx, x[u].x);
      const float f = ex2f(m - mx);
      l *= f;
      o *= f;
#pragma unroll
      for (int u = 0; u < kJoinParts; ++u) {
        if (i + u > parts.last) break;
        const float e = ex2f(x[u].x - mx);
        l = fmaf(x[u].y, e, l);
        o = fmaf(v[u], e, o);
      }
      m = mx;
    }
    if (tid == 0) {
      if (len > 0 && !(l > 0.f && l < INFINITY && isfinite(m)))
        status_or(static_cast<uint32_t*>(a.workspace), RMM_NONFINITE_BIT);
      if (a.lse) a.lse[b * a.h_q + hq] = len > 0 ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
    o = len > 0 ? o / l : 0.f;
    const int64_t at = b * a.o_ss + hq * a.o_hs + tid;
    if (a.out == kBF16)
      static_cast<uint16_t*>(a.o)[at] = uint16_t(pack_bf16x2(o, 0.f));
    else
      static_cast<float*>(a.o)[at] = o;
    return;
  }
  const int32_t i = int32_t(blockIdx.x - o_blocks);
  const int32_t pieces = int32_t((a.cap + kJoinTokens - 1) / kJoinTokens);
  const int64_t item = i / pieces;
  const int64_t b = item / a.h_kv, h = item % a.h_kv;
  const int32_t len = seq_len(a, b);
  const int32_t t0 = int32_t(i % pieces) * kJoinTokens;
  if (t0 >= len) return;
  float x[kJoinEach][GV > 0 ? GV : 1], w[kJoinEach];
#pragma unroll
  for (int e = 0; e < kJoinEach; ++e) {
    const int32_t t = min(t0 + e * kJoinThreads + tid, len - 1);
    const int64_t at = item * a.cap + t;
    if constexpr (GV % 4 == 0) {
#pragma unroll
      for (int v = 0; v < GV / 4; ++v) {
        const float4 u = reinterpret_cast<const float4*>(p.scores + at * GV)[v];
        x[e][4 * v] = u.x, x[e][4 * v + 1] = u.y, x[e][4 * v + 2] = u.z, x[e][4 * v + 3] = u.w;
      }
    } else {
#pragma unroll
      for (int v = 0; v < GV; ++v) x[e][v] = p.scores[at * GV + v];
    }
    w[e] = a.w_in ? a.w_in[at] : 0.f;
  }
  for (int g = warp; g < gq; g += kJoinThreads / 32) {
    const Parts parts = item_parts(p, b, int32_t(h) * p.chunks + g / p.chunk_heads, len);
    const float2 ml = join_ml(p, parts, g % p.chunk_heads, lane);
    if (lane == 0) lse2[g] = ml.x + log2f(ml.y);
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < kJoinEach; ++e) {
    const int32_t t = t0 + e * kJoinThreads + tid;
    if (t >= len) break;
    const int64_t at = item * a.cap + t;
    float s = 0.f;
    if constexpr (GV > 0) {
#pragma unroll
      for (int g = 0; g < GV; ++g) s += ex2f(x[e][g] - lse2[g]);
    } else {
      for (int g = 0; g < gq; ++g) s += ex2f(p.scores[at * gq + g] - lse2[g]);
    }
    a.w_out[at] = w[e] + s;
  }
}

}  // namespace

namespace {
template <typename T>
cudaError_t launch_store(const Kv4StoreArgs& a, cudaStream_t st) {
  constexpr int64_t per = 16 / sizeof(T);  // elements of a 16-byte load
  const bool vec = ((reinterpret_cast<uintptr_t>(a.k.ptr) | reinterpret_cast<uintptr_t>(a.v.ptr)) & 15u) == 0 &&
                   (a.T == 1 || (a.k.ts | a.v.ts) % per == 0) && (a.h_kv == 1 || (a.k.hs | a.v.hs) % per == 0);
  const int64_t rows = kStoreThreads / (a.d / 8);
  const dim3 grid(unsigned((a.T + rows - 1) / rows), unsigned(a.h_kv)), block(kStoreThreads), none(0, 0, 0);
  switch (a.d / kKv4Group) {
    case 1: return launch_pdl(kv4_store_kernel<T, 1>, grid, block, 0, st, none, a, vec);
    case 2: return launch_pdl(kv4_store_kernel<T, 2>, grid, block, 0, st, none, a, vec);
    case 3: return launch_pdl(kv4_store_kernel<T, 3>, grid, block, 0, st, none, a, vec);
    default: return launch_pdl(kv4_store_kernel<T, 4>, grid, block, 0, st, none, a, vec);
  }
}
}  // namespace

cudaError_t launch_kv4_store(const Kv4StoreArgs& a, cudaStream_t st) {
  return a.in == kBF16 ? launch_store<uint16_t>(a, st) : launch_store<uint32_t>(a, st);
}

// CTAs of the decode step: as many as stay resident, two per SM (one with 16 heads' outputs in registers).
static int64_t kv4_grid(int64_t items, int64_t tiles, bool one) {
  return std::min<int64_t>(one ? 2 * 148 : 148, items * tiles);
}

Kv4Ws kv4_ws(int64_t batch, int64_t h_q, int64_t h_kv, int64_t d, int64_t cap, bool weights) {
  Kv4Ws w;
  const int64_t group = h_q / h_kv;
  w.chunk_heads = group <= 8 ? 8 : 16;
  w.chunks = (group + w.chunk_heads - 1) / w.chunk_heads;
  const int64_t items = batch * h_kv * w.chunks;
  w.tile = group <= 4 ? 32 : 16;
  w.grid = kv4_grid(items, (cap + w.tile - 1) / w.tile, w.chunk_heads == 8);
  const int64_t rows = (w.grid + items) * w.chunk_heads;
  auto al = [](int64_t x) { return (x + 1023) / 1024 * 1024; };
  int64_t off = 1024;
  w.line = size_t(off);
  off += al((batch + 2) * 8);
  w.ml = size_t(off);
  off += al(rows * 8);
  w.o = size_t(off);
  off += al(rows * d * 4);
  w.scores = size_t(off);
  if (weights) off += al(batch * h_q * cap * 4);
  w.bytes = size_t(off);
  return w;
}

namespace {
template <int NG, int NT, int HALVES>
cudaError_t launch_split(const Kv4Dev& p, const Kv4Ws& w, cudaStream_t st) {
  using Tile = KvTile<NG, HALVES>;
  constexpr int smem = kKvWarps * Tile::STAGES * Tile::BYTES;
  cudaError_t e =
      cudaFuncSetAttribute(kv4_attn_split_kernel<NG, NT, HALVES>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv4_attn_split_kernel<NG, NT, HALVES>, dim3(unsigned(w.grid)), dim3(kKvWarps * 32), size_t(smem), st,
                    dim3(0, 0, 0), p);
}
template <int NG>
cudaError_t launch_split(const Kv4Dev& p, const Kv4Ws& w, cudaStream_t st) {
  if (w.tile == 32) return launch_split<NG, 1, 2>(p, w, st);
  return w.chunk_heads == 8 ? launch_split<NG, 1, 1>(p, w, st) : launch_split<NG, 2, 1>(p, w, st);
}
}  // namespace

cudaError_t launch_kv4_attn(const Kv4AttnArgs& a, cudaStream_t st) {
  const Kv4Ws w = kv4_ws(a.batch, a.h_q, a.h_kv, a.d, a.cap, a.w_out != nullptr);
  char* base = static_cast<char*>(a.workspace);
  Kv4Dev p;
  p.a = a;
  p.ml = reinterpret_cast<float*>(base + w.ml);
  p.po = reinterpret_cast<float*>(base + w.o);
  p.scores = a.w_out ? reinterpret_cast<float*>(base + w.scores) : nullptr;
  p.line = reinterpret_cast<int64_t*>(base + w.line);
  p.chunks = int32_t(w.chunks);
  p.chunk_heads = int32_t(w.chunk_heads);
  p.tile = int32_t(w.tile);
  cudaError_t e;
  switch (a.d / kKv4Group) {
    case 1: e = launch_split<1>(p, w, st); break;
    case 2: e = launch_split<2>(p, w, st); break;
    case 3: e = launch_split<3>(p, w, st); break;
    default: e = launch_split<4>(p, w, st); break;
  }
  if (e != cudaSuccess) return e;
  const int64_t o_blocks = a.batch * a.h_q;
  const int64_t w_blocks = a.w_out ? a.batch * a.h_kv * ((a.cap + kJoinTokens - 1) / kJoinTokens) : 0;
  const int64_t group = a.h_q / a.h_kv;
  const dim3 grid(unsigned(o_blocks + w_blocks)), block(kJoinThreads), none(0, 0, 0);
  if (group == 1) return launch_pdl(kv4_attn_join_kernel<1>, grid, block, size_t(group) * 4, st, none, p, o_blocks);
  if (group == 2) return launch_pdl(kv4_attn_join_kernel<2>, grid, block, size_t(group) * 4, st, none, p, o_blocks);
  if (group == 4) return launch_pdl(kv4_attn_join_kernel<4>, grid, block, size_t(group) * 4, st, none, p, o_blocks);
  if (group == 8) return launch_pdl(kv4_attn_join_kernel<8>, grid, block, size_t(group) * 4, st, none, p, o_blocks);
  return launch_pdl(kv4_attn_join_kernel<0>, grid, block, size_t(group) * 4, st, none, p, o_blocks);
}

}  // namespace rmm
