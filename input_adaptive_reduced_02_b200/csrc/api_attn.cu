// C ABI of the attention operators: packed prompts, the weight each key
// received, the 4-bit cache and eviction. Argument validation and launches
// only; nothing here allocates or synchronises, except in debug mode.
#include <algorithm>
#include <cmath>

#include "api_common.h"

namespace rmm {
namespace {

constexpr int64_t kMaxI32 = 0x7FFFFFFF;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// [tokens][heads][d] read by 16-byte tiles: base and strides, no overlap along
// one head's tokens.
rmm_status check_tokens(const char* name, const void* p, int64_t ts, int64_t hs, int64_t tokens, int64_t heads,
                        int64_t d) {
  if (tokens == 0) return RMM_OK;
  if (!p) return fail(RMM_ERR_INVALID, "%s is NULL", name);
  if (ts < 0 || hs < 0 || (tokens > 1 && ts < d) || (heads > 1 && hs < d))
    return fail(RMM_ERR_INVALID, "%s layout (token or head stride) is too small", name);
  if (!aligned(p, 16) || (tokens > 1 && ts % 8 != 0) || (heads > 1 && hs % 8 != 0))
    return fail(RMM_ERR_INVALID, "%s must be 16-byte aligned with strides that are multiples of 8 elements", name);
  return RMM_OK;
}

// An output may be token-major or head-major, but no two rows may share memory.
rmm_status check_output(const char* name, const void* p, int64_t ts, int64_t hs, int64_t tokens, int64_t heads,
                        int64_t d) {
  rmm_status r = check_tokens(name, p, ts, hs, tokens, heads, d);
  if (r) return r;
  const bool token_major = tokens <= 1 || ts >= (heads - 1) * hs + d;
  const bool head_major = heads <= 1 || hs >= (tokens - 1) * ts + d;
  if (tokens > 0 && !token_major && !head_major)
    return fail(RMM_ERR_INVALID, "%s rows overlap (token and head stride)", name);
  return RMM_OK;
}

rmm_status check_heads(int64_t h_q, int64_t h_kv, int64_t max_group) {
  if (h_q < 1 || h_kv < 1 || h_q % h_kv != 0 || h_q > 65535)
    return fail(RMM_ERR_INVALID, "h_q must be a multiple of h_kv (both at least 1, h_q at most 65535)");
  if (h_q / h_kv > max_group)
    return fail(RMM_ERR_UNSUPPORTED, "more than %lld query heads share a key head", (long long)max_group);
  return RMM_OK;
}

rmm_status check_scale(float scale) {
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(RMM_ERR_INVALID, "scale must be finite and positive");
  return RMM_OK;
}

rmm_status check_prompt(const AttnArgs& a, rmm_dtype in) {
  rmm_status r;
  if (a.n_seq < 0 || a.T_q < 0 || a.T_k < 0) return fail(RMM_ERR_INVALID, "negative size");
  if (a.n_seq > 65535 || a.T_q > kMaxI32 - 256 || a.T_k > kMaxI32 - 256)
    return fail(RMM_ERR_UNSUPPORTED, "more than 65535 sequences or 2^31 - 257 tokens");
  if (!dtype_ok(in)) return fail(RMM_ERR_INVALID, "unknown input dtype");
  if (in != RMM_BF16) return fail(RMM_ERR_UNSUPPORTED, "attention takes bf16 queries, keys and values");
  if ((r = check_heads(a.h_q, a.h_kv, 128))) return r;
  if (a.d < 1) return fail(RMM_ERR_INVALID, "d must be at least 1");
  if (a.d % 8 != 0 || a.d > 128) return fail(RMM_ERR_UNSUPPORTED, "d must be a multiple of 8, at most 128");
  // one block per tile (256 rows of queries, or 256 keys) and key head
  const int64_t span = 2 * (128 / (a.h_q / a.h_kv));
  if (std::max(a.T_q / span, a.T_k / 256) + a.n_seq + 1 > kMaxI32 / a.h_kv)
    return fail(RMM_ERR_UNSUPPORTED, "more tiles of all sequences and heads than a grid holds");
  if ((r = check_scale(a.scale))) return r;
  if (a.n_seq != 1 && (!a.cu_q || !a.cu_k))
    return fail(RMM_ERR_INVALID, "cu_q and cu_k may be NULL for a single sequence only");
  if ((r = check_tokens("Q", a.q.ptr, a.q.ts, a.q.hs, a.T_q, a.h_q, a.d))) return r;
  return check_tokens("K", a.k.ptr, a.k.ts, a.k.hs, a.T_k, a.h_kv, a.d);
}

rmm_status check_planes(const Kv4Planes& c, int64_t batch, int64_t h_kv, int64_t d, int64_t cap) {
  if (d < 1 || cap < 1) return fail(RMM_ERR_INVALID, "d and cap must be at least 1");
  if (d % kKv4Group != 0 || d > kKv4MaxD)
    return fail(RMM_ERR_UNSUPPORTED, "the 4-bit cache takes d = 32, 64, 96 or 128");
  if (cap > kMaxSelectK) return fail(RMM_ERR_UNSUPPORTED, "cap above 2^21");
  if (batch > 0 && (!c.kc || !c.ks || !c.vc || !c.vs)) return fail(RMM_ERR_INVALID, "a cache plane is NULL");
  if (!aligned(c.kc, 16) || !aligned(c.ks, 16) || !aligned(c.vc, 16) || !aligned(c.vs, 16))
    return fail(RMM_ERR_INVALID, "the cache planes must be 16-byte aligned");
  if (batch > 65535 || h_kv > 65535 || batch * h_kv > 65535) return fail(RMM_ERR_UNSUPPORTED, "more than 65535 (sequence, head) pairs");
  return RMM_OK;
}

bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + uintptr_t(nb) && y < x + uintptr_t(na);
}

int64_t up1k(int64_t x) { return (x + 1023) / 1024 * 1024; }

}  // namespace
}  // namespace rmm

using namespace rmm;

rmm_status rmm_attn_prompt(const void* Q, int64_t q_ts, int64_t q_hs, const void* K, int64_t k_ts, int64_t k_hs,
                           const void* V, int64_t v_ts, int64_t v_hs, const int32_t* cu_q, const int32_t* cu_k,
                           int64_t n_seq, int64_t T_q, int64_t T_k, int64_t h_q, int64_t h_kv, int64_t d, float scale,
                           int causal, rmm_dtype in, void* O, int64_t o_ts, int64_t o_hs, rmm_dtype out, float* lse,
                           uint32_t* status_word, cudaStream_t stream) {
  AttnArgs a = {};
  a.q = TokView{Q, q_ts, q_hs};
  a.k = TokView{K, k_ts, k_hs};
  a.v = TokView{V, v_ts, v_hs};
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.n_seq = n_seq;
  a.T_q = T_q;
  a.T_k = T_k;
  a.h_q = h_q;
  a.h_kv = h_kv;
  a.d = d;
  a.scale = scale;
  a.causal = causal != 0;
  a.o = O;
  a.o_ts = o_ts;
  a.o_hs = o_hs;
  a.out = kind(out);
  a.lse = lse;
  a.status = status_word;
  a.wait_limit_ns = wait_limit();
  rmm_status r = check_prompt(a, in);
  if (r) return r;
  if (!dtype_ok(out)) return fail(RMM_ERR_INVALID, "unknown output dtype");
  if ((r = check_tokens("V", V, v_ts, v_hs, T_k, h_kv, d))) return r;
  if ((r = check_output("O", O, o_ts, o_hs, T_q, h_q, d))) return r;
  if (n_seq == 0 || T_q == 0) return RMM_OK;
  DeviceGuard dg;
  if ((r = bind_device(stream, dg))) return r;
  StageRange range("rmm attention");
  const char* why = nullptr;
  const cudaError_t e = launch_attn_prompt(a, stream, &why);
  return e == cudaSuccess ? RMM_OK : cuda_fail(e, "attention kernel", why);
}

rmm_status rmm_attn_key_weights(const void* Q, int64_t q_ts, int64_t q_hs, const void* K, int64_t k_ts, int64_t k_hs,
                                const int32_t* cu_q, const int32_t* cu_k, int64_t n_seq, int64_t T_q, int64_t T_k,
                                int64_t h_q, int64_t h_kv, int64_t d, float scale, int causal, rmm_dtype in,
                                const float* lse, const float* w_in, float* w_out, uint32_t* status_word,
                                cudaStream_t stream) {
  AttnArgs a = {};
  a.q = TokView{Q, q_ts, q_hs};
  a.k = TokView{K, k_ts, k_hs};
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.n_seq = n_seq;
  a.T_q = T_q;
  a.T_k = T_k;
  a.h_q = h_q;
  a.h_kv = h_kv;
  a.d = d;
  a.scale = scale;
  a.causal = causal != 0;
  a.lse = const_cast<float*>(lse);
  a.w_in = w_in;
  a.w_out = w_out;
  a.status = status_word;
  a.wait_limit_ns = wait_limit();
  rmm_status r = check_prompt(a, in);
  if (r) return r;
  if (T_q > 0 && T_k > 0 && !lse) return fail(RMM_ERR_INVALID, "lse is NULL");
  if (T_k > 0 && !w_out) return fail(RMM_ERR_INVALID, "w_out is NULL");
  if (w_in && w_in != w_out && overlap(w_in, h_kv * T_k * 4, w_out, h_kv * T_k * 4))
    return fail(RMM_ERR_INVALID, "w_in and w_out overlap without being the same");
  if (n_seq == 0 || T_k == 0) return RMM_OK;
  DeviceGuard dg;
  if ((r = bind_device(stream, dg))) return r;
  StageRange range("rmm key weights");
  const char* why = nullptr;
  const cudaError_t e = launch_attn_key_weights(a, stream, &why);
  return e == cudaSuccess ? RMM_OK : cuda_fail(e, "key weight kernel", why);
}

rmm_status rmm_kv4_store(const void* K, int64_t k_ts, int64_t k_hs, const void* V, int64_t v_ts, int64_t v_hs,
                         rmm_dtype in, const int32_t* cu, const int32_t* start, int64_t n_seq, int64_t T, int64_t h_kv,
                         int64_t d, int64_t cap, uint8_t* kc, void* ks, uint8_t* vc, void* vs, const float* w_new,
                         float* w, uint32_t* status_word, cudaStream_t stream) {
  if (n_seq < 0 || T < 0) return fail(RMM_ERR_INVALID, "negative size");
  if (!dtype_ok(in)) return fail(RMM_ERR_INVALID, "unknown input dtype");
  if (h_kv < 1) return fail(RMM_ERR_INVALID, "h_kv must be at least 1");
  if (T > kMaxI32) return fail(RMM_ERR_UNSUPPORTED, "more than 2^31 - 1 tokens");
  Kv4StoreArgs a = {};
  a.k = TokView{K, k_ts, k_hs};
  a.v = TokView{V, v_ts, v_hs};
  a.in = kind(in);
  a.cu = cu;
  a.start = start;
  a.n_seq = n_seq;
  a.T = T;
  a.h_kv = h_kv;
  a.d = d;
  a.cap = cap;
  a.c = Kv4Planes{kc, static_cast<uint16_t*>(ks), vc, static_cast<uint16_t*>(vs)};
  a.w_new = w_new;
  a.w = w;
  a.status = status_word;
  rmm_status r = check_planes(a.c, n_seq, h_kv, d, cap);
  if (r) return r;
  if (!cu && T != n_seq) return fail(RMM_ERR_INVALID, "cu may be NULL only for one token per sequence (T == n_seq)");
  if (w_new && !w) return fail(RMM_ERR_INVALID, "w_new needs w");
  if (n_seq == 0 || T == 0) return RMM_OK;
  if (!K || !V || !start) return fail(RMM_ERR_INVALID, "K, V or start is NULL");
  for (const TokView* x : {&a.k, &a.v})
    if (x->ts < 0 || x->hs < 0 || (T > 1 && x->ts < d) || (h_kv > 1 && x->hs < d))
      return fail(RMM_ERR_INVALID, "K or V layout (token or head stride) is too small");
  if (T * h_kv * 2 * (d / 8) / 256 >= kMaxI32) return fail(RMM_ERR_UNSUPPORTED, "too many tokens in one call");
  DeviceGuard dg;
  if ((r = bind_device(stream, dg))) return r;
  StageRange range("rmm kv4 store");
  const cudaError_t e = launch_kv4_store(a, stream);
  return e == cudaSuccess ? RMM_OK : cuda_fail(e, "kv4 store kernel");
}

size_t rmm_kv4_attn_workspace_size(int64_t batch, int64_t h_q, int64_t h_kv, int64_t d, int64_t cap, int weights) {
  if (batch < 0 || h_q < 1 || h_kv < 1 || d < 1 || cap < 1) return 0;
  if (batch > 65535 || h_q > 65535 || h_kv > 65535 || d > kKv4MaxD || cap > kMaxSelectK) return 0;  // refused
  return kv4_ws(batch, h_q, h_kv, d, cap, weights != 0).bytes;
}

rmm_status rmm_kv4_attn(const void* Q, int64_t q_ss, int64_t q_hs, const uint8_t* kc, const void* ks,
                        const uint8_t* vc, const void* vs, const int32_t* lens, int64_t batch, int64_t h_q,
                        int64_t h_kv, int64_t d, int64_t cap, float scale, rmm_dtype in, void* O, int64_t o_ss,
                        int64_t o_hs, rmm_dtype out, float* lse, const float* w_in, float* w_out, void* workspace,
                        size_t workspace_bytes, cudaStream_t stream) {
  if (batch < 0) return fail(RMM_ERR_INVALID, "negative size");
  if (!dtype_ok(in) || !dtype_ok(out)) return fail(RMM_ERR_INVALID, "unknown dtype");
  if (in != RMM_BF16) return fail(RMM_ERR_UNSUPPORTED, "attention takes bf16 queries");
  Kv4AttnArgs a = {};
  a.q = Q;
  a.q_ss = q_ss;
  a.q_hs = q_hs;
  a.c = Kv4Planes{const_cast<uint8_t*>(kc), static_cast<uint16_t*>(const_cast<void*>(ks)), const_cast<uint8_t*>(vc),
                  static_cast<uint16_t*>(const_cast<void*>(vs))};
  a.lens = lens;
  a.batch = batch;
  a.h_q = h_q;
  a.h_kv = h_kv;
  a.d = d;
  a.cap = cap;
  a.scale = scale;
  a.o = O;
  a.o_ss = o_ss;
  a.o_hs = o_hs;
  a.out = kind(out);
  a.lse = lse;
  a.w_in = w_in;
  a.w_out = w_out;
  a.workspace = workspace;
  rmm_status r = check_heads(h_q, h_kv, 1024);
  if (r) return r;
  if ((r = check_planes(a.c, batch, h_kv, d, cap))) return r;
  if ((r = check_scale(scale))) return r;
  if ((r = check_tokens("Q", Q, q_ss, q_hs, batch, h_q, d))) return r;
  if ((r = check_output("O", O, o_ss, o_hs, batch, h_q, d))) return r;
  if (w_in && !w_out) return fail(RMM_ERR_INVALID, "w_in needs w_out");
  if (w_in && w_in != w_out && overlap(w_in, batch * h_kv * cap * 4, w_out, batch * h_kv * cap * 4))
    return fail(RMM_ERR_INVALID, "w_in and w_out overlap without being the same");
  if (!workspace) return fail(RMM_ERR_INVALID, "workspace is NULL");
  if (!aligned(workspace, 1024)) return fail(RMM_ERR_INVALID, "workspace must be 1 KiB aligned");
  const size_t need = kv4_ws(batch, h_q, h_kv, d, cap, w_out != nullptr).bytes;
  if (workspace_bytes < need)
    return fail(RMM_ERR_INVALID, "workspace too small: %zu < %zu bytes", workspace_bytes, need);
  if (batch > 0 && !lens) return fail(RMM_ERR_INVALID, "lens is NULL");
  DeviceGuard dg;
  if ((r = bind_device(stream, dg))) return r;
  if (batch == 0) {
    const cudaError_t e = cudaMemsetAsync(workspace, 0, 4, stream);
    return e == cudaSuccess ? RMM_OK : cuda_fail(e, "cudaMemsetAsync(status)");
  }
  StageRange range("rmm kv4 attention");
  const cudaError_t e = launch_kv4_attn(a, stream);
  if (e != cudaSuccess) return cuda_fail(e, "kv4 attention kernel");
  return debug_on() ? debug_call_status(static_cast<uint32_t*>(workspace), stream) : RMM_OK;
}

size_t rmm_cache_evict_workspace_size(int64_t batch, int64_t heads, int64_t budget) {
  if (batch < 0 || heads < 1 || budget < 1) return 0;
  if (batch > kMaxI32 || heads > kMaxI32 || batch * heads > kMaxI32 || budget > kMaxSelectK) return 0;  // refused
  return size_t(1024 + up1k(batch * heads * 4) + up1k(batch * heads * budget * 4));
}

rmm_status rmm_cache_evict(const float* w, const int32_t* lens, int64_t batch, int64_t heads, int64_t cap,
                           int64_t budget, int64_t sink, int64_t recent, const rmm_cache_plane* planes,
                           int64_t n_planes, int64_t cap_out, int32_t* lens_out, int32_t* idx_out, void* workspace,
                           size_t workspace_bytes, cudaStream_t stream) {
  if (batch < 0) return fail(RMM_ERR_INVALID, "negative size");
  if (heads < 1 || cap < 1) return fail(RMM_ERR_INVALID, "heads and cap must be at least 1");
  if (cap > kMaxSelectK) return fail(RMM_ERR_UNSUPPORTED, "cap above 2^21");
  if (batch > kMaxI32 || heads > kMaxI32 || batch * heads > kMaxI32)
    return fail(RMM_ERR_UNSUPPORTED, "too many (sequence, head) pairs");
  if (budget < 1 || budget > cap_out) return fail(RMM_ERR_INVALID, "budget must be in [1, cap_out]");
  if (cap_out > kMaxSelectK) return fail(RMM_ERR_UNSUPPORTED, "cap_out above 2^21");
  if (sink < 0 || recent < 0 || sink + recent > budget)
    return fail(RMM_ERR_INVALID, "sink and recent must not be negative, nor exceed budget together");
  if (n_planes < 0 || (n_planes > 0 && !planes)) return fail(RMM_ERR_INVALID, "planes is NULL");
  if (n_planes > kMaxPlanes) return fail(RMM_ERR_UNSUPPORTED, "more than %d planes", kMaxPlanes);
  EvictArgs a = {};
  const int64_t items = batch * heads;
  for (int64_t i = 0; i < n_planes; ++i) {
    const rmm_cache_plane& p = planes[i];
    if (p.row_bytes < 4 || p.row_bytes % 4 != 0) return fail(RMM_ERR_INVALID, "row_bytes must be a multiple of 4");
    if (p.row_bytes > 8192) return fail(RMM_ERR_UNSUPPORTED, "row_bytes above 8192");
    if (batch > 0 && (!p.src || !p.dst)) return fail(RMM_ERR_INVALID, "plane %lld has a NULL pointer", (long long)i);
    if (!aligned(p.src, 4) || !aligned(p.dst, 4)) return fail(RMM_ERR_INVALID, "planes must be 4-byte aligned");
    if (p.src == p.dst && cap_out != cap)
      return fail(RMM_ERR_INVALID, "a plane moved in place keeps its capacity (cap_out == cap)");
    for (int64_t j = 0; j < n_planes; ++j) {
      const rmm_cache_plane& o = planes[j];
      const int64_t n_dst = items * cap_out * p.row_bytes;
      const bool same = i == j && p.src == p.dst;
      if ((!same && overlap(p.dst, n_dst, o.src, items * cap * o.row_bytes)) ||
          (i != j && overlap(p.dst, n_dst, o.dst, items * cap_out * o.row_bytes)))
        return fail(RMM_ERR_INVALID, "planes overlap without being the same plane moved in place");
    }
    a.plane[i] = EvictPlane{p.src, p.dst, p.row_bytes};
  }
  if (!workspace) return fail(RMM_ERR_INVALID, "workspace is NULL");
  if (!aligned(workspace, 1024)) return fail(RMM_ERR_INVALID, "workspace must be 1 KiB aligned");
  const size_t need = rmm_cache_evict_workspace_size(batch, heads, budget);
  if (workspace_bytes < need)
    return fail(RMM_ERR_INVALID, "workspace too small: %zu < %zu bytes", workspace_bytes, need);
  if (batch > 0 && (!w || !lens || !lens_out)) return fail(RMM_ERR_INVALID, "w, lens or lens_out is NULL");
  DeviceGuard dg;
  rmm_status r = bind_device(stream, dg);
  if (r) return r;
  if (batch == 0) {
    const cudaError_t ce = cudaMemsetAsync(workspace, 0, 4, stream);
    return ce == cudaSuccess ? RMM_OK : cuda_fail(ce, "cudaMemsetAsync(status)");
  }
  char* base = static_cast<char*>(workspace);
  a.w = w;
  a.lens = lens;
  a.batch = batch;
  a.heads = heads;
  a.cap = cap;
  a.cap_out = cap_out;
  a.budget = budget;
  a.sink = sink;
  a.recent = recent;
  a.n_planes = int(n_planes);
  a.lens_out = lens_out;
  a.counts = reinterpret_cast<int32_t*>(base + 1024);
  a.idx = idx_out ? idx_out : reinterpret_cast<int32_t*>(base + 1024 + up1k(items * 4));
  a.status = static_cast<uint32_t*>(workspace);
  StageRange range("rmm evict");
  const cudaError_t e = launch_evict(a, stream);
  if (e != cudaSuccess) return cuda_fail(e, "eviction kernel");
  return debug_on() ? debug_call_status(a.status, stream) : RMM_OK;
}
