// C-ABI entry points of librope_attention.so (declared in include/rope_attention.h).
// Host-side validation happens here, before anything is launched.
#include <algorithm>
#include <atomic>
#include <cstdarg>
#include <cmath>
#include <cstdio>
#include <initializer_list>
#include <string>

#include "rope_attention.h"
#include "attention.h"
#include "cache_paging.h"
#include "internal.h"
#include "kv_cache.h"
#include "row_quant.h"

namespace ra {

int device_sm_count() {
  static std::atomic<int> cached{0};
  int v = cached.load();
  if (v > 0) return v;
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    n = 148;
  cached.store(n);
  return n;
}

}  // namespace ra

namespace {

thread_local std::string g_last_error;
std::atomic<int64_t> g_wait_ns{2000000000LL};
std::atomic<int> g_stall_next{0};  // ra_test_stall_next_projection
std::atomic<int> g_stall_next_kv{0};  // ra_test_stall_next_kv_cache
std::atomic<int> g_stall_next_norm{0};  // ra_test_stall_next_norm_rope
std::atomic<int> g_stall_next_attn{0};  // ra_test_stall_next_attention
std::atomic<int> g_validate_only{0};    // ra_test_validate_only

// ra_test_validate_only: a call that passed its host checks returns here, before
// any CUDA runtime call
bool validate_only() { return g_validate_only.load() != 0; }

ra_status fail(ra_status code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
ra_status fail(ra_status code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return code;
}

ra_status ok() {
  g_last_error.clear();
  return RA_OK;
}

ra_status cuda_fail(cudaError_t e, const char* where) {
  return fail(RA_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct QkvShape {
  int64_t T, H, I;
  int32_t q_w, k_w;
  int32_t q_end, k_end;
  int32_t n_part_tiles;
  int32_t s_begin, s_end;   // Q/K columns carried as scaled fp16 between the passes
  int32_t ph_begin, ph_end; // Q/K columns finished in the projection (per-head norm)
  int32_t n_exp_blocks;     // 128-column blocks covering [0, s_end)
  int32_t part_stride, exp_stride;  // token-major row strides (16-byte multiples)
  size_t exps_offset;
  size_t workspace;
};

// which segments the norm/RoPE pass rewrites
// (across-heads norm, and RoPE whatever the norm: a per-head segment is normed in
// the projection and rotated here)
void second_pass_segments(const qkv_cte_mx_params* p, bool* do_q, bool* do_k) {
  *do_q = p->q_norm == RA_NORM_RMS_ACROSS_HEADS || p->fused_rope;
  *do_k = p->num_kv_heads > 0 && (p->k_norm == RA_NORM_RMS_ACROSS_HEADS || p->fused_rope);
}

ra_status check_params(const qkv_cte_mx_params* p, QkvShape* s) {
  if (p == nullptr) return fail(RA_ERR_INVALID_ARG, "params is NULL");
  if (p->B < 1 || p->S < 1) return fail(RA_ERR_INVALID_ARG, "B and S must be >= 1 (no empty tensors)");
  if (p->H < 128 || p->H % 128 != 0)
    return fail(RA_ERR_INVALID_ARG, "H must be a positive multiple of 128 (got %lld)",
                static_cast<long long>(p->H));
  if (p->num_heads < 1) return fail(RA_ERR_INVALID_ARG, "num_heads must be >= 1");
  if (p->num_kv_heads < 0) return fail(RA_ERR_INVALID_ARG, "num_kv_heads must be >= 0");
  if (p->head_dim < 16 || p->head_dim % 16 != 0)
    return fail(RA_ERR_INVALID_ARG, "head_dim must be a positive multiple of 16");
  if (p->q_norm != RA_NORM_NONE && p->q_norm != RA_NORM_RMS_ACROSS_HEADS && p->q_norm != RA_NORM_RMS_PER_HEAD)
    return fail(RA_ERR_INVALID_ARG, "q_norm must be an RA_NORM_* value");
  if (p->k_norm != RA_NORM_NONE && p->k_norm != RA_NORM_RMS_ACROSS_HEADS && p->k_norm != RA_NORM_RMS_PER_HEAD)
    return fail(RA_ERR_INVALID_ARG, "k_norm must be an RA_NORM_* value");
  if ((p->q_norm == RA_NORM_RMS_PER_HEAD || p->k_norm == RA_NORM_RMS_PER_HEAD) &&
      p->head_dim != 64 && p->head_dim != 128)
    return fail(RA_ERR_UNSUPPORTED, "the per-head norm is built for head_dim 64 and 128");
  if (p->k_norm != RA_NORM_NONE && p->num_kv_heads == 0)
    return fail(RA_ERR_INVALID_ARG, "k_norm needs a K segment (num_kv_heads == 0)");
  if (p->fused_rope != 0 && p->fused_rope != 1) return fail(RA_ERR_INVALID_ARG, "fused_rope must be 0 or 1");
  if (!(p->norm_eps >= 0.f) || !std::isfinite(p->norm_eps))
    return fail(RA_ERR_INVALID_ARG, "norm_eps must be finite and >= 0");
  if (p->output_layout != RA_LAYOUT_BSD && p->output_layout != RA_LAYOUT_NBSD)
    return fail(RA_ERR_INVALID_ARG, "unknown output_layout");
  const int64_t T = p->B * p->S;
  const int64_t I = static_cast<int64_t>(p->num_heads + 2 * p->num_kv_heads) * p->head_dim;
  if (T > 0x7fffffffLL || I > 0x7fffffffLL || p->H > 0x7fffffffLL || T * I > (1LL << 40))
    return fail(RA_ERR_INVALID_ARG, "problem too large for 32-bit tile coordinates");
  s->T = T;
  s->H = p->H;
  s->I = I;
  s->q_w = p->num_heads * p->head_dim;
  s->k_w = p->num_kv_heads * p->head_dim;
  s->q_end = s->q_w;
  s->k_end = s->q_w + s->k_w;
  const bool q_across = p->q_norm == RA_NORM_RMS_ACROSS_HEADS;
  const bool k_across = p->k_norm == RA_NORM_RMS_ACROSS_HEADS;
  const int32_t across_end = k_across ? s->k_end : (q_across ? s->q_end : 0);
  s->n_part_tiles = (q_across || k_across) ? (across_end + ra::kPartCols - 1) / ra::kPartCols : 0;
  // segments the second pass rewrites (across-heads norm, or RoPE without a norm) are
  // carried as scaled fp16 between the passes; per-head segments are finished in the
  // projection
  bool do_q, do_k;
  second_pass_segments(p, &do_q, &do_k);
  s->s_begin = do_q ? 0 : s->q_w;
  s->s_end = do_k ? s->k_end : s->q_w;
  if (!do_q && !do_k) s->s_begin = s->s_end = 0;
  const bool q_ph = p->q_norm == RA_NORM_RMS_PER_HEAD;
  const bool k_ph = p->num_kv_heads > 0 && p->k_norm == RA_NORM_RMS_PER_HEAD;
  s->ph_begin = q_ph ? 0 : s->q_w;
  s->ph_end = k_ph ? s->k_end : s->q_w;
  if (!q_ph && !k_ph) s->ph_begin = s->ph_end = 0;
  s->n_exp_blocks = (s->s_end + ra::kPartCols - 1) / ra::kPartCols;
  s->part_stride = (s->n_part_tiles + 1) / 2 * 2;
  s->exp_stride = (s->n_exp_blocks + 15) / 16 * 16;
  const size_t part = static_cast<size_t>(s->part_stride) * T * sizeof(float2);
  const size_t exps = static_cast<size_t>(s->exp_stride) * T;
  s->exps_offset = ra::kWorkspaceHeader + ((part + 255) / 256) * 256;
  s->workspace = s->exps_offset + ((exps + 255) / 256) * 256;
  return RA_OK;
}

ra_status check_project_inputs(const qkv_cte_mx_params* p, const uint8_t* a, const float* a_scale,
                               const void* w_packed, const float* ws, const uint16_t* bias,
                               const float* qg, const float* kg, const uint16_t* out) {
  if (!a || !a_scale || !w_packed || !out)
    return fail(RA_ERR_INVALID_ARG, "a, a_scale, w_packed and out are required");
  if (!aligned16(a) || !aligned16(out) || !aligned16(w_packed))
    return fail(RA_ERR_ALIGNMENT, "a, out and w_packed must be 16-byte aligned");
  if ((ws && !aligned16(ws)) || (bias && !aligned16(bias)))
    return fail(RA_ERR_ALIGNMENT, "weight_scales and bias must be 16-byte aligned");
  if (p->q_norm && !qg) return fail(RA_ERR_INVALID_ARG, "q_norm requires q_gamma");
  if (p->k_norm && !kg) return fail(RA_ERR_INVALID_ARG, "k_norm requires k_gamma");
  if ((qg && !aligned16(qg)) || (kg && !aligned16(kg)))
    return fail(RA_ERR_ALIGNMENT, "gammas must be 16-byte aligned");
  return RA_OK;
}

ra_status check_norm_inputs(const qkv_cte_mx_params* p, const float* cos, const float* sin,
                            const uint16_t* out) {
  if (!out) return fail(RA_ERR_INVALID_ARG, "out is required");
  if (!aligned16(out)) return fail(RA_ERR_ALIGNMENT, "out must be 16-byte aligned");
  if (p->fused_rope && (!cos || !sin))
    return fail(RA_ERR_INVALID_ARG, "fused_rope requires cos_cache and sin_cache");
  if ((cos && !aligned16(cos)) || (sin && !aligned16(sin)))
    return fail(RA_ERR_ALIGNMENT, "cos/sin caches must be 16-byte aligned");
  return RA_OK;
}

ra_status check_workspace(const void* workspace, size_t workspace_bytes, const QkvShape& s) {
  if (!workspace) return fail(RA_ERR_INVALID_ARG, "workspace is required");
  if (!aligned16(workspace)) return fail(RA_ERR_ALIGNMENT, "workspace must be 16-byte aligned");
  if (workspace_bytes < s.workspace)
    return fail(RA_ERR_WORKSPACE, "workspace too small: %zu < %zu", workspace_bytes, s.workspace);
  return RA_OK;
}

ra_status run_project(const qkv_cte_mx_params* p, const QkvShape& s, const uint8_t* a,
                      const float* a_scale, const void* w_packed, const float* ws,
                      const uint16_t* bias, const float* qg, const float* kg, uint16_t* out,
                      void* workspace, cudaStream_t st) {
  ra::ProjLaunch L{};
  L.a = a;
  L.a_scale = a_scale;
  L.w_t = static_cast<const uint8_t*>(w_packed);
  L.sf = static_cast<const uint8_t*>(w_packed) + ra::packed_sf_offset(s.H, s.I);
  L.weight_scales = ws;
  L.bias = bias;
  L.out = out;
  L.status = static_cast<int32_t*>(workspace);
  L.partials = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + ra::kWorkspaceHeader);
  L.T = s.T;
  L.H = s.H;
  L.I = s.I;
  L.q_end = s.q_end;
  L.k_end = p->num_kv_heads > 0 ? s.k_end : s.q_end;
  L.n_part_tiles = s.n_part_tiles;
  L.exps = reinterpret_cast<int8_t*>(static_cast<uint8_t*>(workspace) + s.exps_offset);
  L.n_exp_blocks = s.n_exp_blocks;
  L.part_stride = s.part_stride;
  L.exp_stride = s.exp_stride;
  L.s_begin = s.s_begin;
  L.s_end = s.s_end;
  // the gamma the epilogue folds in: across-heads segments only (the per-head
  // segments take theirs in the per-head norm)
  L.q_gamma = p->q_norm == RA_NORM_RMS_ACROSS_HEADS ? qg : nullptr;
  L.k_gamma = p->k_norm == RA_NORM_RMS_ACROSS_HEADS ? kg : nullptr;
  L.ph_begin = s.ph_begin;
  L.ph_end = s.ph_end;
  L.ph_q_gamma = p->q_norm == RA_NORM_RMS_PER_HEAD ? qg : nullptr;
  L.ph_k_gamma = p->k_norm == RA_NORM_RMS_PER_HEAD ? kg : nullptr;
  L.ph_carry = p->fused_rope;
  L.eps = p->norm_eps;
  L.wait_ns = g_wait_ns.load();
  L.stall_loads = g_stall_next.exchange(0);
  L.head_dim = p->head_dim;
  L.nbsd = p->output_layout == RA_LAYOUT_NBSD;
  const char* why = "launch failed";
  cudaError_t e = ra::launch_qkv_project(L, st, &why);
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "qkv projection: %s (%s)", why, cudaGetErrorString(e));
  return RA_OK;
}

ra_status run_norm_rope(const qkv_cte_mx_params* p, const QkvShape& s, const float* cos,
                        const float* sin, uint16_t* out, void* workspace, cudaStream_t st) {
  bool do_q, do_k;
  second_pass_segments(p, &do_q, &do_k);
  if (!do_q && !do_k) return RA_OK;
  ra::NormRopeLaunch L{};
  L.out = out;
  L.partials =
      reinterpret_cast<const float2*>(static_cast<const uint8_t*>(workspace) + ra::kWorkspaceHeader);
  L.cos = cos;
  L.sin = sin;
  L.T = s.T;
  L.I = s.I;
  L.head_dim = p->head_dim;
  L.num_q_heads = p->num_heads;
  L.num_k_heads = p->num_kv_heads;
  L.q_norm = p->q_norm == RA_NORM_RMS_ACROSS_HEADS;
  L.k_norm = p->k_norm == RA_NORM_RMS_ACROSS_HEADS;
  L.rope = p->fused_rope;
  L.do_q = do_q;
  L.do_k = do_k;
  L.n_part_tiles = s.n_part_tiles;
  L.exps = reinterpret_cast<const int8_t*>(static_cast<const uint8_t*>(workspace) + s.exps_offset);
  L.part_stride = s.part_stride;
  L.n_exp_blocks = s.n_exp_blocks;
  L.exp_stride = s.exp_stride;
  L.eps = p->norm_eps;
  L.nbsd = p->output_layout == RA_LAYOUT_NBSD;
  L.status = static_cast<int32_t*>(workspace);
  L.wait_ns = g_wait_ns.load();
  L.stall_loads = g_stall_next_norm.exchange(0);
  cudaError_t e = ra::launch_qk_norm_rope(L, st);
  if (e != cudaSuccess) return cuda_fail(e, "norm/rope launch");
  return RA_OK;
}

// ---------------------------------------------------------------- attention and the cache read
int32_t quant_kind(int32_t dtype) {
  return dtype == RA_INT8 ? ra::kQuantInt8 : dtype == RA_FP8_E4M3 ? ra::kQuantE4m3 : dtype == RA_FP8_E5M2 ? ra::kQuantE5m2 : -1;
}

// The caches of kv_rms_norm_rope_cache as a reader sees them: the checks of the
// parameters that describe them, and their row widths and types.
struct CacheShape {
  int32_t kw, vw, kq, vq;
};
ra_status check_cache(const kv_rms_norm_rope_cache_params* p, const float* k_scale, const float* v_scale,
                      const float* k_offset, const float* v_offset, CacheShape* s) {
  if (p == nullptr) return fail(RA_ERR_INVALID_ARG, "cache params is NULL");
  if (p->kv_dtype != RA_BF16 && p->kv_dtype != RA_FP16) return fail(RA_ERR_INVALID_ARG, "kv dtype must be bf16 or fp16");
  if (p->rope_size < 8 || p->rope_size % 8 != 0 || p->rope_size > 256)
    return fail(RA_ERR_INVALID_ARG, "rope_size must be a multiple of 8 in [8, 256]");
  if (p->Dkv < 8 || p->Dkv % 8 != 0 || p->Dkv > 4096 || p->Dv < 8 || p->Dv % 8 != 0 || p->Dv > 1024)
    return fail(RA_ERR_INVALID_ARG, "Dkv and Dv must be positive multiples of 8 (Dv <= 1024)");
  if (p->variant == 1) {
    if (p->N != 1) return fail(RA_ERR_INVALID_ARG, "V1 (combined kv) supports N == 1 only");
    if (p->Dv != p->Dkv - p->rope_size) return fail(RA_ERR_INVALID_ARG, "V1 needs Dv == Dkv - rope_size");
  } else if (p->variant == 2) {
    if (!(p->N == 1 || p->N == 2 || p->N == 4 || p->N == 8))
      return fail(RA_ERR_INVALID_ARG, "V2 (separate kv) supports N in {1, 2, 4, 8}");
    if (p->rope_size > p->Dkv) return fail(RA_ERR_INVALID_ARG, "rope_size exceeds Dkv");
  } else {
    return fail(RA_ERR_INVALID_ARG, "variant must be 1 or 2");
  }
  const int64_t rms = p->variant == 1 ? p->Dv : p->Dkv;
  if (rms > 1024) return fail(RA_ERR_INVALID_ARG, "rms_size must be in [8, 1024]");
  if ((k_offset && !k_scale) || (v_offset && !v_scale))
    return fail(RA_ERR_INVALID_ARG, "an offset without its scale is illegal");
  s->kq = k_scale ? quant_kind(p->k_cache_dtype) : 0;
  s->vq = v_scale ? quant_kind(p->ckv_cache_dtype) : 0;
  if (k_scale ? s->kq < 0 : p->k_cache_dtype != p->kv_dtype)
    return fail(RA_ERR_INVALID_ARG, "k_cache dtype must be int8 or fp8 with a k scale, else equal to the kv dtype");
  if (v_scale ? s->vq < 0 : p->ckv_cache_dtype != p->kv_dtype)
    return fail(RA_ERR_INVALID_ARG, "ckv_cache dtype must be int8 or fp8 with a c_kv scale, else equal to the kv dtype");
  const int32_t mode = p->cache_mode;
  if (mode == RA_CACHE_PA_NZ || mode == RA_CACHE_PA_BLK_NZ)
    return fail(RA_ERR_UNSUPPORTED, "FRACTAL_NZ cache modes are not built");
  if (mode != RA_CACHE_NORM && mode != RA_CACHE_PA && mode != RA_CACHE_PA_BNSD && mode != RA_CACHE_PA_BLK_BNSD)
    return fail(RA_ERR_INVALID_ARG, "unknown cache_mode");
  if (mode == RA_CACHE_NORM) {
    if (p->cache_seq_len < 1 || p->cache_seq_len > (1LL << 31))
      return fail(RA_ERR_INVALID_ARG, "NORM mode needs cache_seq_len in [1, 2^31]");
    if (p->B > (1LL << 40) / p->cache_seq_len) return fail(RA_ERR_INVALID_ARG, "too many cache slots");
    if (p->variant == 1 && (k_scale || v_scale))
      return fail(RA_ERR_INVALID_ARG, "V1 in NORM mode takes no quantisation parameters");
  } else {
    if (p->block_num < 1 || p->block_num > 0x7fffffffLL || p->block_size <= 1 || p->block_size > 0x7fffffffLL)
      return fail(RA_ERR_INVALID_ARG, "block_num >= 1 and block_size > 1 (both below 2^31) are required");
    if ((k_scale || v_scale) && p->block_size % 32 != 0)
      return fail(RA_ERR_INVALID_ARG, "1-byte caches need block_size %% 32 == 0");
    if ((!k_scale || !v_scale) && p->block_size % 16 != 0)
      return fail(RA_ERR_INVALID_ARG, "2-byte caches need block_size %% 16 == 0");
    if (p->block_num * p->block_size > (1LL << 40)) return fail(RA_ERR_INVALID_ARG, "too many cache slots");
  }
  if ((p->k_quant_scalar != 0 && p->k_quant_scalar != 1) || (p->c_kv_quant_scalar != 0 && p->c_kv_quant_scalar != 1))
    return fail(RA_ERR_INVALID_ARG, "k_quant_scalar and c_kv_quant_scalar must be 0 or 1");
  if (p->variant == 2 && (p->k_quant_scalar || p->c_kv_quant_scalar))
    return fail(RA_ERR_INVALID_ARG, "V2 quantisation parameters are [N, D]; the [1] form is V1 only");
  if ((p->k_quant_scalar && !k_scale) || (p->c_kv_quant_scalar && !v_scale))
    return fail(RA_ERR_INVALID_ARG, "a [1] quantisation parameter flag needs its scale");
  if ((k_scale && !aligned16(k_scale)) || (v_scale && !aligned16(v_scale)) || (k_offset && !aligned16(k_offset)) ||
      (v_offset && !aligned16(v_offset)))
    return fail(RA_ERR_ALIGNMENT, "scales and offsets must be 16-byte aligned");
  s->kw = static_cast<int32_t>(p->variant == 1 ? p->rope_size : p->Dkv);
  s->vw = static_cast<int32_t>(p->Dv);
  return RA_OK;
}

// where the scales are not at hand: a quantised dtype stands for its scale
ra_status check_cache_alone(const kv_rms_norm_rope_cache_params* p, CacheShape* s) {
  if (p == nullptr) return fail(RA_ERR_INVALID_ARG, "cache params is NULL");
  const float* given = reinterpret_cast<const float*>(uintptr_t{16});
  return check_cache(p, quant_kind(p->k_cache_dtype) > 0 ? given : nullptr, quant_kind(p->ckv_cache_dtype) > 0 ? given : nullptr,
                     nullptr, nullptr, s);
}

ra_status check_window(const attention_window* w, int32_t causal) {
  if (w->window < 1) return fail(RA_ERR_INVALID_ARG, "window must be >= 1");
  if (w->sinks < 0) return fail(RA_ERR_INVALID_ARG, "sinks must be >= 0");
  if (causal != 1) return fail(RA_ERR_INVALID_ARG, "a window needs causal = 1");
  return RA_OK;
}

ra_status check_prefix(const kv_rms_norm_rope_cache_params* c, const paged_attention_params* p, const attention_prefix* x) {
  if (x == nullptr) return fail(RA_ERR_INVALID_ARG, "prefix is NULL");
  if (c->cache_mode == RA_CACHE_NORM)
    return fail(RA_ERR_UNSUPPORTED, "NORM mode has no pages for sequences to share");
  if (x->max_prefix_len < 0 || x->max_prefix_len > ra::kMostPositions)
    return fail(RA_ERR_INVALID_ARG, "max_prefix_len must be in [0, 2^31 - 256]");
  // one call lays a prefix's tiles ahead of a sequence's own
  if (x->max_prefix_len + p->max_seq_len > ra::kMostPositions)
    return fail(RA_ERR_INVALID_ARG, "max_prefix_len + max_seq_len must be at most 2^31 - 256");
  if (x->table_entries < 1 || x->table_entries > (1LL << 31))
    return fail(RA_ERR_INVALID_ARG, "table_entries must be in [1, 2^31]");
  return RA_OK;
}

ra::PackedLaunch packed_launch(const packed_attention_params* p) {
  ra::PackedLaunch L{};
  L.B = p->B;
  L.total_q = p->total_q;
  L.total_k = p->total_k;
  L.q_ts = p->q_token_stride;
  L.q_hs = p->q_head_stride;
  L.k_ts = p->k_token_stride;
  L.k_hs = p->k_head_stride;
  L.v_ts = p->v_token_stride;
  L.v_hs = p->v_head_stride;
  L.o_ts = p->out_token_stride;
  L.o_hs = p->out_head_stride;
  L.nq = p->num_heads;
  L.nkv = p->num_kv_heads;
  L.d = p->head_dim;
  L.causal = p->causal;
  L.f16 = p->dtype == RA_FP16;
  L.scale = p->softmax_scale;
  return L;
}

bool good_scale(float s) { return std::isfinite(s) && s > 0.f; }

ra_status check_packed(const packed_attention_params* p) {
  if (p == nullptr) return fail(RA_ERR_INVALID_ARG, "params is NULL");
  if (p->B < 1 || p->total_q < 1 || p->total_k < 1)
    return fail(RA_ERR_INVALID_ARG, "B, total_q and total_k must be >= 1 (no empty tensors)");
  if (p->total_q > 0x7fffff00LL || p->total_k > 0x7fffff00LL || p->B > 0x00ffffffLL)
    return fail(RA_ERR_INVALID_ARG, "too many tokens or sequences for 32-bit tile coordinates");
  if (p->num_kv_heads < 1 || p->num_heads < 1 || p->num_heads % p->num_kv_heads != 0 || p->num_heads > 65535)
    return fail(RA_ERR_INVALID_ARG, "num_heads must be a positive multiple of num_kv_heads, at most 65535");
  if (p->head_dim < 16 || p->head_dim % 16 != 0)
    return fail(RA_ERR_INVALID_ARG, "head_dim must be a positive multiple of 16");
  if (p->head_dim > 128) return fail(RA_ERR_UNSUPPORTED, "packed_attention is built for head_dim up to 128");
  if (p->dtype != RA_BF16 && p->dtype != RA_FP16) return fail(RA_ERR_INVALID_ARG, "dtype must be bf16 or fp16");
  if (p->causal != 0 && p->causal != 1) return fail(RA_ERR_INVALID_ARG, "causal must be 0 or 1");
  if (!good_scale(p->softmax_scale)) return fail(RA_ERR_INVALID_ARG, "softmax_scale must be finite and > 0");
  const int64_t tokens[4] = {p->total_q, p->total_k, p->total_k, p->total_q};
  const int64_t heads[4] = {p->num_heads, p->num_kv_heads, p->num_kv_heads, p->num_heads};
  const int64_t ts[4] = {p->q_token_stride, p->k_token_stride, p->v_token_stride, p->out_token_stride};
  const int64_t hs[4] = {p->q_head_stride, p->k_head_stride, p->v_head_stride, p->out_head_stride};
  for (int i = 0; i < 4; ++i) {
    if (ts[i] < 0 || hs[i] < 0) return fail(RA_ERR_INVALID_ARG, "strides must not be negative");
    if (ts[i] % 8 != 0 || hs[i] % 8 != 0)
      return fail(RA_ERR_ALIGNMENT, "strides must be multiples of 8 elements (16 bytes)");
    if ((tokens[i] > 1 && ts[i] == 0) || (heads[i] > 1 && hs[i] == 0))
      return fail(RA_ERR_INVALID_ARG, "an axis of more than one element needs a stride");
    if ((tokens[i] > 1 && ts[i] >= (1LL << 39) / tokens[i]) || (heads[i] > 1 && hs[i] >= (1LL << 39) / heads[i]))
      return fail(RA_ERR_INVALID_ARG, "a stride reaches past 2^40 bytes");
  }
  const int64_t d = p->head_dim, to = p->out_token_stride, ho = p->out_head_stride;
  const bool apart = (p->num_heads == 1 || ho >= d) && (p->total_q == 1 || to >= d) &&
                     (p->num_heads == 1 || p->total_q == 1 || to >= (p->num_heads - 1) * ho + d ||
                      ho >= (p->total_q - 1) * to + d);
  if (!apart) return fail(RA_ERR_INVALID_ARG, "out strides put two elements in one place");
  return RA_OK;
}

ra_status check_attn_workspace(const void* workspace, size_t have, size_t need) {
  if (!workspace) return fail(RA_ERR_INVALID_ARG, "workspace is required");
  if (!aligned16(workspace)) return fail(RA_ERR_ALIGNMENT, "workspace must be 16-byte aligned");
  if (have < need) return fail(RA_ERR_WORKSPACE, "workspace too small: %zu < %zu", have, need);
  return RA_OK;
}

ra_status check_paged(const kv_rms_norm_rope_cache_params* c, const paged_attention_params* p, const CacheShape& s) {
  if (p == nullptr) return fail(RA_ERR_INVALID_ARG, "params is NULL");
  if (p->B < 1 || p->total_q < 1) return fail(RA_ERR_INVALID_ARG, "B and total_q must be >= 1 (no empty tensors)");
  if (p->num_heads < 1 || p->num_heads % c->N != 0)
    return fail(RA_ERR_INVALID_ARG, "num_heads must be a positive multiple of the cache's N");
  if (p->B > 0x00ffffffLL || p->total_q > 0x7fffffffLL || p->total_q * p->num_heads > 0x7fffffffLL)
    return fail(RA_ERR_INVALID_ARG, "too many sequences or query rows (total_q * num_heads must stay below 2^31)");
  if (p->causal != 0 && p->causal != 1) return fail(RA_ERR_INVALID_ARG, "causal must be 0 or 1");
  if (p->reserved != 0) return fail(RA_ERR_INVALID_ARG, "reserved must be 0");
  if (!good_scale(p->softmax_scale)) return fail(RA_ERR_INVALID_ARG, "softmax_scale must be finite and > 0");
  if (p->max_seq_len < 0 || p->max_seq_len > 0x7fffff00LL)
    return fail(RA_ERR_INVALID_ARG, "max_seq_len must be in [0, 2^31 - 256]");
  if (c->cache_mode == RA_CACHE_NORM) {
    if (c->B != p->B) return fail(RA_ERR_INVALID_ARG, "NORM mode: the cache's B must equal the call's B");
    if (p->block_table_stride != 0) return fail(RA_ERR_INVALID_ARG, "NORM mode takes no block table");
  } else if (p->block_table_stride < 1 || p->block_table_stride > (1LL << 31)) {
    return fail(RA_ERR_INVALID_ARG, "block_table_stride must be in [1, 2^31]");
  }
  if ((c->cache_mode == RA_CACHE_NORM ? p->B * c->cache_seq_len : c->block_num * c->block_size) * c->N > 0x7fffffffLL)
    return fail(RA_ERR_UNSUPPORTED, "paged_attention addresses cache rows with 31 bits (slots * N)");
  if (c->variant == 1 ? (c->Dv > 512 || c->Dv % 64 != 0 || c->rope_size > 64 || c->rope_size % 16 != 0)
                      : (c->Dkv > 256 || c->Dkv % 16 != 0 || c->Dv > 256 || c->Dv % 16 != 0))
    return fail(RA_ERR_UNSUPPORTED,
                "paged_attention is built for V1 with Dv a multiple of 64 up to 512 and rope_size 16..64, and V2 with "
                "Dkv and Dv multiples of 16 up to 256");
  (void)s;
  return RA_OK;
}

ra::PagedLaunch paged_launch(const kv_rms_norm_rope_cache_params* c, const paged_attention_params* p,
                             const CacheShape& s) {
  ra::PagedLaunch L{};
  L.B = p->B;
  L.total_q = p->total_q;
  L.N = c->N;
  L.heads = p->num_heads;
  L.Dkv = static_cast<int32_t>(c->Dkv);
  L.Dv = static_cast<int32_t>(c->Dv);
  L.R = c->rope_size;
  L.variant = c->variant;
  L.mode = c->cache_mode;
  L.f16 = c->kv_dtype == RA_FP16;
  L.kq = s.kq;
  L.vq = s.vq;
  L.k_scalar = c->k_quant_scalar;
  L.v_scalar = c->c_kv_quant_scalar;
  L.causal = p->causal;
  L.scale = p->softmax_scale;
  L.max_seq_len = p->max_seq_len;
  L.block_num = c->block_num;
  L.block_size = c->cache_mode == RA_CACHE_NORM ? 1 : c->block_size;
  L.cache_seq = c->cache_seq_len;
  L.table_stride = p->block_table_stride;
  L.cu_step = 1;
  return L;
}

// the call over the prefix: the tokens of all sequences as one's
ra::PagedLaunch over_prefix(const ra::PagedLaunch& L, const attention_prefix* x) {
  ra::PagedLaunch P = L;
  P.cu_step = static_cast<int32_t>(L.B);
  P.B = 1;
  P.causal = 0;
  P.max_seq_len = x->max_prefix_len;
  P.table_stride = x->table_entries;
  return P;
}

// the one call with the prefix ahead of every sequence's own positions
ra::PagedLaunch behind_prefix(const ra::PagedLaunch& L, const attention_prefix* x, const int32_t* len, const int32_t* table) {
  ra::PagedLaunch C = L;
  C.prefix_len = len;
  C.prefix_table = table;
  C.prefix_entries = x->table_entries;
  C.max_prefix_len = x->max_prefix_len;
  return C;
}

// The workspace of paged_prefix_attention: the header and the parts of the call over the prefix, the
// other call's, the fp32 rows that go from one to the other, and their statistics; or the one
// call's parts.
struct PrefixPlan {
  size_t partials, rows, stats, bytes;
};
size_t next_256(size_t n) { return (n + 255) / 256 * 256; }
uint8_t* aligned_in(uint8_t* ws, size_t at) {  // the step from any 16 bytes to the next 32 has room
  return ws + at + (0 - reinterpret_cast<uintptr_t>(ws + at)) % 32;
}
PrefixPlan prefix_plan(const ra::PagedLaunch& L, const attention_prefix* x) {
  const size_t rows = static_cast<size_t>(L.total_q) * L.heads;
  static const int32_t given = 0;              // sizes alone: the pointers are not looked at
  PrefixPlan p;
  p.partials = next_256(ra::paged_attention_workspace(over_prefix(L, x)));
  p.rows = std::max(p.partials + next_256(ra::paged_attention_workspace(L) - ra::kAttnHeader),
                    next_256(ra::paged_attention_workspace(behind_prefix(L, x, &given, &given))));
  p.stats = p.rows + next_256(rows * L.Dv * sizeof(float) + 32);
  p.bytes = p.stats + next_256(rows * sizeof(float4) + 32);
  return p;
}
}  // namespace

namespace ra {
void set_last_error(int code, const char* where, const char* what) {
  fail(static_cast<ra_status>(code), "%s: %s", where, what);
}

ra_status qkv_cte_mx_on_library_workspace(const qkv_cte_mx_params* p, const uint8_t* a,
                                          const float* a_scale, const void* w_packed,
                                          const float* weight_scales, const uint16_t* bias,
                                          const float* cos_cache, const float* sin_cache,
                                          const float* q_gamma, const float* k_gamma, uint16_t* out,
                                          size_t capacity, ra_status (*get_workspace)(void**),
                                          void* stream) {
  QkvShape s;
  ra_status st = check_params(p, &s);
  if (st != RA_OK) return st;
  if (s.workspace > capacity)
    return fail(RA_ERR_WORKSPACE,
                "qkv_cte_mx_noalloc: this call needs %zu bytes of scratch; the static workspace holds %zu",
                s.workspace, capacity);
  st = check_project_inputs(p, a, a_scale, w_packed, weight_scales, bias, q_gamma, k_gamma, out);
  if (st == RA_OK) st = check_norm_inputs(p, cos_cache, sin_cache, out);
  if (st != RA_OK) return st;
  if (validate_only()) return ok();
  void* ws = nullptr;
  st = get_workspace(&ws);
  if (st != RA_OK) return st;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  // the only scratch that must start at zero is the status word: the partial sums
  // and the exponents are written by the projection before the second pass reads them
  const cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(int32_t), cs);
  if (e != cudaSuccess) return cuda_fail(e, "clearing the static workspace status word");
  st = run_project(p, s, a, a_scale, w_packed, weight_scales, bias, q_gamma, k_gamma, out, ws, cs);
  if (st != RA_OK) return st;
  st = run_norm_rope(p, s, cos_cache, sin_cache, out, ws, cs);
  return st == RA_OK ? ok() : st;
}
}  // namespace ra

extern "C" {

const char* ra_last_error(void) { return g_last_error.c_str(); }

int32_t ra_abi_version(void) { return 9; }

void ra_set_wait_timeout_ns(int64_t ns) { g_wait_ns.store(ns < 1000 ? 1000 : ns); }

void ra_test_stall_next_projection(void) { g_stall_next.store(1); }

void ra_test_stall_next_kv_cache(void) { g_stall_next_kv.store(1); }

void ra_test_stall_next_norm_rope(void) { g_stall_next_norm.store(1); }

void ra_test_validate_only(int32_t on) { g_validate_only.store(on != 0 ? 1 : 0); }

ra_status qkv_cte_mx_packed_weight_bytes(int64_t H, int64_t I, size_t* bytes) {
  if (!bytes) return fail(RA_ERR_INVALID_ARG, "bytes is NULL");
  if (H < 128 || H % 128 != 0) return fail(RA_ERR_INVALID_ARG, "H must be a positive multiple of 128");
  if (I < 16 || I % 16 != 0) return fail(RA_ERR_INVALID_ARG, "I must be a positive multiple of 16");
  *bytes = ra::packed_weight_bytes(H, I);
  return ok();
}

ra_status qkv_cte_mx_pack_weight(const uint8_t* w, const uint8_t* w_block_exp, int64_t H, int64_t I,
                                 void* packed, size_t packed_bytes, void* stream) {
  size_t need = 0;
  ra_status st = qkv_cte_mx_packed_weight_bytes(H, I, &need);
  if (st != RA_OK) return st;
  if (!w || !w_block_exp || !packed) return fail(RA_ERR_INVALID_ARG, "w, w_block_exp and packed are required");
  if (!aligned16(packed)) return fail(RA_ERR_ALIGNMENT, "packed must be 16-byte aligned");
  if (packed_bytes < need) return fail(RA_ERR_WORKSPACE, "packed buffer too small: %zu < %zu", packed_bytes, need);
  if (H > 0x7fffffffLL || I > 0x7fffffffLL) return fail(RA_ERR_INVALID_ARG, "H or I too large");
  if (validate_only()) return ok();
  cudaError_t e = ra::launch_pack_weight(w, w_block_exp, H, I, static_cast<uint8_t*>(packed),
                                         static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "pack_weight launch");
  return ok();
}

ra_status qkv_cte_mx_workspace_bytes(const qkv_cte_mx_params* p, size_t* bytes) {
  if (!bytes) return fail(RA_ERR_INVALID_ARG, "bytes is NULL");
  QkvShape s;
  ra_status st = check_params(p, &s);
  if (st != RA_OK) return st;
  *bytes = s.workspace;
  return ok();
}

ra_status qkv_cte_mx_project(const qkv_cte_mx_params* p, const uint8_t* a, const float* a_scale,
                             const void* w_packed, const float* weight_scales, const uint16_t* bias,
                             const float* q_gamma, const float* k_gamma, uint16_t* out, void* workspace,
                             size_t workspace_bytes, void* stream) {
  QkvShape s;
  ra_status st = check_params(p, &s);
  if (st == RA_OK) st = check_project_inputs(p, a, a_scale, w_packed, weight_scales, bias, q_gamma, k_gamma, out);
  if (st == RA_OK) st = check_workspace(workspace, workspace_bytes, s);
  if (st != RA_OK) return st;
  if (validate_only()) return ok();
  st = run_project(p, s, a, a_scale, w_packed, weight_scales, bias, q_gamma,
                   k_gamma, out, workspace, static_cast<cudaStream_t>(stream));
  return st == RA_OK ? ok() : st;
}

ra_status qkv_cte_mx_norm_rope(const qkv_cte_mx_params* p, const float* cos_cache,
                               const float* sin_cache, uint16_t* out, void* workspace,
                               size_t workspace_bytes, void* stream) {
  QkvShape s;
  ra_status st = check_params(p, &s);
  if (st == RA_OK) st = check_norm_inputs(p, cos_cache, sin_cache, out);
  if (st == RA_OK) st = check_workspace(workspace, workspace_bytes, s);
  if (st != RA_OK) return st;
  if (validate_only()) return ok();
  st = run_norm_rope(p, s, cos_cache, sin_cache, out, workspace, static_cast<cudaStream_t>(stream));
  return st == RA_OK ? ok() : st;
}

ra_status qkv_cte_mx(const qkv_cte_mx_params* p, const uint8_t* a, const float* a_scale,
                     const void* w_packed, const float* weight_scales, const uint16_t* bias,
                     const float* cos_cache, const float* sin_cache, const float* q_gamma,
                     const float* k_gamma, uint16_t* out, void* workspace, size_t workspace_bytes,
                     void* stream) {
  QkvShape s;
  ra_status st = check_params(p, &s);
  if (st == RA_OK) st = check_project_inputs(p, a, a_scale, w_packed, weight_scales, bias, q_gamma, k_gamma, out);
  if (st == RA_OK) st = check_norm_inputs(p, cos_cache, sin_cache, out);
  if (st == RA_OK) st = check_workspace(workspace, workspace_bytes, s);
  if (st != RA_OK) return st;
  if (validate_only()) return ok();
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  st = run_project(p, s, a, a_scale, w_packed, weight_scales, bias, q_gamma,
                   k_gamma, out, workspace, cs);
  if (st != RA_OK) return st;
  st = run_norm_rope(p, s, cos_cache, sin_cache, out, workspace, cs);
  return st == RA_OK ? ok() : st;
}

ra_status qkv_cte_mx_status(void* workspace, void* stream, int32_t* device_status) {
  if (!device_status) return fail(RA_ERR_INVALID_ARG, "device_status is required");
  if (validate_only()) {
    *device_status = 0;
    return ok();
  }
  if (!workspace) {  // the static workspace of qkv_cte_mx_noalloc on the current device
    const ra_status st = ra::noalloc_workspace(&workspace);
    if (st != RA_OK) return st;
  }
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  int32_t v = 0;
  cudaError_t e = cudaMemcpyAsync(&v, workspace, sizeof(v), cudaMemcpyDeviceToHost, cs);
  if (e == cudaSuccess) e = cudaStreamSynchronize(cs);
  if (e == cudaSuccess && v != 0) e = cudaMemsetAsync(workspace, 0, sizeof(int32_t), cs);
  if (e == cudaSuccess) e = cudaStreamSynchronize(cs);
  if (e != cudaSuccess) return cuda_fail(e, "status read");
  *device_status = v;
  if (v != 0) return fail(RA_ERR_TIMEOUT, "a projection pipeline wait ran out of time (status %d)", v);
  return ok();
}

static ra_status row_quantize_common(const uint16_t* x, int64_t T, int64_t H, uint8_t* codes,
                                     float* scale, bool packed, void* stream) {
  if (!x || !codes || (!packed && !scale)) return fail(RA_ERR_INVALID_ARG, "x, codes (and scale) are required");
  if (T < 1 || H < 8 || H % 8 != 0 || H > (int64_t(1) << 30))
    return fail(RA_ERR_INVALID_ARG, "T >= 1 and H a positive multiple of 8 are required");
  if (!aligned16(x)) return fail(RA_ERR_ALIGNMENT, "x must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(codes) & (packed ? 3u : 7u)) != 0 ||
      (scale && (reinterpret_cast<uintptr_t>(scale) & 3u) != 0))
    return fail(RA_ERR_ALIGNMENT, packed ? "packed must be 4-byte aligned"
                                         : "codes must be 8-byte and scale 4-byte aligned");
  if (validate_only()) return ok();
  cudaError_t e = ra::launch_row_quantize(x, T, H, codes, scale, packed, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "row_quantize launch");
  return ok();
}

ra_status row_quantize_e4m3(const uint16_t* x, int64_t T, int64_t H, uint8_t* codes, float* scale,
                            void* stream) {
  return row_quantize_common(x, T, H, codes, scale, false, stream);
}

ra_status row_quantize_e4m3_packed(const uint16_t* x, int64_t T, int64_t H, uint8_t* packed,
                                   void* stream) {
  return row_quantize_common(x, T, H, packed, nullptr, true, stream);
}

ra_status kv_rms_norm_rope_cache(const kv_rms_norm_rope_cache_params* p, const uint16_t* kv,
                                 const uint16_t* gamma, const uint16_t* cos, const uint16_t* sin,
                                 const int64_t* index, void* k_cache, void* ckv_cache,
                                 const float* k_rope_scale, const float* c_kv_scale,
                                 const float* k_rope_offset, const float* c_kv_offset,
                                 const uint16_t* v_optional, uint16_t* k_rope, uint16_t* c_kv,
                                 int32_t* dev_error_count, void* stream) {
  if (p == nullptr) return fail(RA_ERR_INVALID_ARG, "params is NULL");
  if (!kv || !gamma || !cos || !sin || !index || !k_cache || !ckv_cache)
    return fail(RA_ERR_INVALID_ARG, "kv, gamma, cos, sin, index, k_cache and ckv_cache are required");
  if (p->B < 1 || p->N < 1 || p->S < 1 || p->Dkv < 1)
    return fail(RA_ERR_INVALID_ARG, "empty tensors are not supported");
  if (p->kv_dtype != RA_BF16 && p->kv_dtype != RA_FP16)
    return fail(RA_ERR_INVALID_ARG, "kv dtype must be bf16 or fp16");
  const int64_t R = p->rope_size;
  if (R < 8 || R % 8 != 0 || R > 256)
    return fail(RA_ERR_INVALID_ARG, "rope_size must be even; this build needs a multiple of 8 in [8, 256]");
  if (p->Dkv % 8 != 0 || p->Dv % 8 != 0 || p->Dv < 8)
    return fail(RA_ERR_INVALID_ARG, "Dkv and Dv must be positive multiples of 8");
  int64_t rms = 0;
  if (p->variant == 1) {
    if (p->N != 1) return fail(RA_ERR_INVALID_ARG, "V1 (combined kv) supports N == 1 only");
    if (v_optional) return fail(RA_ERR_INVALID_ARG, "v_optional must be NULL in V1");
    if (p->Dv != p->Dkv - R) return fail(RA_ERR_INVALID_ARG, "V1 needs Dv == Dkv - rope_size");
    rms = p->Dv;
  } else if (p->variant == 2) {
    if (!(p->N == 1 || p->N == 2 || p->N == 4 || p->N == 8))
      return fail(RA_ERR_INVALID_ARG, "V2 (separate kv) supports N in {1, 2, 4, 8}");
    if (!v_optional) return fail(RA_ERR_INVALID_ARG, "V2 needs v_optional");
    if (R > p->Dkv) return fail(RA_ERR_INVALID_ARG, "rope_size exceeds Dkv");
    if (p->Dv > 1024) return fail(RA_ERR_INVALID_ARG, "V2 needs Dv <= 1024 in this build");
    rms = p->Dkv;
  } else {
    return fail(RA_ERR_INVALID_ARG, "variant must be 1 or 2");
  }
  if (rms < 8 || rms > 1024) return fail(RA_ERR_INVALID_ARG, "rms_size must be in [8, 1024]");
  if ((k_rope_offset && !k_rope_scale) || (c_kv_offset && !c_kv_scale))
    return fail(RA_ERR_INVALID_ARG, "an offset without its scale is illegal");
  const bool qk = k_rope_scale != nullptr, qv = c_kv_scale != nullptr;
  auto quant_type = [](int32_t d) -> int32_t {
    return d == RA_INT8 ? ra::kQuantInt8 : d == RA_FP8_E4M3 ? ra::kQuantE4m3 : d == RA_FP8_E5M2 ? ra::kQuantE5m2 : -1;
  };
  const int32_t kq = qk ? quant_type(p->k_cache_dtype) : 0;
  const int32_t vq = qv ? quant_type(p->ckv_cache_dtype) : 0;
  if (qk ? kq < 0 : p->k_cache_dtype != p->kv_dtype)
    return fail(RA_ERR_INVALID_ARG, "k_cache dtype must be int8 or fp8 with a k scale, else equal to the kv dtype");
  if (qv ? vq < 0 : p->ckv_cache_dtype != p->kv_dtype)
    return fail(RA_ERR_INVALID_ARG, "ckv_cache dtype must be int8 or fp8 with a c_kv scale, else equal to the kv dtype");
  const int32_t mode = p->cache_mode;
  if (mode == RA_CACHE_PA_NZ || mode == RA_CACHE_PA_BLK_NZ)
    return fail(RA_ERR_UNSUPPORTED, "FRACTAL_NZ cache modes are not built");
  if (mode != RA_CACHE_NORM && mode != RA_CACHE_PA && mode != RA_CACHE_PA_BNSD && mode != RA_CACHE_PA_BLK_BNSD)
    return fail(RA_ERR_INVALID_ARG, "unknown cache_mode");
  if (mode == RA_CACHE_NORM) {
    if (p->cache_seq_len < p->S) return fail(RA_ERR_INVALID_ARG, "NORM mode needs cache_seq_len >= S");
    if (p->variant == 1 && (qk || qv))
      return fail(RA_ERR_INVALID_ARG, "V1 in NORM mode takes no quantisation parameters");
  } else {
    if (p->block_num < 1 || p->block_size <= 1)
      return fail(RA_ERR_INVALID_ARG, "block_num >= 1 and block_size > 1 are required");
    if ((qk || qv) && p->block_size % 32 != 0)
      return fail(RA_ERR_INVALID_ARG, "1-byte caches need block_size %% 32 == 0");
    if ((!qk || !qv) && p->block_size % 16 != 0)
      return fail(RA_ERR_INVALID_ARG, "2-byte caches need block_size %% 16 == 0");
  }
  if ((p->k_quant_scalar != 0 && p->k_quant_scalar != 1) || (p->c_kv_quant_scalar != 0 && p->c_kv_quant_scalar != 1))
    return fail(RA_ERR_INVALID_ARG, "k_quant_scalar and c_kv_quant_scalar must be 0 or 1");
  if (p->variant == 2 && (p->k_quant_scalar || p->c_kv_quant_scalar))
    return fail(RA_ERR_INVALID_ARG, "V2 quantisation parameters are [N, D]; the [1] form is V1 only");
  if ((p->k_quant_scalar && !qk) || (p->c_kv_quant_scalar && !qv))
    return fail(RA_ERR_INVALID_ARG, "a [1] quantisation parameter flag needs its scale");
  if (p->rope_s_broadcast != 0 && p->rope_s_broadcast != 1)
    return fail(RA_ERR_INVALID_ARG, "rope_s_broadcast must be 0 or 1");
  if (!(p->epsilon >= 0.f) || !std::isfinite(p->epsilon))
    return fail(RA_ERR_INVALID_ARG, "epsilon must be finite and >= 0");
  const bool outputs = p->is_output_kv && (mode != RA_CACHE_NORM || (p->variant == 2 && (qk || qv)));
  if (outputs && (!k_rope || !c_kv))
    return fail(RA_ERR_INVALID_ARG, "is_output_kv requires k_rope and c_kv");
  if (!aligned16(kv) || !aligned16(gamma) || !aligned16(cos) || !aligned16(sin) ||
      !aligned16(k_cache) || !aligned16(ckv_cache) || (v_optional && !aligned16(v_optional)) ||
      (k_rope && !aligned16(k_rope)) || (c_kv && !aligned16(c_kv)) ||
      (k_rope_scale && !aligned16(k_rope_scale)) || (c_kv_scale && !aligned16(c_kv_scale)) ||
      (k_rope_offset && !aligned16(k_rope_offset)) || (c_kv_offset && !aligned16(c_kv_offset)) ||
      (reinterpret_cast<uintptr_t>(index) & 7u))
    return fail(RA_ERR_ALIGNMENT, "tensor pointers must be 16-byte aligned (index 8-byte)");
  if (p->B * p->N * p->S > (1LL << 40)) return fail(RA_ERR_INVALID_ARG, "too many rows");
  if (mode == RA_CACHE_NORM && p->cache_seq_len > (1LL << 31)) return fail(RA_ERR_INVALID_ARG, "cache_seq_len too large");
  if (p->S > (1LL << 31)) return fail(RA_ERR_INVALID_ARG, "S too large");
  if (validate_only()) return ok();

  ra::KvLaunch L{};
  L.kv = kv;
  L.gamma = gamma;
  L.cos = cos;
  L.sin = sin;
  L.index = index;
  L.k_cache = k_cache;
  L.ckv_cache = ckv_cache;
  L.k_scale = k_rope_scale;
  L.k_offset = k_rope_offset;
  L.v_scale = c_kv_scale;
  L.v_offset = c_kv_offset;
  L.v = v_optional;
  L.k_rope = k_rope;
  L.c_kv = c_kv;
  L.err_count = dev_error_count;
  L.B = p->B;
  L.N = p->N;
  L.S = p->S;
  L.Dkv = p->Dkv;
  L.Dv = p->Dv;
  L.R = p->rope_size;
  L.variant = p->variant;
  L.mode = p->cache_mode;
  L.block_num = p->block_num;
  L.block_size = p->block_size;
  L.eps = p->epsilon;
  L.out_kv = outputs;
  L.f16 = p->kv_dtype == RA_FP16;
  L.kq = kq;
  L.vq = vq;
  L.rope_bcast = p->rope_s_broadcast;
  L.k_scalar = p->k_quant_scalar;
  L.v_scalar = p->c_kv_quant_scalar;
  L.cache_seq = mode == RA_CACHE_NORM ? p->cache_seq_len : 0;
  L.wait_ns = g_wait_ns.load();
  L.stall_loads = g_stall_next_kv.exchange(0);
  L.status = ra::kv_status_word();
  cudaError_t e = ra::launch_kv_rms_norm_rope_cache(L, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kv_rms_norm_rope_cache launch");
  return ok();
}

ra_status kv_rms_norm_rope_cache_status(void* stream, int32_t* device_status) {
  if (!device_status) return fail(RA_ERR_INVALID_ARG, "device_status is required");
  if (validate_only()) {
    *device_status = 0;
    return ok();
  }
  int32_t* word = ra::kv_status_word();
  if (!word) return fail(RA_ERR_CUDA, "the KV status word cannot be found on this device");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int32_t v = 0;
  cudaError_t e = cudaMemcpyAsync(&v, word, sizeof(v), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && v != 0) e = cudaMemsetAsync(word, 0, sizeof(v), st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(e, "KV status read");
  *device_status = v;
  if (v != 0) return fail(RA_ERR_TIMEOUT, "a KV cache pipeline wait ran out of time (status %d)", v);
  return ok();
}

void ra_test_stall_next_attention(void) { g_stall_next_attn.store(1); }

ra_status packed_attention_workspace_bytes(const packed_attention_params* p, size_t* bytes) {
  if (!bytes) return fail(RA_ERR_INVALID_ARG, "bytes is NULL");
  const ra_status st = check_packed(p);
  if (st != RA_OK) return st;
  *bytes = ra::packed_attention_workspace(packed_launch(p));
  return ok();
}

// packed_attention, or with `w` packed_window_attention
static ra_status packed_call(const packed_attention_params* p, const attention_window* w, const uint16_t* q, const uint16_t* k,
                             const uint16_t* v, uint16_t* out, float* lse, const int32_t* cu_seqlens_q,
                             const int32_t* cu_seqlens_k, void* workspace, size_t workspace_bytes, void* stream) {
  ra_status st = check_packed(p);
  if (st == RA_OK && w) st = check_window(w, p->causal);
  if (st != RA_OK) return st;
  if (!q || !k || !v || !out) return fail(RA_ERR_INVALID_ARG, "q, k, v and out are required");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out))
    return fail(RA_ERR_ALIGNMENT, "q, k, v and out must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(lse) & 3u) || (reinterpret_cast<uintptr_t>(cu_seqlens_q) & 3u) ||
      (reinterpret_cast<uintptr_t>(cu_seqlens_k) & 3u))
    return fail(RA_ERR_ALIGNMENT, "lse and cu_seqlens must be 4-byte aligned");
  if (!cu_seqlens_q && p->total_q % p->B != 0)
    return fail(RA_ERR_INVALID_ARG, "without cu_seqlens_q, total_q must be a multiple of B");
  if (!cu_seqlens_k && p->total_k % p->B != 0)
    return fail(RA_ERR_INVALID_ARG, "without cu_seqlens_k, total_k must be a multiple of B");
  ra::PackedLaunch L = packed_launch(p);
  st = check_attn_workspace(workspace, workspace_bytes, ra::packed_attention_workspace(L));
  if (st != RA_OK) return st;
  if (validate_only()) return ok();
  L.q = q;
  L.k = k;
  L.v = v;
  L.out = out;
  L.lse = lse;
  L.cu_q = cu_seqlens_q;
  L.cu_k = cu_seqlens_k;
  L.status = static_cast<int32_t*>(workspace);
  L.partials = static_cast<uint8_t*>(workspace) + ra::kAttnHeader;
  L.wait_ns = g_wait_ns.load();
  L.stall_loads = g_stall_next_attn.exchange(0);
  const char* why = "launch failed";
  if (w) {
    L.window = w->window;
    L.sinks = w->sinks;
  }
  const cudaError_t e = w ? ra::launch_packed_window(L, static_cast<cudaStream_t>(stream), &why)
                          : ra::launch_packed_attention(L, static_cast<cudaStream_t>(stream), &why);
  if (e != cudaSuccess)
    return fail(RA_ERR_CUDA, "%s: %s (%s)", w ? "packed_window_attention" : "packed_attention", why, cudaGetErrorString(e));
  return ok();
}

ra_status packed_attention(const packed_attention_params* p, const uint16_t* q, const uint16_t* k,
                           const uint16_t* v, uint16_t* out, float* lse, const int32_t* cu_seqlens_q,
                           const int32_t* cu_seqlens_k, void* workspace, size_t workspace_bytes, void* stream) {
  return packed_call(p, nullptr, q, k, v, out, lse, cu_seqlens_q, cu_seqlens_k, workspace, workspace_bytes, stream);
}

ra_status packed_window_attention(const packed_attention_params* p, const attention_window* window, const uint16_t* q,
                                  const uint16_t* k, const uint16_t* v, uint16_t* out, float* lse,
                                  const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  if (!window) return fail(RA_ERR_INVALID_ARG, "window is NULL");
  return packed_call(p, window, q, k, v, out, lse, cu_seqlens_q, cu_seqlens_k, workspace, workspace_bytes, stream);
}

ra_status paged_attention_workspace_bytes(const kv_rms_norm_rope_cache_params* cache,
                                          const paged_attention_params* p, size_t* bytes) {
  if (!bytes) return fail(RA_ERR_INVALID_ARG, "bytes is NULL");
  CacheShape s;
  ra_status st = check_cache_alone(cache, &s);
  if (st == RA_OK) st = check_paged(cache, p, s);
  if (st != RA_OK) return st;
  *bytes = ra::paged_attention_workspace(paged_launch(cache, p, s));
  return ok();
}

// paged_attention; with `w` paged_window_attention, with `x` and its two tensors paged_prefix_attention
static ra_status paged_call(const kv_rms_norm_rope_cache_params* cache, const paged_attention_params* p,
                            const attention_window* w, const attention_prefix* x, const int32_t* prefix_len,
                            const int32_t* prefix_table, const uint16_t* q, const void* k_cache, const void* ckv_cache,
                            const int32_t* seq_lens, const int32_t* block_table, const int32_t* cu_seqlens_q,
                            const float* k_rope_scale, const float* c_kv_scale, const float* k_rope_offset,
                            const float* c_kv_offset, uint16_t* out, float* lse, int32_t* dev_error_count,
                            void* workspace, size_t workspace_bytes, void* stream) {
  CacheShape s;
  ra_status st = check_cache(cache, k_rope_scale, c_kv_scale, k_rope_offset, c_kv_offset, &s);
  if (st == RA_OK) st = check_paged(cache, p, s);
  if (st == RA_OK && w) st = check_window(w, p->causal);
  if (st == RA_OK && x) st = check_prefix(cache, p, x);
  if (st != RA_OK) return st;
  if (!q || !k_cache || !ckv_cache || !seq_lens || !out)
    return fail(RA_ERR_INVALID_ARG, "q, k_cache, ckv_cache, seq_lens and out are required");
  if (x && (!prefix_len || !prefix_table)) return fail(RA_ERR_INVALID_ARG, "prefix_len and prefix_table are required");
  if ((cache->cache_mode == RA_CACHE_NORM) != (block_table == nullptr))
    return fail(RA_ERR_INVALID_ARG, "the PA modes need a block_table, NORM mode takes none");
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(ckv_cache) || !aligned16(out))
    return fail(RA_ERR_ALIGNMENT, "q, out and the caches must be 16-byte aligned");
  if (((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(seq_lens) |
        reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(cu_seqlens_q) |
        reinterpret_cast<uintptr_t>(dev_error_count) | reinterpret_cast<uintptr_t>(prefix_len) |
        reinterpret_cast<uintptr_t>(prefix_table)) & 3u) != 0)
    return fail(RA_ERR_ALIGNMENT, "lse, lengths, block tables, cu_seqlens_q and dev_error_count must be 4-byte aligned");
  if (!cu_seqlens_q && p->total_q % p->B != 0)
    return fail(RA_ERR_INVALID_ARG, "without cu_seqlens_q, total_q must be a multiple of B");
  ra::PagedLaunch L = paged_launch(cache, p, s);
  PrefixPlan plan{};
  if (x) plan = prefix_plan(L, x);
  st = check_attn_workspace(workspace, workspace_bytes, x ? plan.bytes : ra::paged_attention_workspace(L));
  if (st != RA_OK) return st;
  if (validate_only()) return ok();
  L.q = q;
  L.out = out;
  L.lse = lse;
  L.shifts = lse != nullptr;
  L.k_cache = k_cache;
  L.v_cache = ckv_cache;
  L.k_scale = k_rope_scale;
  L.k_offset = k_rope_offset;
  L.v_scale = c_kv_scale;
  L.v_offset = c_kv_offset;
  L.cu_q = cu_seqlens_q;
  L.seq_lens = seq_lens;
  L.table = block_table;
  L.err_count = dev_error_count;
  L.status = static_cast<int32_t*>(workspace);
  L.partials = static_cast<uint8_t*>(workspace) + ra::kAttnHeader;
  L.wait_ns = g_wait_ns.load();
  L.stall_loads = g_stall_next_attn.exchange(0);
  const char* why = "launch failed";
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (w) {
    L.window = w->window;
    L.sinks = w->sinks;
  }
  if (x) {
    // each sequence's own keys, then the prefix's for the rows of all sequences, which join those
    uint8_t* const ws = static_cast<uint8_t*>(workspace);
    ra::PagedLaunch own = L, over = over_prefix(L, x);
    own.lse = nullptr;
    own.rows_out = reinterpret_cast<float*>(aligned_in(ws, plan.rows));
    own.stats_out = reinterpret_cast<float4*>(aligned_in(ws, plan.stats));
    own.partials = ws + plan.partials;
    over.seq_lens = prefix_len;
    over.table = prefix_table;
    over.prior = own.rows_out;
    over.prior_stats = own.stats_out;
    e = ra::launch_paged_prefix(own, over, behind_prefix(L, x, prefix_len, prefix_table), cs, &why);
  } else {
    e = w ? ra::launch_paged_extended(L, cs, &why) : ra::launch_paged_attention(L, cs, &why);
  }
  if (e != cudaSuccess)
    return fail(RA_ERR_CUDA, "%s: %s (%s)", x ? "paged_prefix_attention" : w ? "paged_window_attention" : "paged_attention", why,
                cudaGetErrorString(e));
  return ok();
}

ra_status paged_attention(const kv_rms_norm_rope_cache_params* cache, const paged_attention_params* p,
                          const uint16_t* q, const void* k_cache, const void* ckv_cache,
                          const int32_t* seq_lens, const int32_t* block_table, const int32_t* cu_seqlens_q,
                          const float* k_rope_scale, const float* c_kv_scale, const float* k_rope_offset,
                          const float* c_kv_offset, uint16_t* out, float* lse, int32_t* dev_error_count,
                          void* workspace, size_t workspace_bytes, void* stream) {
  return paged_call(cache, p, nullptr, nullptr, nullptr, nullptr, q, k_cache, ckv_cache, seq_lens, block_table, cu_seqlens_q,
                    k_rope_scale, c_kv_scale, k_rope_offset, c_kv_offset, out, lse, dev_error_count, workspace,
                    workspace_bytes, stream);
}

ra_status paged_window_attention(const kv_rms_norm_rope_cache_params* cache, const paged_attention_params* p,
                                 const attention_window* window, const uint16_t* q, const void* k_cache,
                                 const void* ckv_cache, const int32_t* seq_lens, const int32_t* block_table,
                                 const int32_t* cu_seqlens_q, const float* k_rope_scale, const float* c_kv_scale,
                                 const float* k_rope_offset, const float* c_kv_offset, uint16_t* out, float* lse,
                                 int32_t* dev_error_count, void* workspace, size_t workspace_bytes, void* stream) {
  if (!window) return fail(RA_ERR_INVALID_ARG, "window is NULL");
  return paged_call(cache, p, window, nullptr, nullptr, nullptr, q, k_cache, ckv_cache, seq_lens, block_table, cu_seqlens_q,
                    k_rope_scale, c_kv_scale, k_rope_offset, c_kv_offset, out, lse, dev_error_count, workspace,
                    workspace_bytes, stream);
}

ra_status paged_prefix_attention_workspace_bytes(const kv_rms_norm_rope_cache_params* cache, const paged_attention_params* p,
                                                 const attention_prefix* prefix, size_t* bytes) {
  if (!bytes) return fail(RA_ERR_INVALID_ARG, "bytes is NULL");
  CacheShape s;
  ra_status st = check_cache_alone(cache, &s);
  if (st == RA_OK) st = check_paged(cache, p, s);
  if (st == RA_OK) st = check_prefix(cache, p, prefix);
  if (st != RA_OK) return st;
  *bytes = prefix_plan(paged_launch(cache, p, s), prefix).bytes;
  return ok();
}

ra_status paged_prefix_attention(const kv_rms_norm_rope_cache_params* cache, const paged_attention_params* p,
                                 const attention_prefix* prefix, const uint16_t* q, const void* k_cache,
                                 const void* ckv_cache, const int32_t* prefix_len, const int32_t* prefix_table,
                                 const int32_t* seq_lens, const int32_t* block_table, const int32_t* cu_seqlens_q,
                                 const float* k_rope_scale, const float* c_kv_scale, const float* k_rope_offset,
                                 const float* c_kv_offset, uint16_t* out, float* lse, int32_t* dev_error_count,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  if (!prefix) return fail(RA_ERR_INVALID_ARG, "prefix is NULL");
  return paged_call(cache, p, nullptr, prefix, prefix_len, prefix_table, q, k_cache, ckv_cache, seq_lens, block_table,
                    cu_seqlens_q, k_rope_scale, c_kv_scale, k_rope_offset, c_kv_offset, out, lse, dev_error_count, workspace,
                    workspace_bytes, stream);
}

ra_status attention_status(void* workspace, void* stream, int32_t* device_status) {
  if (!device_status) return fail(RA_ERR_INVALID_ARG, "device_status is required");
  if (!workspace) return fail(RA_ERR_INVALID_ARG, "workspace is required");
  if (!aligned16(workspace)) return fail(RA_ERR_ALIGNMENT, "workspace must be 16-byte aligned");
  if (validate_only()) {
    *device_status = 0;
    return ok();
  }
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  int32_t v = 0;
  cudaError_t e = cudaMemcpyAsync(&v, workspace, sizeof(v), cudaMemcpyDeviceToHost, cs);
  if (e == cudaSuccess) e = cudaStreamSynchronize(cs);
  if (e == cudaSuccess && v != 0) e = cudaMemsetAsync(workspace, 0, sizeof(int32_t), cs);
  if (e == cudaSuccess) e = cudaStreamSynchronize(cs);
  if (e != cudaSuccess) return cuda_fail(e, "attention status read");
  *device_status = v;
  if (v != 0) return fail(RA_ERR_TIMEOUT, "an attention pipeline wait ran out of time (status %d)", v);
  return ok();
}

static ra_status check_paging(const kv_cache_paging_params* p) {
  if (p == nullptr) return fail(RA_ERR_INVALID_ARG, "params is NULL");
  if (p->B < 1 || p->max_tokens < 1) return fail(RA_ERR_INVALID_ARG, "B and max_tokens must be >= 1 (no empty tensors)");
  if (p->block_num < 1 || p->block_num > 0x7fffffffLL || p->block_size < 1 || p->block_size > 0x7fffffffLL)
    return fail(RA_ERR_INVALID_ARG, "block_num and block_size must be in [1, 2^31)");
  if (p->block_table_stride < 1 || p->block_table_stride > 0x7fffffffLL)
    return fail(RA_ERR_INVALID_ARG, "block_table_stride must be in [1, 2^31)");
  if (p->B > ra::kPagingRequests) return fail(RA_ERR_UNSUPPORTED, "the paging calls are built for up to 16384 requests");
  if (p->B * p->block_table_stride > ra::kPagingEntries || p->max_tokens > ra::kPagingTokens)
    return fail(RA_ERR_UNSUPPORTED, "the paging calls are built for block tables of up to 2^31 - 256 entries and up to 2^30 tokens");
  return RA_OK;
}
static bool aligned4(std::initializer_list<const void*> ptrs) {
  for (const void* q : ptrs)
    if (reinterpret_cast<uintptr_t>(q) & 3u) return false;
  return true;
}
static ra::PagingLaunch paging_launch(const kv_cache_paging_params* p) {
  ra::PagingLaunch L{};
  L.B = p->B;
  L.block_num = p->block_num;
  L.block_size = p->block_size;
  L.table_stride = p->block_table_stride;
  L.max_tokens = p->max_tokens;
  return L;
}

ra_status kv_cache_extend(const kv_cache_paging_params* p, const int32_t* new_tokens, const int32_t* seq_lens,
                          int32_t* block_table, const int32_t* free_pages, const int32_t* free_count, int64_t* index,
                          int32_t* cu_seqlens, int32_t* new_seq_lens, int32_t* new_free_count, int32_t* dev_error_count,
                          void* stream) {
  const ra_status st = check_paging(p);
  if (st != RA_OK) return st;
  if (!new_tokens || !seq_lens || !block_table || !free_pages || !free_count || !index || !cu_seqlens || !new_seq_lens ||
      !new_free_count)
    return fail(RA_ERR_INVALID_ARG, "every tensor but dev_error_count is required");
  if ((reinterpret_cast<uintptr_t>(index) & 7u) || !aligned4({new_tokens, seq_lens, block_table, free_pages, free_count, cu_seqlens,
                                                              new_seq_lens, new_free_count, dev_error_count}))
    return fail(RA_ERR_ALIGNMENT, "index must be 8-byte aligned, the other tensors 4-byte");
  if (validate_only()) return ok();
  ra::PagingLaunch L = paging_launch(p);
  L.counts = new_tokens;
  L.seq_lens = seq_lens;
  L.table = block_table;
  L.free_pages = const_cast<int32_t*>(free_pages);  // only read
  L.free_count = free_count;
  L.index = index;
  L.cu = cu_seqlens;
  L.new_lens = new_seq_lens;
  L.new_free_count = new_free_count;
  L.err_count = dev_error_count;
  const cudaError_t e = ra::launch_cache_extend(L, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kv_cache_extend launch");
  return ok();
}

ra_status kv_cache_slots(const kv_cache_paging_params* p, const int32_t* starts, const int32_t* counts,
                         const int32_t* block_table, int64_t* index, int32_t* cu_seqlens, int32_t* dev_error_count,
                         void* stream) {
  const ra_status st = check_paging(p);
  if (st != RA_OK) return st;
  if (!counts || !block_table || !index || !cu_seqlens)
    return fail(RA_ERR_INVALID_ARG, "counts, block_table, index and cu_seqlens are required");
  if ((reinterpret_cast<uintptr_t>(index) & 7u) || !aligned4({starts, counts, block_table, cu_seqlens, dev_error_count}))
    return fail(RA_ERR_ALIGNMENT, "index must be 8-byte aligned, the other tensors 4-byte");
  if (validate_only()) return ok();
  ra::PagingLaunch L = paging_launch(p);
  L.counts = counts;
  L.starts = starts;
  L.table = const_cast<int32_t*>(block_table);  // only read
  L.index = index;
  L.cu = cu_seqlens;
  L.err_count = dev_error_count;
  const cudaError_t e = ra::launch_cache_slots(L, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kv_cache_slots launch");
  return ok();
}

ra_status kv_cache_truncate(const kv_cache_paging_params* p, const int32_t* keep, const int32_t* seq_lens,
                            const int32_t* block_table, int32_t* free_pages, const int32_t* free_count,
                            int32_t* new_seq_lens, int32_t* new_free_count, int32_t* dev_error_count, void* stream) {
  const ra_status st = check_paging(p);
  if (st != RA_OK) return st;
  if (!seq_lens || !block_table || !free_pages || !free_count || !new_seq_lens || !new_free_count)
    return fail(RA_ERR_INVALID_ARG, "every tensor but keep and dev_error_count is required");
  if (!aligned4({keep, seq_lens, block_table, free_pages, free_count, new_seq_lens, new_free_count, dev_error_count}))
    return fail(RA_ERR_ALIGNMENT, "the tensors must be 4-byte aligned");
  if (validate_only()) return ok();
  ra::PagingLaunch L = paging_launch(p);
  L.counts = keep;
  L.seq_lens = seq_lens;
  L.table = const_cast<int32_t*>(block_table);  // only read
  L.free_pages = free_pages;
  L.free_count = free_count;
  L.new_lens = new_seq_lens;
  L.new_free_count = new_free_count;
  L.err_count = dev_error_count;
  const cudaError_t e = ra::launch_cache_truncate(L, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kv_cache_truncate launch");
  return ok();
}

ra_status kv_cache_read(const kv_rms_norm_rope_cache_params* p, const int64_t* index, const void* k_cache,
                        const void* ckv_cache, const float* k_rope_scale, const float* c_kv_scale,
                        const float* k_rope_offset, const float* c_kv_offset, uint16_t* k_out,
                        uint16_t* c_kv_out, int32_t* dev_error_count, void* stream) {
  CacheShape s;
  const ra_status st = check_cache(p, k_rope_scale, c_kv_scale, k_rope_offset, c_kv_offset, &s);
  if (st != RA_OK) return st;
  if (p->B < 1 || p->S < 1) return fail(RA_ERR_INVALID_ARG, "empty tensors are not supported");
  if (p->S > (1LL << 31) || p->B > (1LL << 31) || p->B * p->S > (1LL << 40) / p->N)  // no product passes 2^62
    return fail(RA_ERR_INVALID_ARG, "too many rows");
  if (!index || (!k_out && !c_kv_out) || (k_out && !k_cache) || (c_kv_out && !ckv_cache))
    return fail(RA_ERR_INVALID_ARG, "index, and an output with its cache, are required");
  if ((reinterpret_cast<uintptr_t>(index) & 7u) != 0 || !aligned16(k_cache) || !aligned16(ckv_cache) ||
      !aligned16(k_out) || !aligned16(c_kv_out))
    return fail(RA_ERR_ALIGNMENT, "caches and outputs must be 16-byte aligned (index 8-byte)");
  if ((reinterpret_cast<uintptr_t>(dev_error_count) & 3u) != 0)
    return fail(RA_ERR_ALIGNMENT, "dev_error_count must be 4-byte aligned");
  if (validate_only()) return ok();
  ra::ReadLaunch L{};
  L.index = index;
  L.k_cache = k_cache;
  L.v_cache = ckv_cache;
  L.k_scale = k_rope_scale;
  L.k_offset = k_rope_offset;
  L.v_scale = c_kv_scale;
  L.v_offset = c_kv_offset;
  L.k_out = k_out;
  L.v_out = c_kv_out;
  L.err_count = dev_error_count;
  L.B = p->B;
  L.N = p->N;
  L.S = p->S;
  L.block_num = p->block_num;
  L.block_size = p->cache_mode == RA_CACHE_NORM ? 1 : p->block_size;
  L.cache_seq = p->cache_seq_len;
  L.kw = s.kw;
  L.vw = s.vw;
  L.mode = p->cache_mode;
  L.f16 = p->kv_dtype == RA_FP16;
  L.kq = s.kq;
  L.vq = s.vq;
  L.k_scalar = p->k_quant_scalar;
  L.v_scalar = p->c_kv_quant_scalar;
  L.variant = p->variant;
  const cudaError_t e = ra::launch_cache_read(L, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kv_cache_read launch");
  return ok();
}

}  // extern "C"
