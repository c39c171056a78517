// C-ABI entry points of the norm + rotary pass, the appends that apply it, and the 4-bit store:
// argument validation and launch descriptions.  The contracts are in include/ps.h.
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <string>

#include "../../include/ps.h"
#include "ps_internal.h"
#include "ps_ranges.cuh"

using namespace ps;

namespace {

int check_aligned(const void* p, uintptr_t mask, const char* name, bool nullable = false) {
  if (!p && !nullable) return fail(PS_ERR_INVALID_ARG, std::string(name) + " is NULL");
  if ((reinterpret_cast<uintptr_t>(p) & mask) != 0)
    return fail(PS_ERR_INVALID_ARG, std::string(name) + " is not " + std::to_string(mask + 1) +
                                        "-byte aligned");
  return PS_OK;
}

int check_stride(int64_t stride, int64_t heads, const char* name) {
  if (stride < heads * kHeadDim || stride % 8 != 0)
    return fail(PS_ERR_INVALID_ARG,
                std::string(name) + " must be a multiple of 8 and hold every head");
  return PS_OK;
}

// In place needs the output's own layout.
int check_alias(const void* in, const void* out, int64_t stride, int64_t heads, const char* name) {
  if (in && in == out && stride != heads * kHeadDim)
    return fail(PS_ERR_INVALID_ARG, std::string(name) + " in place needs contiguous heads");
  return PS_OK;
}

int make_rope_args(const ps_rope* rope, RopeArgs* r) {
  if (!rope) return fail(PS_ERR_INVALID_ARG, "rope is NULL");
  if (rope->reserved != 0) return fail(PS_ERR_INVALID_ARG, "rope->reserved must be 0");
  if (rope->layout != PS_ROPE_HALF && rope->layout != PS_ROPE_INTERLEAVED)
    return fail(PS_ERR_INVALID_ARG, "rope->layout is not a PS_ROPE_* layout");
  if (rope->rotary_dim < 0 || rope->rotary_dim > kHeadDim || rope->rotary_dim % 16 != 0)
    return fail(PS_ERR_UNSUPPORTED, "rotary_dim must be a multiple of 16 in [0, head_dim]");
  if (!(rope->attn_factor > 0.f) || !isfinite(rope->attn_factor))
    return fail(PS_ERR_INVALID_ARG, "rope->attn_factor must be finite and > 0");
  r->interleaved = rope->layout;
  r->dim = rope->rotary_dim;
  r->attn = rope->attn_factor;
  for (int i = 0; i < kHeadDim / 2; ++i) {
    const double f = i < rope->rotary_dim / 2 ? rope->inv_freq[i] : 0.0;
    if (!(f >= 0.0 && f <= 1.0))
      return fail(PS_ERR_INVALID_ARG, "rope->inv_freq must lie in [0, 1]");
    r->inv_freq[i] = f;
  }
  return PS_OK;
}

int make_norm_args(const ps_qk_norm* norm, NormArgs* n) {
  *n = NormArgs{nullptr, nullptr, 0, 0.f};
  if (!norm) return PS_OK;
  if (norm->weight_type != PS_TYPE_BF16 && norm->weight_type != PS_TYPE_FP32)
    return fail(PS_ERR_INVALID_ARG, "norm->weight_type is not a PS_TYPE_* type");
  if (!(norm->eps >= 0.f) || !isfinite(norm->eps))
    return fail(PS_ERR_INVALID_ARG, "norm->eps must be finite and >= 0");
  PS_TRY(check_ptr(norm->q_weight, "norm->q_weight", true));
  PS_TRY(check_ptr(norm->k_weight, "norm->k_weight", true));
  n->wq = norm->q_weight;
  n->wk = norm->k_weight;
  n->fp32 = norm->weight_type;
  n->eps = norm->eps;
  return PS_OK;
}

cudaStream_t as_stream(ps_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

uint8_t* bytes(void* p) { return static_cast<uint8_t*>(p); }

// A store in 64-row blocks of one pool.
int check_blocks(const ps_params* params, int64_t n_blocks, const int32_t* block_table,
                 int32_t table_stride, StoreArgs* st) {
  if (params->window % kDecodeTile != 0)
    return fail(PS_ERR_UNSUPPORTED, "a paged store needs a window that is a multiple of 64");
  if (n_blocks < 1 || n_blocks > 0x7fffffffLL)
    return fail(PS_ERR_INVALID_ARG, "n_blocks out of range");
  const int64_t pre = ((int64_t)params->l_prefix + kDecodeTile - 1) / kDecodeTile;
  if (table_stride < pre + params->window / kDecodeTile)
    return fail(PS_ERR_INVALID_ARG, "table_stride smaller than the blocks a sequence needs");
  PS_TRY(check_aligned(block_table, 3, "block_table"));
  st->table = block_table;
  st->table_stride = table_stride;
  st->pre_blocks = static_cast<int32_t>(pre);
  st->n_blocks = n_blocks;
  return PS_OK;
}

StoreArgs empty_store(const ps_params* params) {
  StoreArgs st{};
  st.lp = params->l_prefix;
  st.w = params->window;
  return st;
}

// The 4-bit store a cache describes; `whole`: the prefix must be there (a decode reads it).
int make_store_q4(const ps_params* params, const ps_kv_cache_q4* c, bool whole, StoreArgs* st) {
  if (c->reserved != 0) return fail(PS_ERR_INVALID_ARG, "cache->reserved must be 0");
  *st = empty_store(params);
  const bool ring = c->k_ring || c->v_ring || c->s_ring;
  if (c->block_table) {
    if (ring) return fail(PS_ERR_INVALID_ARG, "a paged store has no ring pointers");
    PS_TRY(check_blocks(params, c->n_blocks, c->block_table, c->table_stride, st));
  } else if (c->n_blocks != 0 || c->table_stride != 0) {
    return fail(PS_ERR_INVALID_ARG, "n_blocks and table_stride without a block_table");
  }
  if (ring) {
    PS_TRY(check_ptr(c->k_ring, "cache->k_ring"));
    PS_TRY(check_ptr(c->v_ring, "cache->v_ring"));
    PS_TRY(check_ptr(c->s_ring, "cache->s_ring"));
  } else if (!c->block_table) {
    if (params->l_prefix < 1)
      return fail(PS_ERR_INVALID_ARG, "a linear store (ring NULL) needs l_prefix = Lmax >= 1");
    st->linear = 1;
  }
  const bool prefix = c->k_prefix || c->v_prefix || c->s_prefix;
  if (prefix || !ring || (whole && params->l_prefix > 0)) {
    PS_TRY(check_ptr(c->k_prefix, "cache->k_prefix"));
    PS_TRY(check_ptr(c->v_prefix, "cache->v_prefix"));
    PS_TRY(check_ptr(c->s_prefix, "cache->s_prefix"));
  }
  st->k[0] = bytes(c->k_prefix), st->k[1] = bytes(c->k_ring);
  st->v[0] = bytes(c->v_prefix), st->v[1] = bytes(c->v_ring);
  st->s[0] = bytes(c->s_prefix), st->s[1] = bytes(c->s_ring);
  return PS_OK;
}

// What the three appends share once the store is known.
int append_norm(const ps_params* params, const ps_rope* rope, const ps_qk_norm* norm,
                const StoreArgs& store, bool q4, int64_t batch, const void* k_new,
                int64_t k_stride, const void* v_new, int64_t v_stride, const void* q,
                int64_t q_stride, void* q_out, const int64_t* pos0, int32_t T,
                int32_t* dev_status, ps_stream_t stream) {
  AppendNormArgs a{};
  PS_TRY(make_rope_args(rope, &a.rope));
  PS_TRY(make_norm_args(norm, &a.norm));
  if (T < 1) return fail(PS_ERR_INVALID_ARG, "T must be >= 1");
  PS_TRY(check_ptr(k_new, "k_new"));
  PS_TRY(check_ptr(v_new, "v_new"));
  PS_TRY(check_stride(k_stride, params->n_kv_heads, "k_stride"));
  PS_TRY(check_stride(v_stride, params->n_kv_heads, "v_stride"));
  if (!q != !q_out) return fail(PS_ERR_INVALID_ARG, "q and q_out go together");
  if (q) {
    PS_TRY(check_ptr(q, "q"));
    PS_TRY(check_ptr(q_out, "q_out"));
    PS_TRY(check_stride(q_stride, params->n_q_heads, "q_stride"));
    PS_TRY(check_alias(q, q_out, q_stride, params->n_q_heads, "q"));
  }
  PS_TRY(check_aligned(pos0, 7, "pos0"));
  PS_TRY(check_aligned(dev_status, 3, "dev_status", true));
  if (batch > 0x7fffffffffLL / T) return fail(PS_ERR_UNSUPPORTED, "too many tokens");
  a.k = static_cast<const __nv_bfloat16*>(k_new);
  a.v = static_cast<const __nv_bfloat16*>(v_new);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_stride = q_stride;
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.pos0 = pos0;
  a.status = dev_status;
  a.batch = batch;
  a.T = T;
  a.hq = params->n_q_heads;
  a.hkv = params->n_kv_heads;
  a.store = store;
  return launch_append_norm(a, q4, as_stream(stream));
}

}  // namespace

extern "C" {

int ps_rope_init(ps_rope* rope, const ps_params* params, int32_t layout, int32_t rotary_dim,
                 const ps_rope_scaling* scaling, float attn_factor) {
  clear_error();
  if (!rope) return fail(PS_ERR_INVALID_ARG, "rope is NULL");
  PS_TRY(check_params(params, false));
  const int32_t kind = scaling ? scaling->kind : PS_ROPE_SCALE_NONE;
  if (scaling && scaling->reserved != 0)
    return fail(PS_ERR_INVALID_ARG, "scaling->reserved must be 0");
  if (kind < PS_ROPE_SCALE_NONE || kind > PS_ROPE_SCALE_YARN)
    return fail(PS_ERR_INVALID_ARG, "scaling->kind is not a PS_ROPE_SCALE_* kind");
  const double theta = params->rope_theta;
  if (theta < 1.0 || (kind == PS_ROPE_SCALE_YARN && theta == 1.0))
    return fail(PS_ERR_UNSUPPORTED, "rope_theta must be >= 1 (> 1 for YARN)");
  if (kind != PS_ROPE_SCALE_NONE && !(scaling->factor >= 1.0 && isfinite(scaling->factor)))
    return fail(PS_ERR_INVALID_ARG, "scaling->factor must be finite and >= 1");
  const bool blend = kind == PS_ROPE_SCALE_BY_PARTS || kind == PS_ROPE_SCALE_YARN;
  if (blend && !(scaling->low > 0.0 && scaling->high > scaling->low && isfinite(scaling->high)))
    return fail(PS_ERR_INVALID_ARG, "scaling needs 0 < low < high");
  if (blend && !(scaling->original_len > 0.0 && isfinite(scaling->original_len)))
    return fail(PS_ERR_INVALID_ARG, "scaling->original_len must be finite and > 0");
  ps_rope r{};
  r.layout = layout;
  r.rotary_dim = rotary_dim;
  r.attn_factor = attn_factor;
  RopeArgs unused;
  PS_TRY(make_rope_args(&r, &unused));  // layout, dims, factor
  const double two_pi = 6.283185307179586477;
  const double dim = rotary_dim;
  double ramp_lo = 0.0, ramp_hi = 1.0;  // YARN: pair indexes where the ramp starts and ends
  if (kind == PS_ROPE_SCALE_YARN) {
    auto index_of = [&](double turns) {
      return dim * log(scaling->original_len / (two_pi * turns)) / (2.0 * log(theta));
    };
    ramp_lo = std::max(floor(index_of(scaling->high)), 0.0);
    ramp_hi = std::min(ceil(index_of(scaling->low)), dim - 1.0);
    if (!(ramp_hi > ramp_lo)) ramp_hi = ramp_lo + 0.001;  // a step
  }
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const double f = pow(theta, -2.0 * i / dim);
    double keep = 1.0;
    if (kind == PS_ROPE_SCALE_LINEAR) keep = 0.0;
    if (kind == PS_ROPE_SCALE_BY_PARTS)
      keep = (scaling->original_len * f / two_pi - scaling->low) / (scaling->high - scaling->low);
    if (kind == PS_ROPE_SCALE_YARN) keep = 1.0 - (i - ramp_lo) / (ramp_hi - ramp_lo);
    keep = std::min(std::max(keep, 0.0), 1.0);
    r.inv_freq[i] =
        kind == PS_ROPE_SCALE_NONE ? f : keep * f + (1.0 - keep) * f / scaling->factor;
  }
  *rope = r;
  return PS_OK;
}

int ps_qk_norm_rope(const ps_params* params, const ps_rope* rope, const ps_qk_norm* norm,
                    const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                    const int64_t* pos, int64_t n_tokens, void* q_out, void* k_out,
                    int32_t* dev_status, ps_stream_t stream) {
  clear_error();
  PS_TRY(check_params(params, false));
  NormRopeArgs a{};
  PS_TRY(make_rope_args(rope, &a.rope));
  PS_TRY(make_norm_args(norm, &a.norm));
  if (n_tokens < 0) return fail(PS_ERR_INVALID_ARG, "n_tokens must be >= 0");
  if (n_tokens == 0) return PS_OK;
  if (!q != !q_out) return fail(PS_ERR_INVALID_ARG, "q and q_out go together");
  if (!k != !k_out) return fail(PS_ERR_INVALID_ARG, "k and k_out go together");
  if (!q && !k) return fail(PS_ERR_INVALID_ARG, "q and k are both NULL");
  if (q) {
    PS_TRY(check_ptr(q, "q"));
    PS_TRY(check_ptr(q_out, "q_out"));
    PS_TRY(check_stride(q_stride, params->n_q_heads, "q_stride"));
    PS_TRY(check_alias(q, q_out, q_stride, params->n_q_heads, "q"));
  }
  if (k) {
    PS_TRY(check_ptr(k, "k"));
    PS_TRY(check_ptr(k_out, "k_out"));
    PS_TRY(check_stride(k_stride, params->n_kv_heads, "k_stride"));
    PS_TRY(check_alias(k, k_out, k_stride, params->n_kv_heads, "k"));
  }
  PS_TRY(check_aligned(pos, 7, "pos"));
  PS_TRY(check_aligned(dev_status, 3, "dev_status", true));
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.pos = pos;
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.k_out = static_cast<__nv_bfloat16*>(k_out);
  a.status = dev_status;
  a.n = n_tokens;
  a.hq = params->n_q_heads;
  a.hkv = params->n_kv_heads;
  return launch_norm_rope(a, as_stream(stream));
}

size_t ps_qk_norm_rope_bwd_workspace_bytes(const ps_params* params, int64_t n_tokens) {
  if (check_params(params, false) != PS_OK || n_tokens < 0) return 0;
  return norm_rope_bwd_workspace_bytes(n_tokens);
}

int ps_qk_norm_rope_bwd(const ps_params* params, const ps_rope* rope, const ps_qk_norm* norm,
                        const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                        const int64_t* pos, int64_t n_tokens, const void* dq_out,
                        const void* dk_out, void* dq, int64_t dq_stride, void* dk,
                        int64_t dk_stride, float* dq_weight, float* dk_weight, void* workspace,
                        size_t ws_bytes, int32_t* dev_status, ps_stream_t stream) {
  clear_error();
  PS_TRY(check_params(params, false));
  NormRopeBwdArgs a{};
  PS_TRY(make_rope_args(rope, &a.rope));
  PS_TRY(make_norm_args(norm, &a.norm));
  if (n_tokens < 0) return fail(PS_ERR_INVALID_ARG, "n_tokens must be >= 0");
  if (!dq_out != !dq) return fail(PS_ERR_INVALID_ARG, "dq_out and dq go together");
  if (!dk_out != !dk) return fail(PS_ERR_INVALID_ARG, "dk_out and dk go together");
  if ((dq_weight && !a.norm.wq) || (dk_weight && !a.norm.wk))
    return fail(PS_ERR_INVALID_ARG, "a weight gradient without a weight");
  PS_TRY(check_ptr(dq_weight, "dq_weight", true));
  PS_TRY(check_ptr(dk_weight, "dk_weight", true));
  const bool any_dw = dq_weight || dk_weight;
  if (any_dw) {
    if (!workspace || ws_bytes < norm_rope_bwd_workspace_bytes(n_tokens))
      return fail(PS_ERR_WORKSPACE, "workspace smaller than ps_qk_norm_rope_bwd_workspace_bytes()");
    PS_TRY(check_aligned(workspace, 255, "workspace"));
  }
  PS_TRY(check_aligned(dev_status, 3, "dev_status", true));
  if (n_tokens > 0) {
    if (!dq_out && !dk_out) return fail(PS_ERR_INVALID_ARG, "dq_out and dk_out are both NULL");
    if ((dq_weight && !dq_out) || (dk_weight && !dk_out))
      return fail(PS_ERR_INVALID_ARG, "a weight gradient without its output's gradient");
    if (dq_out) {
      PS_TRY(check_ptr(dq_out, "dq_out"));
      PS_TRY(check_ptr(dq, "dq"));
      PS_TRY(check_stride(dq_stride, params->n_q_heads, "dq_stride"));
      PS_TRY(check_alias(dq_out, dq, dq_stride, params->n_q_heads, "dq_out"));
      if (a.norm.wq) {
        PS_TRY(check_ptr(q, "q"));
        PS_TRY(check_stride(q_stride, params->n_q_heads, "q_stride"));
      }
    }
    if (dk_out) {
      PS_TRY(check_ptr(dk_out, "dk_out"));
      PS_TRY(check_ptr(dk, "dk"));
      PS_TRY(check_stride(dk_stride, params->n_kv_heads, "dk_stride"));
      PS_TRY(check_alias(dk_out, dk, dk_stride, params->n_kv_heads, "dk_out"));
      if (a.norm.wk) {
        PS_TRY(check_ptr(k, "k"));
        PS_TRY(check_stride(k_stride, params->n_kv_heads, "k_stride"));
      }
    }
    PS_TRY(check_aligned(pos, 7, "pos"));
  } else if (!any_dw) {
    return PS_OK;
  }
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.pos = pos;
  a.dq_out = static_cast<const __nv_bfloat16*>(dq_out);
  a.dk_out = static_cast<const __nv_bfloat16*>(dk_out);
  a.dq = static_cast<__nv_bfloat16*>(dq);
  a.dk = static_cast<__nv_bfloat16*>(dk);
  a.dq_stride = dq_stride;
  a.dk_stride = dk_stride;
  a.partial = any_dw ? static_cast<float*>(workspace) : nullptr;
  a.status = dev_status;
  a.n = n_tokens;
  a.hq = params->n_q_heads;
  a.hkv = params->n_kv_heads;
  return launch_norm_rope_bwd(a, dq_weight, dk_weight, as_stream(stream));
}

int ps_kv_append_norm_rope(const ps_params* params, const ps_rope* rope, const ps_qk_norm* norm,
                           const ps_kv_cache* cache, const void* k_new, int64_t k_stride,
                           const void* v_new, int64_t v_stride, const void* q, int64_t q_stride,
                           void* q_out, const int64_t* pos0, int32_t T, int32_t* dev_status,
                           ps_stream_t stream) {
  clear_error();
  PS_TRY(check_params(params, true));
  if (!cache) return fail(PS_ERR_INVALID_ARG, "cache is NULL");
  if (cache->batch < 0) return fail(PS_ERR_INVALID_ARG, "cache->batch must be >= 0");
  if (cache->batch == 0) return PS_OK;
  StoreArgs st = empty_store(params);
  const bool ring = cache->k_ring || cache->v_ring;
  const bool prefix = cache->k_prefix || cache->v_prefix;
  if (ring) {
    PS_TRY(check_ptr(cache->k_ring, "cache->k_ring"));
    PS_TRY(check_ptr(cache->v_ring, "cache->v_ring"));
  } else {
    if (params->l_prefix < 1)
      return fail(PS_ERR_INVALID_ARG, "a linear cache (ring NULL) needs l_prefix = Lmax >= 1");
    st.linear = 1;
  }
  if (prefix || !ring) {
    PS_TRY(check_ptr(cache->k_prefix, "cache->k_prefix"));
    PS_TRY(check_ptr(cache->v_prefix, "cache->v_prefix"));
  }
  st.k[0] = bytes(cache->k_prefix), st.k[1] = bytes(cache->k_ring);
  st.v[0] = bytes(cache->v_prefix), st.v[1] = bytes(cache->v_ring);
  return append_norm(params, rope, norm, st, false, cache->batch, k_new, k_stride, v_new,
                     v_stride, q, q_stride, q_out, pos0, T, dev_status, stream);
}

int ps_kv_append_norm_rope_paged(const ps_params* params, const ps_rope* rope,
                                 const ps_qk_norm* norm, void* k_pool, void* v_pool,
                                 int64_t n_blocks, const int32_t* block_table,
                                 int32_t table_stride, int64_t batch, const void* k_new,
                                 int64_t k_stride, const void* v_new, int64_t v_stride,
                                 const void* q, int64_t q_stride, void* q_out,
                                 const int64_t* pos0, int32_t T, int32_t* dev_status,
                                 ps_stream_t stream) {
  clear_error();
  PS_TRY(check_params(params, true));
  if (batch < 0) return fail(PS_ERR_INVALID_ARG, "batch must be >= 0");
  StoreArgs st = empty_store(params);
  PS_TRY(check_blocks(params, n_blocks, block_table, table_stride, &st));
  PS_TRY(check_ptr(k_pool, "k_pool"));
  PS_TRY(check_ptr(v_pool, "v_pool"));
  if (batch == 0) return PS_OK;
  st.k[0] = bytes(k_pool);
  st.v[0] = bytes(v_pool);
  return append_norm(params, rope, norm, st, false, batch, k_new, k_stride, v_new, v_stride, q,
                     q_stride, q_out, pos0, T, dev_status, stream);
}

int ps_kv_append_norm_rope_q4(const ps_params* params, const ps_rope* rope,
                              const ps_qk_norm* norm, const ps_kv_cache_q4* cache,
                              const void* k_new, int64_t k_stride, const void* v_new,
                              int64_t v_stride, const void* q, int64_t q_stride, void* q_out,
                              const int64_t* pos0, int32_t T, int32_t* dev_status,
                              ps_stream_t stream) {
  clear_error();
  PS_TRY(check_params(params, true));
  if (!cache) return fail(PS_ERR_INVALID_ARG, "cache is NULL");
  if (cache->batch < 0) return fail(PS_ERR_INVALID_ARG, "cache->batch must be >= 0");
  if (cache->batch == 0) return PS_OK;
  StoreArgs st;
  PS_TRY(make_store_q4(params, cache, false, &st));
  return append_norm(params, rope, norm, st, true, cache->batch, k_new, k_stride, v_new,
                     v_stride, q, q_stride, q_out, pos0, T, dev_status, stream);
}

int ps_kv_read_q4(const ps_params* params, const ps_kv_cache_q4* cache, const int64_t* pos0,
                  int32_t T, void* k_out, void* v_out, int32_t* dev_status, ps_stream_t stream) {
  clear_error();
  PS_TRY(check_params(params, true));
  if (!cache) return fail(PS_ERR_INVALID_ARG, "cache is NULL");
  if (cache->batch < 0) return fail(PS_ERR_INVALID_ARG, "cache->batch must be >= 0");
  if (T < 1) return fail(PS_ERR_INVALID_ARG, "T must be >= 1");
  if (cache->batch == 0) return PS_OK;
  ReadQ4Args a{};
  PS_TRY(make_store_q4(params, cache, false, &a.store));
  PS_TRY(check_ptr(k_out, "k_out", true));
  PS_TRY(check_ptr(v_out, "v_out", true));
  if (!k_out && !v_out) return fail(PS_ERR_INVALID_ARG, "k_out and v_out are both NULL");
  PS_TRY(check_aligned(pos0, 7, "pos0"));
  PS_TRY(check_aligned(dev_status, 3, "dev_status", true));
  if (cache->batch > 0x7fffffffffLL / T) return fail(PS_ERR_UNSUPPORTED, "too many tokens");
  a.k_out = static_cast<__nv_bfloat16*>(k_out);
  a.v_out = static_cast<__nv_bfloat16*>(v_out);
  a.pos0 = pos0;
  a.status = dev_status;
  a.batch = cache->batch;
  a.T = T;
  a.hkv = params->n_kv_heads;
  return launch_read_q4(a, as_stream(stream));
}

size_t ps_decode_q4_workspace_bytes(const ps_params* params, int64_t batch) {
  if (check_params(params, true) != PS_OK || batch < 0) return 0;
  return decode_q4_workspace_bytes(batch, params->n_kv_heads,
                                   (int64_t)params->l_prefix + params->window);
}

int ps_decode_attn_q4(const ps_params* params, const ps_kv_cache_q4* cache, const void* q,
                      const int64_t* pos, void* out, float* lse, void* workspace,
                      size_t ws_bytes, int32_t* dev_status, ps_stream_t stream) {
  clear_error();
  PS_TRY(check_params(params, true));
  if (params->n_q_heads / params->n_kv_heads > kMaxGroup)
    return fail(PS_ERR_UNSUPPORTED, "decode supports at most 8 query heads per KV head");
  if (!cache) return fail(PS_ERR_INVALID_ARG, "cache is NULL");
  if (cache->batch < 0) return fail(PS_ERR_INVALID_ARG, "cache->batch must be >= 0");
  if (cache->batch == 0) return PS_OK;
  if (cache->batch > 0x7fffffffLL / params->n_q_heads)
    return fail(PS_ERR_UNSUPPORTED, "batch too large");
  DecodeQ4Launch l{};
  PS_TRY(make_store_q4(params, cache, true, &l.store));
  PS_TRY(check_ptr(q, "q"));
  PS_TRY(check_aligned(pos, 7, "pos"));
  PS_TRY(check_ptr(out, "out"));
  PS_TRY(check_aligned(lse, 3, "lse", true));
  PS_TRY(check_aligned(dev_status, 3, "dev_status", true));
  const size_t need = decode_q4_workspace_bytes(cache->batch, params->n_kv_heads,
                                                (int64_t)params->l_prefix + params->window);
  if (need > 0) {
    if (!workspace || ws_bytes < need)
      return fail(PS_ERR_WORKSPACE, "workspace smaller than ps_decode_q4_workspace_bytes()");
    PS_TRY(check_ptr(workspace, "workspace"));
  }
  l.q = q;
  l.pos = pos;
  l.out = out;
  l.lse = lse;
  l.workspace = workspace;
  l.status = dev_status;
  l.batch = cache->batch;
  l.hq = params->n_q_heads;
  l.hkv = params->n_kv_heads;
  l.scale = resolve_scale(params);
  if (l.scale > 0x1p32f)  // (scores come out of the products times 2^-85)
    return fail(PS_ERR_UNSUPPORTED, "softmax_scale must be <= 2^32");
  return launch_decode_q4(l, as_stream(stream));
}

}  // extern "C"
