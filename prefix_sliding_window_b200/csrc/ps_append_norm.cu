// Appends that normalise and rotate on the way into the store (bf16, or quantised to 4 bits), and
// the read-back of a 4-bit store, sm_100a.
//
// One pass: a token's packed q, k and v heads are read once; keys are normalised, rotated at the
// token's position and written to their prefix row or ring slot, values go straight there, queries
// to q_out.  Bound by HBM for long prompts (one read and one write a row) and by latency for a
// decode step's single tokens.  Of tokens that share a ring slot only the newest of the call is
// written, so the result does not depend on which block runs first.
//
// 4-bit rows: eight lanes hold a row, so the least and greatest value of a group of 64 dims take
// three shuffles each; every lane packs its two 8-dim chunks into two of the row's sixteen words.
#include <cuda_bf16.h>

#include "ps_norm_rope.cuh"
#include "ps_store.cuh"

namespace ps {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float row_min(float v) {
  v = fminf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  v = fminf(v, __shfl_xor_sync(0xffffffffu, v, 2));
  return fminf(v, __shfl_xor_sync(0xffffffffu, v, 4));
}
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
}

// Quantises a row held by eight lanes (chunks p.c1, p.c2 of a lane: x[0..7], x[8..15], on the
// bf16 grid) and writes it: payload words at `pay`, (s, m) of both groups at `rec` (8 bytes).
// All lanes take part; only `live` ones write.
__device__ __forceinline__ void quantise_row(const RopeLane& p, const float (&x)[16], bool live,
                                             int lane8, uint8_t* pay, uint8_t* rec) {
  // least and greatest of each group; a value that is not finite makes the spread a NaN
  float lo[2], hi[2], odd[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    lo[c] = hi[c] = x[8 * c];
    odd[c] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo[c] = fminf(lo[c], x[8 * c + e]);
      hi[c] = fmaxf(hi[c], x[8 * c + e]);
      odd[c] = fmaf(x[8 * c + e], 0.f, odd[c]);  // 0, or NaN
    }
  }
  const int g1 = p.c1 >> 3, g2 = p.c2 >> 3;
  float m[2], s[2];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const float a = fminf(g1 == g ? lo[0] : INFINITY, g2 == g ? lo[1] : INFINITY);
    const float b = fmaxf(g1 == g ? hi[0] : -INFINITY, g2 == g ? hi[1] : -INFINITY);
    const float least = row_min(a), most = row_max(b);
    const float o = (g1 == g ? odd[0] : 0.f) + (g2 == g ? odd[1] : 0.f);
    const bool bad = row_max(o != o ? 1.f : 0.f) > 0.f;
    const float sc = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(most - least, 15.f)));
    m[g] = least;
    s[g] = sc;
    if (bad || !(sc < INFINITY)) m[g] = s[g] = __uint_as_float(0x7fc00000u);
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int chunk = c ? p.c2 : p.c1;
    const int g = chunk >> 3, b = chunk & 7;
    const float mm = g ? m[1] : m[0], ss = g ? s[1] : s[0];
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float u = ss > 0.f ? rintf(__fdiv_rn(x[8 * c + e] - mm, ss)) : 0.f;
      u = fminf(fmaxf(u, 0.f), 15.f);
      word |= static_cast<uint32_t>(u) << (4 * (e >> 1) + 16 * (e & 1));
    }
    if (live) *reinterpret_cast<uint32_t*>(pay + 4 * (2 * b + g)) = word;
  }
  if (live && lane8 == 0)
    *reinterpret_cast<uint2*>(rec) =
        make_uint2(cvt_bf16x2(s[0], m[0]), cvt_bf16x2(s[1], m[1]));
}

__device__ __forceinline__ void round_bf16(float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w = cvt_bf16x2(x[2 * i], x[2 * i + 1]);
    x[2 * i] = __uint_as_float(w << 16);
    x[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
  }
}

// One block per TT tokens of the call.
template <int TT, bool Q4>
__global__ void __launch_bounds__(kThreads) append_norm_kernel(const AppendNormArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ __align__(16) float s_cos[TT][kHalfDim];
  __shared__ __align__(16) float s_sin[TT][kHalfDim];
  __shared__ __align__(16) float s_w[2 * kHeadDim];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t tokens = a.batch * a.T;
  const int64_t tok0 = (int64_t)blockIdx.x * TT;
  const int ntok = static_cast<int>(tokens - tok0 < TT ? tokens - tok0 : TT);
  const RopeLane p = rope_lane(a.rope, lane & 7);
  const int nq = a.q ? (a.hq + 3) / 4 : 0;
  const int nk = (a.hkv + 3) / 4;
  const int per = nq + 2 * nk;

  for (int i = threadIdx.x; i < ntok * (a.rope.dim / 2); i += kThreads) {
    const int t = i / (a.rope.dim / 2), f = i % (a.rope.dim / 2);
    const int64_t tok = tok0 + t;
    const int64_t pos = a.pos0[tok / a.T] + tok % a.T;
    if (!bad_rope_position(pos)) rope_angle(a.rope, pos, f, s_cos[t], s_sin[t]);
  }
  load_norm_weights(a.norm, s_w);
  __syncthreads();

  for (int it = warp; it < ntok * per; it += kWarps) {
    const int t = it / per;
    int sub = it % per;
    const int64_t tok = tok0 + t, b = tok / a.T;
    const int64_t p0 = a.pos0[b];
    const int64_t pos = p0 + tok % a.T;
    const bool is_q = sub < nq;
    const bool is_v = !is_q && sub >= nq + nk;
    if (!is_q) sub -= is_v ? nq + nk : nq;
    const int head = 4 * sub + (lane >> 3);
    const int heads = is_q ? a.hq : a.hkv;
    StoreRow row = store_row(a.store, a.hkv, b, pos);
    // a token the store has no place for is skipped; its queries become zeros.  A bad table
    // entry only loses the row
    const bool skip = bad_rope_position(pos) || (row.flag && !a.store.table);
    if (row.flag && a.status && it % per == nq && lane == 0) atomicOr(a.status, row.flag);
    if (!is_q) {
      // a newer token of this call owns the ring slot
      const bool stale = pos >= a.store.lp && pos <= p0 + a.T - 1 - a.store.w;
      if (row.flag || (stale && !a.store.linear)) continue;
    }
    bool live = head < heads;
    const __nv_bfloat16* src = (is_q ? a.q + tok * a.q_stride
                                     : is_v ? a.v + tok * a.v_stride : a.k + tok * a.k_stride) +
                               head * kHeadDim;
    uint4 v1 = make_uint4(0, 0, 0, 0), v2 = v1;
    if (live) {
      v1 = *reinterpret_cast<const uint4*>(src + 8 * p.c1);
      v2 = *reinterpret_cast<const uint4*>(src + 8 * p.c2);
    }
    const int64_t at = row.unit + head * row.stride;
    float x[16];
    if (!is_v || Q4) {
      unpack8(v1, x);
      unpack8(v2, x + 8);
    }
    if (!is_v) {
      norm_and_turn(a.rope, p, (is_q ? a.norm.wq : a.norm.wk) != nullptr,
                    s_w + (is_q ? 0 : kHeadDim), a.norm.eps, s_cos[t], s_sin[t], x);
      v1 = pack8(x);
      v2 = pack8(x + 8);
    }
    if (Q4 && !is_q) {
      if (!is_v) round_bf16(x);
      uint8_t* pay = (is_v ? a.store.v[row.ring] : a.store.k[row.ring]) + at * kQ4RowBytes;
      uint8_t* rec = a.store.s[row.ring] + at * kQ4RecordBytes + (is_v ? 8 : 0);
      quantise_row(p, x, live, lane & 7, pay, rec);
      continue;
    }
    __nv_bfloat16* dst =
        is_q ? a.q_out + (tok * a.hq + head) * kHeadDim
             : reinterpret_cast<__nv_bfloat16*>(is_v ? a.store.v[row.ring] : a.store.k[row.ring]) +
                   at * kHeadDim;
    if (is_q && skip) v1 = v2 = make_uint4(0, 0, 0, 0);
    if (live) {
      *reinterpret_cast<uint4*>(dst + 8 * p.c1) = v1;
      *reinterpret_cast<uint4*>(dst + 8 * p.c2) = v2;
    }
  }
}

// Eight lanes a row: lane l takes the 8-dim block l of both groups (words 2 l, 2 l + 1).
__global__ void __launch_bounds__(kThreads) read_q4_kernel(const ReadQ4Args a) {
  pdl_wait();
  pdl_trigger();
  const int lane8 = threadIdx.x & 7;
  const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 3;  // (b, t, head)
  if (i >= a.batch * a.T * a.hkv) return;
  const int head = static_cast<int>(i % a.hkv);
  const int64_t tok = i / a.hkv, b = tok / a.T;
  const int64_t p0 = a.pos0[b], pos = p0 + tok % a.T;
  const StoreRow row = store_row(a.store, a.hkv, b, pos);
  if (row.flag && a.status && lane8 == 0 && head == 0) atomicOr(a.status, row.flag);
  const bool stale = !a.store.linear && pos >= a.store.lp && pos <= p0 + a.T - 1 - a.store.w;
  const bool held = !row.flag && !stale;
  const int64_t at = row.unit + head * row.stride;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    __nv_bfloat16* out = kv ? a.v_out : a.k_out;
    if (!out) continue;
    uint4 y[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (held) {
      const uint8_t* pay = (kv ? a.store.v[row.ring] : a.store.k[row.ring]) + at * kQ4RowBytes;
      const uint2 words = *reinterpret_cast<const uint2*>(pay + 8 * lane8);
      const uint2 rec = *reinterpret_cast<const uint2*>(a.store.s[row.ring] +
                                                        at * kQ4RecordBytes + 8 * kv);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const uint32_t w = g ? words.y : words.x, r = g ? rec.y : rec.x;
        const float s = __uint_as_float(r << 16), m = __uint_as_float(r & 0xffff0000u);
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          x[e] = fmaf(s, static_cast<float>((w >> (4 * (e >> 1) + 16 * (e & 1))) & 15u), m);
        y[g] = pack8(x);
      }
    }
    __nv_bfloat16* dst = out + i * kHeadDim + 8 * lane8;
    *reinterpret_cast<uint4*>(dst) = y[0];
    *reinterpret_cast<uint4*>(dst + kHalfDim) = y[1];
  }
}

}  // namespace

int launch_append_norm(const AppendNormArgs& a, bool q4, cudaStream_t stream) {
  const int64_t tokens = a.batch * a.T;
  if (tokens <= 0) return PS_OK;
  // four tokens a block share the set-up once there are blocks enough for every SM
  const bool wide = tokens > 8 * (int64_t)sm_count();
  const int64_t grid = wide ? (tokens + 3) / 4 : tokens;
  if (grid > 0x7fffffff) return fail(PS_ERR_UNSUPPORTED, "too many tokens");
  auto kern = q4 ? (wide ? append_norm_kernel<4, true> : append_norm_kernel<1, true>)
                 : (wide ? append_norm_kernel<4, false> : append_norm_kernel<1, false>);
  return check_cuda(
      launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, stream, a),
      "append_norm_kernel launch");
}

int launch_read_q4(const ReadQ4Args& a, cudaStream_t stream) {
  const int64_t threads = a.batch * a.T * a.hkv * 8;
  if (threads <= 0) return PS_OK;
  const int64_t grid = (threads + kThreads - 1) / kThreads;
  if (grid > 0x7fffffff) return fail(PS_ERR_UNSUPPORTED, "too many rows");
  return check_cuda(launch_pdl(read_q4_kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads),
                               0, stream, a),
                    "read_q4_kernel launch");
}

}  // namespace ps
