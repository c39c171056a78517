// Appends that normalise and rotate on the way into the store (bf16, or quantised to 4 bits), and
// the read-back of a 4-bit store, sm_100a.
//
// One pass: a token's packed q, k and v heads are read once; keys are normalised, rotated at the
// token's position and written to their prefix row or ring slot, values go straight there, queries
// to q_out.  Bound by HBM for long prompts (one read and one write a row) and by latency for a
// decode step's single tokens.  Of tokens that share a ring slot only the newest of the call is
// written, so the result does not depend on which block runs first.
//
// A warp keeps a token's angles and weights in registers over all of its heads, as in the pass
// without a store; with few tokens eight warps share one.
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

// Least and greatest of two or of a row's eight lanes; a NaN stays one.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float row_min(float v) {
  v = min_nan(v, __shfl_xor_sync(0xffffffffu, v, 1));
  v = min_nan(v, __shfl_xor_sync(0xffffffffu, v, 2));
  return min_nan(v, __shfl_xor_sync(0xffffffffu, v, 4));
}
__device__ __forceinline__ float row_max(float v) {
  v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, 1));
  v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, 2));
  return max_nan(v, __shfl_xor_sync(0xffffffffu, v, 4));
}

// Quantises a row held by eight lanes (chunks p.c1, p.c2 of a lane, bf16) and writes it: payload
// words at `pay`, (s, m) of both groups at `rec` (8 bytes).  All lanes take part; only `live` ones
// write.  A code is the rounded quotient (x - m) / s; the product with 1 / s is within 2e-6 of it,
// so only a product that near to a half needs the division.
__device__ __forceinline__ void quantise_row(const RopeLane& p, const uint4& r1, const uint4& r2,
                                             bool live, int lane8, uint8_t* pay, uint8_t* rec) {
  float x[2][8], lo[2], hi[2];
  const uint32_t w[2][4] = {{r1.x, r1.y, r1.z, r1.w}, {r2.x, r2.y, r2.z, r2.w}};
#pragma unroll
  for (int c = 0; c < 2; ++c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[c][2 * i] = __uint_as_float(w[c][i] << 16);
      x[c][2 * i + 1] = __uint_as_float(w[c][i] & 0xffff0000u);
    }
    lo[c] = hi[c] = x[c][0];
#pragma unroll
    for (int e = 1; e < 8; ++e) {
      lo[c] = min_nan(lo[c], x[c][e]);
      hi[c] = max_nan(hi[c], x[c][e]);
    }
  }
  const int g1 = p.c1 >> 3, g2 = p.c2 >> 3;
  float m[2], s[2];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    m[g] = row_min(min_nan(g1 == g ? lo[0] : INFINITY, g2 == g ? lo[1] : INFINITY));
    const float most =
        row_max(max_nan(g1 == g ? hi[0] : -INFINITY, g2 == g ? hi[1] : -INFINITY));
    s[g] = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(most - m[g], 15.f)));
    if (!(s[g] < INFINITY)) m[g] = s[g] = __uint_as_float(0x7fc00000u);
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int chunk = c ? p.c2 : p.c1;
    const int g = chunk >> 3, b = chunk & 7;
    const float mm = g ? m[1] : m[0], ss = g ? s[1] : s[0];
    const float inv = __fdiv_rn(1.f, ss);
    float u[8];
    bool sure = true;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float t = (x[c][e] - mm) * inv;
      u[e] = rintf(t);
      sure = sure && fabsf(t - u[e]) < 0.499996f;
    }
    if (!sure) {
#pragma unroll 1
      for (int e = 0; e < 8; ++e) {
        const float q = ss > 0.f ? rintf(__fdiv_rn(x[c][e] - mm, ss)) : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i == e) u[i] = q;
      }
    }
    // halves of the word as sums of codes times 16^i, exact in fp32
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = fminf(u[e], 15.f);
    const float lo16 = fmaf(u[6], 4096.f, fmaf(u[4], 256.f, fmaf(u[2], 16.f, u[0])));
    const float hi16 = fmaf(u[7], 4096.f, fmaf(u[5], 256.f, fmaf(u[3], 16.f, u[1])));
    const uint32_t word = static_cast<uint32_t>(lo16) | (static_cast<uint32_t>(hi16) << 16);
    if (live) *reinterpret_cast<uint32_t*>(pay + 4 * (2 * b + g)) = word;
  }
  if (live && lane8 == 0)
    *reinterpret_cast<uint2*>(rec) =
        make_uint2(cvt_bf16x2(s[0], m[0]), cvt_bf16x2(s[1], m[1]));
}

constexpr int kTokens = 2;  // consecutive tokens of a warp, where there are tokens enough

// SPLIT warps share a token (1 or 8).
template <int SPLIT, bool Q4, bool INTER>
__global__ void __launch_bounds__(kThreads, Q4 ? 2 : 3)
    append_norm_kernel(const AppendNormArgs a) {
  __shared__ __align__(16) float s_cos[kWarps][kHalfDim];
  __shared__ __align__(16) float s_sin[kWarps][kHalfDim];
  __shared__ __align__(16) float s_w[2 * kHeadDim];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const RopeLane p = rope_lane<INTER>(a.rope, lane & 7);
  const int nq = a.q ? (a.hq + 3) / 4 : 0;
  const int nk = (a.hkv + 3) / 4;
  const int64_t gw = (int64_t)blockIdx.x * kWarps + warp;
  const int sub0 = SPLIT == 1 ? 0 : static_cast<int>(gw % SPLIT);
  int64_t tok = SPLIT == 1 ? gw * kTokens : gw / SPLIT;
  int64_t end = tok + (SPLIT == 1 ? kTokens : 1);
  if (end > a.batch * a.T) end = a.batch * a.T;
  pdl_wait();
  pdl_trigger();
  load_norm_weights(a.norm, s_w);
  __syncthreads();

  for (; tok < end; ++tok) {
    const int64_t b = tok / a.T;
    const int64_t p0 = a.pos0[b], pos = p0 + (tok - b * a.T);
    const StoreRow row = store_row(a.store, a.hkv, b, pos);
    if (row.flag && sub0 == 0 && a.status && lane == 0) atomicOr(a.status, row.flag);
    // a token the store has no place for is skipped; its queries become zeros.  A bad table
    // entry only loses the row.  A row whose ring slot a newer token of the call owns is not written
    const bool bad = bad_rope_position(pos);
    const bool skip = bad || (row.flag && !a.store.table);
    const bool stale =
        !a.store.linear && pos >= a.store.lp && pos <= p0 + a.T - 1 - a.store.w;
    const int per = nq + (row.flag || stale ? 0 : 2 * nk);

    auto load = [&](int sub, uint4& r1, uint4& r2) {
      r1 = r2 = make_uint4(0, 0, 0, 0);
      if (sub >= per) return;
      const bool is_q = sub < nq, is_v = sub >= nq + nk;
      const int head = 4 * (is_q ? sub : is_v ? sub - nq - nk : sub - nq) + (lane >> 3);
      if (head >= (is_q ? a.hq : a.hkv)) return;
      const __nv_bfloat16* src = (is_q ? a.q + tok * a.q_stride
                                       : is_v ? a.v + tok * a.v_stride : a.k + tok * a.k_stride) +
                                 head * kHeadDim;
      r1 = *reinterpret_cast<const uint4*>(src + 8 * p.c1);
      r2 = *reinterpret_cast<const uint4*>(src + 8 * p.c2);
    };
    uint4 n1, n2;
    load(sub0, n1, n2);
    if (sub0 < per) rope_angles(a.rope, bad ? 0 : pos, lane, s_cos[warp], s_sin[warp]);
    RowCoef coef;
    int side = -1;  // whose weights are in coef
    for (int sub = sub0; sub < per; sub += SPLIT) {
      uint4 r1 = n1, r2 = n2;
      load(sub + SPLIT, n1, n2);
      const bool is_q = sub < nq, is_v = sub >= nq + nk;
      const int head = 4 * (is_q ? sub : is_v ? sub - nq - nk : sub - nq) + (lane >> 3);
      const bool live = head < (is_q ? a.hq : a.hkv);
      if (!is_v) {
        const bool norm = (is_q ? a.norm.wq : a.norm.wk) != nullptr;
        if (side != is_q) {
          side = is_q;
          row_coef<INTER>(p, norm, s_w + (is_q ? 0 : kHeadDim), s_cos[warp], s_sin[warp], coef);
        }
        float u[8], v[8];
        unpack_pairs<INTER>(r1, r2, u, v);
        norm_and_turn(p, norm, coef, a.norm.eps, u, v);
        pack_pairs<INTER>(u, v, r1, r2);
        if (is_q && skip) r1 = r2 = make_uint4(0, 0, 0, 0);
      }
      const int64_t at = row.unit + head * row.stride;
      if (Q4 && !is_q) {
        uint8_t* pay = (is_v ? a.store.v[row.ring] : a.store.k[row.ring]) + at * kQ4RowBytes;
        uint8_t* rec = a.store.s[row.ring] + at * kQ4RecordBytes + (is_v ? 8 : 0);
        quantise_row(p, r1, r2, live, lane & 7, pay, rec);
        continue;
      }
      __nv_bfloat16* dst =
          is_q ? a.q_out + (tok * a.hq + head) * kHeadDim
               : reinterpret_cast<__nv_bfloat16*>(is_v ? a.store.v[row.ring]
                                                       : a.store.k[row.ring]) + at * kHeadDim;
      if (live) {
        *reinterpret_cast<uint4*>(dst + 8 * p.c1) = r1;
        *reinterpret_cast<uint4*>(dst + 8 * p.c2) = r2;
      }
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
        y[g] = make_uint4(cvt_bf16x2(x[0], x[1]), cvt_bf16x2(x[2], x[3]), cvt_bf16x2(x[4], x[5]),
                          cvt_bf16x2(x[6], x[7]));
      }
    }
    __nv_bfloat16* dst = out + i * kHeadDim + 8 * lane8;
    *reinterpret_cast<uint4*>(dst) = y[0];
    *reinterpret_cast<uint4*>(dst + kHalfDim) = y[1];
  }
}

}  // namespace

template <bool INTER>
static auto pick_append(bool split, bool q4) {
  return q4 ? (split ? append_norm_kernel<kWarps, true, INTER> : append_norm_kernel<1, true, INTER>)
            : (split ? append_norm_kernel<kWarps, false, INTER>
                     : append_norm_kernel<1, false, INTER>);
}

int launch_append_norm(const AppendNormArgs& a, bool q4, cudaStream_t stream) {
  const int64_t tokens = a.batch * a.T;
  if (tokens <= 0) return PS_OK;
  const bool split = tokens < 16 * (int64_t)sm_count();  // fewer than one a warp slot
  const int64_t grid = split ? tokens : (tokens + kWarps * kTokens - 1) / (kWarps * kTokens);
  if (grid > 0x7fffffff) return fail(PS_ERR_UNSUPPORTED, "too many tokens");
  auto kern = pick_append<false>(split, q4);
  if (a.rope.interleaved) kern = pick_append<true>(split, q4);
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
