// Per-head RMS norm and rotary positions on bf16 rows of 128 dims, shared by the kernels that
// normalise and rotate (forward, backward, and the appends).
//
// Eight lanes hold one head row, sixteen dims a lane: two 16-byte chunks (8 dims each) chosen so
// that the two dims of every rotated pair sit in one lane.  Rotation then needs no exchange, the
// norm's sum of squares three shuffles, and a warp's loads are whole 128-byte half rows.
//   half layout, R rotated dims, m = R / 16: lanes l < m hold chunks (l, l + m), dims (i, i + R/2);
//     the unrotated chunks 2m .. 15 go two by two to the other lanes
//   interleaved: chunks (l, l + 8); pairs (2i, 2i + 1) never leave a chunk
// A warp takes four heads of one token at a time; q and k heads are never mixed in one item.
#pragma once

#include <cuda_bf16.h>

#include "ps_device.cuh"
#include "ps_internal.h"

namespace ps {

constexpr int kHalfDim = kHeadDim / 2;

// Where a lane's two chunks are and which angles turn them.
struct RopeLane {
  int c1, c2;      // chunks (dims 8 c .. 8 c + 7)
  int a1, a2;      // first of four angle indices each: half layout (8 l, 8 l + 4)
  bool rot1, rot2; // whether the chunk is rotated
};

__device__ __forceinline__ RopeLane rope_lane(const RopeArgs& r, int l) {
  RopeLane p;
  if (r.interleaved) {
    p.c1 = l;
    p.c2 = l + 8;
    p.rot1 = 8 * l < r.dim;
    p.rot2 = 8 * l + 64 < r.dim;
    p.a1 = 4 * p.c1;
    p.a2 = 4 * p.c2;
  } else {
    const int m = r.dim / 16;
    p.rot1 = p.rot2 = l < m;
    p.c1 = l < m ? l : 2 * l;  // 2 m + 2 (l - m)
    p.c2 = l < m ? l + m : 2 * l + 1;
    p.a1 = 8 * l;
    p.a2 = 8 * l + 4;
  }
  return p;
}

// Angles of one token, 64-bit range reduction (rope_cos_sin), into cos[i], sin[i].
__device__ __forceinline__ void rope_angle(const RopeArgs& r, int64_t pos, int i, float* cos,
                                           float* sin) {
  const float2 cs = rope_cos_sin(double(pos), r.inv_freq[i]);
  cos[i] = cs.x * r.attn;
  sin[i] = cs.y * r.attn;
}

__device__ __forceinline__ bool bad_rope_position(int64_t p) { return p < 0 || p >= (1ll << 31); }
__device__ __forceinline__ int32_t rope_position_flag(int64_t p) {
  return p < 0 ? PS_DEV_BAD_POS : PS_DEV_POS_RANGE;
}

__device__ __forceinline__ void unpack8(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(cvt_bf16x2(x[0], x[1]), cvt_bf16x2(x[2], x[3]), cvt_bf16x2(x[4], x[5]),
                    cvt_bf16x2(x[6], x[7]));
}

// Sum over the eight lanes of a row (every lane gets it; the same order in all of them).
__device__ __forceinline__ float row_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  return v;
}

// 1 / sqrt(mean(x^2) + eps) of a row held by eight lanes, fp32.
__device__ __forceinline__ float row_rstd(const float (&x)[16], float eps) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) s = fmaf(x[i], x[i], s);
  return rsqrtf(row_sum(s) * (1.f / kHeadDim) + eps);
}

// Turns a lane's sixteen values (chunk 1, chunk 2) by the token's angles; DIR -1 turns back.
template <int DIR>
__device__ __forceinline__ void rope_turn(const RopeArgs& r, const RopeLane& p, const float* cos,
                                          const float* sin, float (&x)[16]) {
  if (!p.rot1) return;  // chunk 2 is rotated only where chunk 1 is
  const float4 ca = *reinterpret_cast<const float4*>(cos + p.a1);
  const float4 sa = *reinterpret_cast<const float4*>(sin + p.a1);
  const float cA[4] = {ca.x, ca.y, ca.z, ca.w};
  const float sA[4] = {DIR * sa.x, DIR * sa.y, DIR * sa.z, DIR * sa.w};
  if (r.interleaved) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float u = x[2 * j], v = x[2 * j + 1];
      x[2 * j] = rope_lo(u, v, cA[j], sA[j]);
      x[2 * j + 1] = rope_hi(u, v, cA[j], sA[j]);
    }
    if (!p.rot2) return;
  }
  const float4 cb = *reinterpret_cast<const float4*>(cos + p.a2);
  const float4 sb = *reinterpret_cast<const float4*>(sin + p.a2);
  const float cB[4] = {cb.x, cb.y, cb.z, cb.w};
  const float sB[4] = {DIR * sb.x, DIR * sb.y, DIR * sb.z, DIR * sb.w};
  if (r.interleaved) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float u = x[8 + 2 * j], v = x[9 + 2 * j];
      x[8 + 2 * j] = rope_lo(u, v, cB[j], sB[j]);
      x[9 + 2 * j] = rope_hi(u, v, cB[j], sB[j]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float c = e < 4 ? cA[e & 3] : cB[e & 3], s = e < 4 ? sA[e & 3] : sB[e & 3];
      const float u = x[e], v = x[8 + e];
      x[e] = rope_lo(u, v, c, s);
      x[8 + e] = rope_hi(u, v, c, s);
    }
  }
}

// The norm's weights as fp32 in shared memory: [0, 128) queries, [128, 256) keys (1 where there
// is none, and then no norm is applied).
__device__ __forceinline__ void load_norm_weights(const NormArgs& n, float* s_w) {
  for (int i = threadIdx.x; i < 2 * kHeadDim; i += blockDim.x) {
    const void* w = i < kHeadDim ? n.wq : n.wk;
    const int d = i & (kHeadDim - 1);
    s_w[i] = !w ? 1.f
                : n.fp32 ? static_cast<const float*>(w)[d]
                         : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[d]);
  }
}

__device__ __forceinline__ void lane_weights(const float* w, const RopeLane& p, float (&out)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 a = *reinterpret_cast<const float4*>(w + 8 * p.c1 + 4 * i);
    const float4 b = *reinterpret_cast<const float4*>(w + 8 * p.c2 + 4 * i);
    out[4 * i] = a.x, out[4 * i + 1] = a.y, out[4 * i + 2] = a.z, out[4 * i + 3] = a.w;
    out[8 + 4 * i] = b.x, out[9 + 4 * i] = b.y, out[10 + 4 * i] = b.z, out[11 + 4 * i] = b.w;
  }
}

// Norm (where `norm`) and rotation of a lane's sixteen raw values, in fp32.
__device__ __forceinline__ void norm_and_turn(const RopeArgs& r, const RopeLane& p, bool norm,
                                              const float* s_w, float eps, const float* cos,
                                              const float* sin, float (&x)[16]) {
  if (norm) {
    float w[16];
    const float rstd = row_rstd(x, eps);
    lane_weights(s_w, p, w);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = x[i] * rstd * w[i];
  }
  rope_turn<1>(r, p, cos, sin, x);
}

}  // namespace ps
