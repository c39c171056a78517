// Per-head RMS norm and rotary positions on bf16 rows of 128 dims, shared by the kernels that
// normalise and rotate (forward, backward, and the appends).
//
// Eight lanes hold one head row, sixteen dims a lane: two 16-byte chunks (8 dims each) chosen so
// that the two dims of every rotated pair sit in one lane.  Rotation then needs no exchange, the
// norm's sum of squares three shuffles, and a warp's loads are whole 128-byte half rows.
//   half layout, R rotated dims, m = R / 16: lanes l < m hold chunks (l, l + m), dims (i, i + R/2);
//     the unrotated chunks 2m .. 15 go to the other lanes, first halves then second, so that a
//     warp's loads cover whole sectors (neighbouring chunks to one lane, nothing rotated: 138 us
//     where this took 99)
//   interleaved: chunks (l, l + 8); pairs (2i, 2i + 1) never leave a chunk
// A warp takes four heads of one token at a time; q and k heads are never mixed in one item.
//
// A lane's eight pairs (u, v) of queries become rstd (u a - v b), rstd (v c + u d) with
// coefficients that hold the weights and the angles, a = w_u cos, b = w_v sin, c = w_v cos,
// d = w_u sin: formed once for all heads of a token (4 us of 34 at 24000 tokens of 8 + 1 heads),
// they leave six operations a pair.
#pragma once

#include <cuda_bf16.h>

#include "ps_device.cuh"
#include "ps_internal.h"

namespace ps {

constexpr int kHalfDim = kHeadDim / 2;

// Where a lane's two chunks are and which angles turn them.  Pairs 0..3 and 4..7 of a lane are
// rotated or not together: in the half layout pair e is (chunk 1, chunk 2) dim e, interleaved pair
// j is dims 2 j, 2 j + 1 of chunk 1, and pair 4 + j of chunk 2.
struct RopeLane {
  int c1, c2;       // chunks (dims 8 c .. 8 c + 7)
  int a1, a2;       // angles of pairs 0..3 start at a1, of 4..7 at a2
  bool rot1, rot2;  // whether pairs 0..3 and 4..7 are rotated
  bool all;         // whether every lane's are
  bool halves;      // whether every lane's chunks are eight apart
};

template <bool INTER>
__device__ __forceinline__ RopeLane rope_lane(const RopeArgs& r, int l) {
  RopeLane p;
  p.all = r.dim == kHeadDim;
  p.halves = INTER || p.all;
  if (INTER) {
    p.c1 = l;
    p.c2 = l + 8;
    p.rot1 = 8 * l < r.dim;
    p.rot2 = 8 * l + 64 < r.dim;
    p.a1 = 4 * p.c1;
    p.a2 = 4 * p.c2;
  } else {
    const int m = r.dim / 16;
    p.rot1 = p.rot2 = l < m;
    p.c1 = l < m ? l : l + m;  // 2 m + (l - m), and 8 - m chunks on
    p.c2 = l < m ? l + m : l + 8;
    p.a1 = 8 * l;
    p.a2 = 8 * l + 4;
  }
  return p;
}

__device__ __forceinline__ bool bad_rope_position(int64_t p) { return p < 0 || p >= (1ll << 31); }
__device__ __forceinline__ int32_t rope_position_flag(int64_t p) {
  return p < 0 ? PS_DEV_BAD_POS : PS_DEV_POS_RANGE;
}

// A lane's chunks as its eight (u, v) and back, two neighbouring floats to an operand of the packed
// fp32 instructions, which do two lanes of the work in one issue.  INTER: the interleaved layout (a
// template parameter: as a flag it costs a select an element).
__device__ __forceinline__ uint64_t both(uint32_t lo, uint32_t hi) {
  return pack_f32x2(__uint_as_float(lo), __uint_as_float(hi));
}
template <bool INTER>
__device__ __forceinline__ void unpack_pairs(const uint4& c1, const uint4& c2, uint64_t (&u)[4],
                                             uint64_t (&v)[4]) {
  const uint32_t a[4] = {c1.x, c1.y, c1.z, c1.w}, b[4] = {c2.x, c2.y, c2.z, c2.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (INTER) {
      const uint32_t x = i < 2 ? a[2 * i] : b[2 * i - 4], y = i < 2 ? a[2 * i + 1] : b[2 * i - 3];
      u[i] = both(x << 16, y << 16);
      v[i] = both(x & 0xffff0000u, y & 0xffff0000u);
    } else {
      u[i] = both(a[i] << 16, a[i] & 0xffff0000u);
      v[i] = both(b[i] << 16, b[i] & 0xffff0000u);
    }
  }
}
template <bool INTER>
__device__ __forceinline__ void pack_pairs(const uint64_t (&u)[4], const uint64_t (&v)[4],
                                           uint4& c1, uint4& c2) {
  uint32_t a[4], b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpack_f32x2(u[i]), y = unpack_f32x2(v[i]);
    if (INTER) {
      (i < 2 ? a[2 * i] : b[2 * i - 4]) = cvt_bf16x2(x.x, y.x);
      (i < 2 ? a[2 * i + 1] : b[2 * i - 3]) = cvt_bf16x2(x.y, y.y);
    } else {
      a[i] = cvt_bf16x2(x.x, x.y);
      b[i] = cvt_bf16x2(y.x, y.y);
    }
  }
  c1 = make_uint4(a[0], a[1], a[2], a[3]);
  c2 = make_uint4(b[0], b[1], b[2], b[3]);
}

// cos and sin of p * inv_f: reduced to [-pi/4, pi/4] in float64 (pi/2 in two parts; the first
// difference is exact, so the remainder is good to 2^-53 of pi/2 beside the product's own
// rounding), then Taylor sums, off by 2e-10 (cos, to r^10) and 2e-9 (sin, to r^9): what is added to
// the first terms in fp32, the sum in float64, so that nearly all results are the correctly rounded
// ones.  About 30 operations where the library's other rotations, through sincosf, take 240
// instructions: with 16 + 2 heads a token's 64 angles were a fifth of the forward's time (73 us at
// 32768 tokens, 64 with these).
__device__ __forceinline__ float2 cos_sin_of(double p, double inv_f) {
  const double ang = p * inv_f;
  const double shifter = 6755399441055744.0;  // 1.5 2^52: the sum's low word holds the integer
  const double t = fma(ang, 0.63661977236758134308, shifter);
  const int quadrant = __double2loint(t);
  const double k = t - shifter;
  double red = fma(-k, 1.5707963267948965580, ang);
  red = fma(-k, 6.1232339957367660359e-17, red);
  const double red2 = red * red;
  const float r2 = static_cast<float>(red2);
  float s = fmaf(r2, 1.f / 362880.f, -1.f / 5040.f);
  s = fmaf(s, r2, 1.f / 120.f);
  s = fmaf(s, r2, -1.f / 6.f) * r2;
  s = static_cast<float>(fma(red, static_cast<double>(s), red));
  float c = fmaf(r2, -1.f / 3628800.f, 1.f / 40320.f);
  c = fmaf(c, r2, -1.f / 720.f);
  c = fmaf(c, r2, 1.f / 24.f) * (r2 * r2);
  c = static_cast<float>(1.0 + fma(red2, -0.5, static_cast<double>(c)));
  const float x = (quadrant & 1) ? -s : c, y = (quadrant & 1) ? c : s;
  return (quadrant & 2) ? make_float2(-x, -y) : make_float2(x, y);
}

// The frequencies into shared memory, by the whole block.  (Every lane wants another one: read
// from the kernel's arguments, which serve one address at a time, they took 3.6 us of 37 at 24000
// tokens of 8 + 1 heads.)
__device__ __forceinline__ void load_frequencies(const RopeArgs& r, double* freq) {
  if (threadIdx.x < kHalfDim) freq[threadIdx.x] = r.inv_freq[threadIdx.x];
}

// One warp forms all angles of a token, into its own cos[64], sin[64] in shared memory.
__device__ __forceinline__ void rope_angles(const RopeArgs& r, const double* freq, int64_t pos,
                                            int lane, float* cos, float* sin) {
  __syncwarp();  // the last token's are no longer read
#pragma unroll
  for (int i = lane; i < kHalfDim; i += 32) {
    if (i >= r.dim / 2) break;
    const float2 cs = cos_sin_of(double(pos), freq[i]);
    cos[i] = cs.x * r.attn;
    sin[i] = cs.y * r.attn;
  }
  __syncwarp();
}

// The items of a warp, in order: of every `step`-th token four q heads each, then four k heads
// each; where SPLIT warps share a token, every SPLIT-th of them.  A segment is one side (q or k) of
// a token: inside it, pointers move by a constant.
struct Segment {
  int64_t tok;
  int32_t rows;  // heads from the item's first one on (fewer than four: a partial item)
  bool is_k;
};
template <int SPLIT>
struct Items {
  int64_t step;
  int32_t q0, k0;        // the warp's first q and k item
  int32_t rows_q, rows_k;  // heads from there on; <= 0: the warp has none on that side
  static constexpr int kStride = SPLIT * 4 * kHeadDim;  // elements from one item to the next

  __device__ __forceinline__ Items(int64_t step_, int sub, int hq, int hkv) : step(step_), q0(sub) {
    const int nq = (hq + 3) / 4;
    k0 = SPLIT == 1 ? 0 : (sub + SPLIT - nq % SPLIT) % SPLIT;
    rows_q = hq - 4 * q0;
    rows_k = hkv - 4 * k0;
  }
  __device__ __forceinline__ bool any() const { return rows_q > 0 || rows_k > 0; }
  __device__ __forceinline__ Segment first(int64_t tok) const {
    return rows_q > 0 ? Segment{tok, rows_q, false} : Segment{tok, rows_k, true};
  }
  // Moves on; true: to another segment.
  __device__ __forceinline__ bool next(Segment& s) const {
    s.rows -= 4 * SPLIT;
    if (s.rows > 0) return false;
    s = !s.is_k && rows_k > 0 ? Segment{s.tok, rows_k, true} : first(s.tok + step);
    return true;
  }
};

// Sum over the eight lanes of a row (every lane gets it; the same order in all of them).
__device__ __forceinline__ float row_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  return v;
}

// A product that is rounded by itself, whatever is done with it.
__device__ __forceinline__ uint64_t fmul2_rn(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// 1 / sqrt(mean(x^2) + eps) of a row held by eight lanes, fp32.
__device__ __forceinline__ float row_rstd(const uint64_t (&u)[4], const uint64_t (&v)[4],
                                          float eps) {
  uint64_t s = 0, t = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = ffma2(u[i], u[i], s);
    t = ffma2(v[i], v[i], t);
  }
  const float2 x = unpack_f32x2(fadd2(s, t));
  return rsqrtf(row_sum(x.x + x.y) * (1.f / kHeadDim) + eps);
}

// The same, with the squares summed four neighbours in turn, then halves onto halves: the order of
// a plain evaluation's sum.  Only where every lane's chunks are eight apart (p.halves: interleaved
// pairs, or heads rotated whole); half pairs of a part of the head take the other order.
template <bool INTER>
__device__ __forceinline__ float row_rstd_by_halves(const uint64_t (&u)[4], const uint64_t (&v)[4],
                                                    float eps) {
  float part[2][2];  // [chunk][first or second four dims]
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float2 a, b;
      if (INTER) {
        const float2 x = unpack_f32x2(u[2 * c + h]), y = unpack_f32x2(v[2 * c + h]);
        a = make_float2(x.x, y.x), b = make_float2(x.y, y.y);
      } else {
        a = unpack_f32x2(c ? v[2 * h] : u[2 * h]);
        b = unpack_f32x2(c ? v[2 * h + 1] : u[2 * h + 1]);
      }
      part[c][h] = fmaf(b.y, b.y, fmaf(b.x, b.x, fmaf(a.y, a.y, a.x * a.x)));
    }
  float s0 = part[0][0] + part[1][0], s1 = part[0][1] + part[1][1];
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
    s0 += __shfl_xor_sync(0xffffffffu, s0, o);
    s1 += __shfl_xor_sync(0xffffffffu, s1, o);
  }
  return rsqrtf((s0 + s1) * (1.f / kHeadDim) + eps);
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

// A lane's weights as pairs.
template <bool INTER>
__device__ __forceinline__ void lane_weights(const float* w, const RopeLane& p, uint64_t (&wu)[4],
                                             uint64_t (&wv)[4]) {
  uint64_t x[8];  // both chunks
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(
        w + 8 * (i < 2 ? p.c1 : p.c2) + 4 * (i & 1));
    x[2 * i] = y.x, x[2 * i + 1] = y.y;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (INTER) {
      const float2 a = unpack_f32x2(x[2 * i]), b = unpack_f32x2(x[2 * i + 1]);
      wu[i] = pack_f32x2(a.x, b.x);
      wv[i] = pack_f32x2(a.y, b.y);
    } else {
      wu[i] = x[i];
      wv[i] = x[4 + i];
    }
  }
}

// A lane's cosines and sines (1 and 0 where a pair is not rotated).
__device__ __forceinline__ void lane_angles(const RopeLane& p, const float* cos, const float* sin,
                                            uint64_t (&c)[4], uint64_t (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint64_t one = pack_f32x2(1.f, 1.f);
    ulonglong2 x = make_ulonglong2(one, one), y = make_ulonglong2(0, 0);
    if (i ? p.rot2 : p.rot1) {
      x = *reinterpret_cast<const ulonglong2*>(cos + (i ? p.a2 : p.a1));
      y = *reinterpret_cast<const ulonglong2*>(sin + (i ? p.a2 : p.a1));
    }
    c[2 * i] = x.x, c[2 * i + 1] = x.y;
    s[2 * i] = y.x, s[2 * i + 1] = y.y;
  }
}

// What turns a lane's pairs of one token's heads.  Of queries: the weights (ones where there is no
// norm) are in the angles, and b is negative.  Of normalised keys: a and c are the weights of u and
// v, b and d cosines and sines.
struct RowCoef {
  uint64_t a[4], b[4], c[4], d[4];
};
template <bool INTER>
__device__ __forceinline__ void row_coef(const RopeLane& p, bool key, const float* w,
                                         const float* cos, const float* sin, RowCoef& k) {
  if (key) {
    lane_angles(p, cos, sin, k.b, k.d);
    lane_weights<INTER>(w, p, k.a, k.c);
    return;
  }
  uint64_t c[4], s[4], wu[4], wv[4];
  lane_angles(p, cos, sin, c, s);
  lane_weights<INTER>(w, p, wu, wv);
  const uint64_t minus = pack_f32x2(-1.f, -1.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    k.a[i] = fmul2(wu[i], c[i]);
    k.b[i] = fmul2(fmul2(wv[i], s[i]), minus);
    k.c[i] = fmul2(wv[i], c[i]);
    k.d[i] = fmul2(wu[i], s[i]);
  }
}

// Normalised keys are rounded step by step, x rstd, times w, the rotation's products and their sum,
// as the formula's plain evaluation does: a 4-bit store turns a last bit that differs into a whole
// code at times (of 9 million codes ten with folded coefficients, none or one so), and a token has
// few key heads.  ALL: every pair is rotated (asked per pair it costs
// an eighth of the forward's instructions; a pair that is not must not see the other's infinity).
template <bool ALL>
__device__ __forceinline__ void norm_and_turn_key(const RopeLane& p, const RowCoef& k, uint64_t r2,
                                                  uint64_t (&u)[4], uint64_t (&v)[4]) {
  const uint64_t minus = pack_f32x2(-1.f, -1.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint64_t x = fmul2_rn(fmul2_rn(u[i], r2), k.a[i]);
    uint64_t y = fmul2_rn(fmul2_rn(v[i], r2), k.c[i]);
    if (ALL || (i < 2 ? p.rot1 : p.rot2)) {
      const uint64_t xs = fmul2_rn(x, k.d[i]), ys = fmul2_rn(y, k.d[i]);
      x = ffma2(ys, minus, fmul2_rn(x, k.b[i]));
      y = fadd2(fmul2_rn(y, k.b[i]), xs);
    }
    u[i] = x;
    v[i] = y;
  }
}
template <bool ALL>
__device__ __forceinline__ void norm_and_turn_query(const RopeLane& p, const RowCoef& k,
                                                    uint64_t r2, uint64_t (&u)[4],
                                                    uint64_t (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint64_t x = fmul2(u[i], k.a[i]), y = fmul2(v[i], k.c[i]);
    if (ALL || (i < 2 ? p.rot1 : p.rot2)) {
      x = ffma2(v[i], k.b[i], x);
      y = ffma2(u[i], k.d[i], y);
    }
    u[i] = fmul2(x, r2);
    v[i] = fmul2(y, r2);
  }
}

// Norm (where `norm`) and rotation of a lane's pairs in place, fp32.
template <bool INTER>
__device__ __forceinline__ void norm_and_turn(const RopeLane& p, bool norm, bool key,
                                              const RowCoef& k, float eps, uint64_t (&u)[4],
                                              uint64_t (&v)[4]) {
  if (norm) {
    const float rstd =
        key && p.halves ? row_rstd_by_halves<INTER>(u, v, eps) : row_rstd(u, v, eps);
    const uint64_t r2 = pack_f32x2(rstd, rstd);
    if (key) {
      if (p.all) norm_and_turn_key<true>(p, k, r2, u, v);
      else norm_and_turn_key<false>(p, k, r2, u, v);
    } else {
      if (p.all) norm_and_turn_query<true>(p, k, r2, u, v);
      else norm_and_turn_query<false>(p, k, r2, u, v);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < 2 ? p.rot1 : p.rot2) {
        const float2 x = unpack_f32x2(u[i]), y = unpack_f32x2(v[i]);
        const float2 a = unpack_f32x2(k.a[i]), b = unpack_f32x2(k.b[i]);
        const float2 c = unpack_f32x2(k.c[i]), d = unpack_f32x2(k.d[i]);
        u[i] = pack_f32x2(rope_lo(x.x, y.x, a.x, -b.x), rope_lo(x.y, y.y, a.y, -b.y));
        v[i] = pack_f32x2(rope_hi(x.x, y.x, c.x, d.x), rope_hi(x.y, y.y, c.y, d.y));
      }
  }
}

}  // namespace ps
