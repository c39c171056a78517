// Decode attention over the 4-bit store, sm_100a.
//
// The query of sequence b at position p attends its visible rows (prefix rows, then the window's
// ring slots), each standing for m_g + s_g u_d in its two groups g of 64 dims:
//   S_k = sum_g s_kg (sum_{d in g} q_d u_kd) + m_kg sum_{d in g} q_d
//   o_d = sum_k p_k m_kg + sum_k (p_k s_kg) u_kd,  p = softmax(scale S)
// A row is 144 bytes (64 of K, 64 of V, 16 of scales and minima), so the kernel is bound by HBM
// once the codes can be fed to the tensor cores cheaply:
//  * a code u enters the matrix product as the bf16 number 128 + u, which is its four bits or-ed
//    into 0x4300: one shift and one lop a pair, nothing rounded.  The 128s are taken off exactly:
//    the score accumulators start at -128 sum q, and a product with a matrix of -128s sums the
//    same rounded weights that the codes are multiplied by
//  * the dims of a row are stored so that one 16-byte load gives a lane the words of a whole
//    K fragment row; which dim goes to which position of the product does not matter as long as
//    the query's fragment agrees
//  * scales multiply scores (K) and weights (V), never the 128 codes of a row
// Eight query heads of a KV head share a row's bytes (the columns of the products).
//
// Work: a unit is (sequence, KV head).  With fewer units than block slots, one wave of blocks takes
// equal shares of all visible rows back to back (a share may span units; a unit's pieces are
// combined by merge_q4_kernel); otherwise one block a unit.  Inside a block every warp streams its
// own 32-row tiles (every eighth) through three stages of shared memory with bulk copies of exactly
// the rows it needs: no warp waits for another until the piece ends.
#include <cuda_bf16.h>
#include <math.h>

#include "ps_device.cuh"
#include "ps_internal.h"
#include "ps_ranges.cuh"
#include "ps_store.cuh"

namespace ps {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kBlocksPerSm = 2;
constexpr int kTile = 32;  // rows of a warp's tile
constexpr int kStages = 3;
constexpr int kStageBytes = kTile * (2 * kQ4RowBytes + kQ4RecordBytes);
constexpr int kWarpBytes = kStages * kStageBytes;
constexpr int kSmemBytes = kWarps * kWarpBytes;
static_assert(kWarpBytes >= (kHeadDim + 2) * kMaxGroup * 4, "a warp's result fits its stages");
constexpr int kMinRowsPerBlock = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A running maximum is moved only when a score passes it by more than this (in log2): weights
// then stay below 2^8, and a row of tiles rarely rescales its accumulators.
constexpr float kMaxSlack = 8.f;

struct DecodeQ4Args {
  const __nv_bfloat16* q;
  const int64_t* pos;
  __nv_bfloat16* out;
  float* lse;
  float* ws_o;    // [units + grid, 8, D] normalised pieces, or NULL: one block a unit
  float* ws_lse;  // [units + grid, 8] base-2 lse of each piece
  int32_t* status;
  int32_t batch, hq, hkv, group;
  float scale_log2;
  StoreArgs store;
};

__device__ __forceinline__ int64_t visible_rows(const DecodeQ4Args& a, int64_t p) {
  if (p < 0 || p >= (1ll << 31) || (a.store.linear && p >= a.store.lp)) return 0;
  const int64_t n = p + 1, cap = (int64_t)a.store.lp + (a.store.linear ? 0 : a.store.w);
  return n < cap ? n : cap;
}

// x / y for 0 <= x, 0 < y, in 32 bits where both fit (the case in practice).
__device__ __forceinline__ int64_t div_nonneg(int64_t x, int64_t y) {
  if ((x | y) < (int64_t(1) << 32)) return uint32_t(x) / uint32_t(y);
  return x / y;
}

// Rows of sequences before lane's chunk, and of all sequences; a chunk is `per` sequences.
struct RowScan {
  int32_t per;
  int64_t before, mine, total;
};
__device__ __forceinline__ RowScan scan_rows(const DecodeQ4Args& a, int lane, bool flag) {
  RowScan s;
  s.per = (a.batch + 31) / 32;
  s.mine = 0;
  for (int i = 0; i < s.per; ++i) {
    const int b = lane * s.per + i;
    if (b >= a.batch) break;
    const int64_t p = a.pos[b], n = visible_rows(a, p);
    s.mine += n;
    if (flag && n == 0 && a.status) atomicOr(a.status, p < 0 ? PS_DEV_BAD_POS : PS_DEV_POS_RANGE);
  }
  int64_t v = s.mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += u;
  }
  s.before = v - s.mine;
  s.total = __shfl_sync(0xffffffffu, v, 31);
  return s;
}

// Rows of one sequence that a warp's lane 0 copies, and where they are.
struct Sequence {
  int64_t p, n, pre;  // position, visible rows, visible prefix rows
  int32_t b, h;
};

// Copies visible rows [v, v + cnt) of a unit into a stage; returns (all lanes) the mask of rows
// that are there (a bad block table entry leaves its rows out).  Lane 0 works.
__device__ __forceinline__ void load_tile(const DecodeQ4Args& a, const Sequence& sq, int64_t v,
                                          int cnt, uint8_t* stage, uint64_t* bar,
                                          uint32_t* mask) {
  const StoreArgs& st = a.store;
  uint32_t tx = 0, there = 0;
  for (int done = 0; done < cnt;) {
    const int64_t x = v + done;
    const bool ring = x >= sq.pre;
    // prefix position x, or the window's (x - pre)-th oldest
    const int64_t row = ring ? mod_nonneg(sq.p + 1 - (sq.n - x) - st.lp, st.w) : x;
    int64_t run = cnt - done;
    const int64_t left = ring ? st.w - row : sq.pre - x;
    if (run > left) run = left;
    int64_t at;  // row in its array
    const int arr = (ring && !st.table) ? 1 : 0;
    bool ok = true;
    if (st.table) {
      const int64_t in_block = row & 63;
      if (run > 64 - in_block) run = 64 - in_block;
      const int32_t blk =
          st.table[(int64_t)sq.b * st.table_stride + (ring ? st.pre_blocks : 0) + (row >> 6)];
      ok = blk >= 0 && blk < st.n_blocks;
      at = ((int64_t)blk * a.hkv + sq.h) * 64 + in_block;
    } else {
      at = ((int64_t)sq.b * a.hkv + sq.h) * (ring ? st.w : st.lp) + row;
    }
    const uint32_t n = static_cast<uint32_t>(run);
    if (ok) {
      bulk_load(stage + done * kQ4RowBytes, st.k[arr] + at * kQ4RowBytes, n * kQ4RowBytes, bar);
      bulk_load(stage + (kTile + done) * kQ4RowBytes, st.v[arr] + at * kQ4RowBytes,
                n * kQ4RowBytes, bar);
      bulk_load(stage + 2 * kTile * kQ4RowBytes + done * kQ4RecordBytes,
                st.s[arr] + at * kQ4RecordBytes, n * kQ4RecordBytes, bar);
      tx += n * (2 * kQ4RowBytes + kQ4RecordBytes);
      there |= (n == 32 ? 0xffffffffu : ((1u << n) - 1u)) << done;
    } else if (a.status) {
      atomicOr(a.status, PS_DEV_POS_RANGE);
    }
    done += static_cast<int>(n);
  }
  *mask = there;
  mbar_arrive_expect_tx(bar, tx);
}

// D = A B + C
__device__ __forceinline__ void mma_bf16_c(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                           uint32_t a3, uint32_t b0, uint32_t b1, float c0,
                                           float c1, float c2, float c3) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// Codes i (low half) and i + 4 (high half) of a word's eight as the bf16 pair 128 + u.
template <int I>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  uint32_t r;
  asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xea;" : "=r"(r) : "r"(w >> (4 * I)));
  return r;
}

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// One warp's running softmax and accumulators over the heads (2 t, 2 t + 1) of its lane's t.
struct State {
  float m[2], l[2];
  float o[8][4];    // tile 4 g + i: dims 64 g + 8 (lane / 4) + 2 i + {0, 1}, heads 2 t + {0, 1}
  float off[2][4];  // -128 sum of a group's weights (rows alike)
  float mn[2][2];   // sum p m of a group, over this lane's rows
};

// The tile row of product row r (0..7): even rows first, so that the four rows a lane's V words
// come from fall into different halves of the shared memory banks.
__device__ __forceinline__ int tile_row(int r) { return (r & 1) ? 4 + ((r >> 1) ^ 1) : r >> 1; }

__global__ void __launch_bounds__(kThreads, kBlocksPerSm) decode_q4_kernel(const DecodeQ4Args a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t s_full[kWarps][kStages];
  __shared__ uint32_t s_mask[kWarps][kStages];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g8 = lane >> 2, t4 = lane & 3;
  uint8_t* mine = smem + warp * kWarpBytes;
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&s_full[warp][s], 1);
    fence_mbar_init();
  }
  __syncwarp();
  pdl_wait();
  pdl_trigger();

  // ------------------------------------------------ this block's share of the rows
  Sequence sq;
  int64_t off = 0, left;  // first row in the current unit, rows of the share still to do
  if (a.ws_o) {
    const RowScan sc = scan_rows(a, lane, blockIdx.x == 0 && warp == 0);
    const int64_t total = sc.total * a.hkv;
    const int64_t t0 = div_nonneg(total * blockIdx.x, gridDim.x);
    left = div_nonneg(total * (blockIdx.x + 1), gridDim.x) - t0;
    if (left <= 0) return;
    // the chunk of sequences holding row t0, then the sequence in it
    const uint32_t has = __ballot_sync(0xffffffffu, a.hkv * sc.before <= t0 &&
                                                        t0 < a.hkv * (sc.before + sc.mine));
    const int src = __ffs(has) - 1;
    int64_t rest = t0 - a.hkv * __shfl_sync(0xffffffffu, sc.before, src);
    sq.b = src * sc.per;
    while (true) {
      sq.p = a.pos[sq.b];
      sq.n = visible_rows(a, sq.p);
      if (rest < a.hkv * sq.n) break;
      rest -= a.hkv * sq.n;
      ++sq.b;
    }
    sq.h = static_cast<int32_t>(div_nonneg(rest, sq.n));
    off = rest - sq.h * sq.n;
  } else {
    sq.b = blockIdx.x / a.hkv;
    sq.h = blockIdx.x % a.hkv;
    sq.p = a.pos[sq.b];
    sq.n = left = visible_rows(a, sq.p);
    if (left == 0 && threadIdx.x == 0 && a.status)
      atomicOr(a.status, sq.p < 0 ? PS_DEV_BAD_POS : PS_DEV_POS_RANGE);
  }

  int issued = 0, used = 0;  // tiles of this warp so far: stage i % kStages, phase i / kStages
  while (true) {
    sq.pre = sq.n < a.store.lp ? sq.n : a.store.lp;
    const int64_t piece = left < sq.n - off ? left : sq.n - off;
    const int tiles = static_cast<int>((piece + kTile - 1) / kTile);
    const int my_tiles = tiles > warp ? (tiles - warp + kWarps - 1) / kWarps : 0;
    auto issue = [&](int i) {  // this warp's i-th tile of the piece
      if (lane == 0) {
        const int64_t r = (int64_t)(warp + kWarps * i) * kTile;
        const int cnt = static_cast<int>(piece - r < kTile ? piece - r : kTile);
        const int s = issued % kStages;
        load_tile(a, sq, off + r, cnt, mine + s * kStageBytes, &s_full[warp][s],
                  &s_mask[warp][s]);
      }
      ++issued;
    };
    for (int i = 0; i < my_tiles && i < kStages; ++i) issue(i);

    // the query's fragments: head g8, blocks 2 t and 2 t + 1 of both groups
    uint4 qf[2][2];
    float qs[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      qf[g][0] = qf[g][1] = make_uint4(0, 0, 0, 0);
      if (g8 < a.group) {
        const uint4* src = reinterpret_cast<const uint4*>(
            a.q + ((int64_t)sq.b * a.hq + sq.h * a.group + g8) * kHeadDim + 64 * g + 16 * t4);
        qf[g][0] = src[0];
        qf[g][1] = src[1];
      }
      const uint32_t w[8] = {qf[g][0].x, qf[g][0].y, qf[g][0].z, qf[g][0].w,
                             qf[g][1].x, qf[g][1].y, qf[g][1].z, qf[g][1].w};
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) v += lo_f(w[i]) + hi_f(w[i]);
      v += __shfl_xor_sync(0xffffffffu, v, 1);
      qs[g] = v + __shfl_xor_sync(0xffffffffu, v, 2);
    }
    float Q[2][2];  // sum of a group's query dims, heads 2 t + e
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int e = 0; e < 2; ++e) Q[g][e] = __shfl_sync(0xffffffffu, qs[g], 4 * (2 * t4 + e));

    State st;
    st.m[0] = st.m[1] = -INFINITY;
    st.l[0] = st.l[1] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) st.o[i][0] = st.o[i][1] = st.o[i][2] = st.o[i][3] = 0.f;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      st.off[g][0] = st.off[g][1] = st.off[g][2] = st.off[g][3] = 0.f;
      st.mn[g][0] = st.mn[g][1] = 0.f;
    }

    const int kr = tile_row(g8);  // this lane's K rows: kr, kr + 8
    for (int i = 0; i < my_tiles; ++i) {
      const int s = used % kStages;
      if (!__all_sync(0xffffffffu, mbar_wait(&s_full[warp][s], (used / kStages) & 1, a.status))) {
        // given up on (and flagged): see the other copies in flight to their end as well
        for (++used; used < issued; ++used)
          mbar_wait(&s_full[warp][used % kStages], (used / kStages) & 1, a.status);
        break;
      }
      ++used;
      const uint8_t* stage = mine + s * kStageBytes;
      const uint8_t* rec = stage + 2 * kTile * kQ4RowBytes;
      const uint32_t mask = s_mask[warp][s];
      // ---------------------------------------- scores of 2 x 16 rows
      float x[2][4];
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        const int r0 = 16 * blk + kr, r1 = r0 + 8;
        const uint4 w0 = *reinterpret_cast<const uint4*>(stage + r0 * kQ4RowBytes + 16 * t4);
        const uint4 w1 = *reinterpret_cast<const uint4*>(stage + r1 * kQ4RowBytes + 16 * t4);
        const uint2 c0 = *reinterpret_cast<const uint2*>(rec + r0 * kQ4RecordBytes);
        const uint2 c1 = *reinterpret_cast<const uint2*>(rec + r1 * kQ4RecordBytes);
        float acc[2][4];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const float n0 = -128.f * Q[g][0], n1 = -128.f * Q[g][1];
          const uint32_t a0 = g ? w0.y : w0.x, a1 = g ? w1.y : w1.x;
          const uint32_t b0 = g ? w0.w : w0.z, b1 = g ? w1.w : w1.z;
          mma_bf16_c(acc[g], code_pair<0>(a0), code_pair<0>(a1), code_pair<1>(a0),
                     code_pair<1>(a1), qf[g][0].x, qf[g][0].y, n0, n1, n0, n1);
          mma_bf16_16816(acc[g], code_pair<2>(a0), code_pair<2>(a1), code_pair<3>(a0),
                         code_pair<3>(a1), qf[g][0].z, qf[g][0].w);
          mma_bf16_16816(acc[g], code_pair<0>(b0), code_pair<0>(b1), code_pair<1>(b0),
                         code_pair<1>(b1), qf[g][1].x, qf[g][1].y);
          mma_bf16_16816(acc[g], code_pair<2>(b0), code_pair<2>(b1), code_pair<3>(b0),
                         code_pair<3>(b1), qf[g][1].z, qf[g][1].w);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float s0 = lo_f(c0.x) * acc[0][e], s1 = lo_f(c1.x) * acc[0][2 + e];
          s0 = fmaf(lo_f(c0.y), acc[1][e], s0);
          s1 = fmaf(lo_f(c1.y), acc[1][2 + e], s1);
          s0 = fmaf(hi_f(c0.x), Q[0][e], s0);
          s1 = fmaf(hi_f(c1.x), Q[0][e], s1);
          s0 = fmaf(hi_f(c0.y), Q[1][e], s0);
          s1 = fmaf(hi_f(c1.y), Q[1][e], s1);
          x[blk][e] = s0 * a.scale_log2;
          x[blk][2 + e] = s1 * a.scale_log2;
        }
      }
      if (mask != 0xffffffffu) {
#pragma unroll
        for (int blk = 0; blk < 2; ++blk)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (!((mask >> (16 * blk + kr + (j >> 1) * 8)) & 1u)) x[blk][j] = -INFINITY;
      }
      // ---------------------------------------- running maximum
      float mx[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[e] = fmaxf(fmaxf(x[0][e], x[0][2 + e]), fmaxf(x[1][e], x[1][2 + e]));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], o));
      }
      if (__any_sync(0xffffffffu, mx[0] > st.m[0] + kMaxSlack || mx[1] > st.m[1] + kMaxSlack)) {
        float c[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mn = fmaxf(st.m[e], mx[e]);
          c[e] = st.m[e] == -INFINITY ? 0.f : fast_exp2(st.m[e] - mn);
          st.m[e] = mn;
          st.l[e] *= c[e];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            st.off[g][e] *= c[e];
            st.off[g][2 + e] *= c[e];
            st.mn[g][e] *= c[e];
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          st.o[j][0] *= c[0];
          st.o[j][1] *= c[1];
          st.o[j][2] *= c[0];
          st.o[j][3] *= c[1];
        }
      }
      const float ref0 = st.m[0] == -INFINITY ? 0.f : st.m[0];
      const float ref1 = st.m[1] == -INFINITY ? 0.f : st.m[1];
      // ---------------------------------------- weights and values
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        const int r0 = 16 * blk + kr, r1 = r0 + 8;
        uint2 c0 = *reinterpret_cast<const uint2*>(rec + r0 * kQ4RecordBytes + 8);
        uint2 c1 = *reinterpret_cast<const uint2*>(rec + r1 * kQ4RecordBytes + 8);
        if (mask != 0xffffffffu) {  // what an absent row's record holds may be a NaN
          if (!((mask >> r0) & 1u)) c0 = make_uint2(0, 0);
          if (!((mask >> r1) & 1u)) c1 = make_uint2(0, 0);
        }
        float p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] = fast_exp2(x[blk][j] - ((j & 1) ? ref1 : ref0));
        st.l[0] += p[0] + p[2];
        st.l[1] += p[1] + p[3];
        // this lane's V words: rows of the product's k = 2 t, 2 t + 1, 2 t + 8, 2 t + 9
        const uint8_t* vb = stage + (kTile + 16 * blk) * kQ4RowBytes + 8 * g8;
        const int va = t4, vc = 4 + (t4 ^ 1);
        const uint2 v0 = *reinterpret_cast<const uint2*>(vb + va * kQ4RowBytes);
        const uint2 v1 = *reinterpret_cast<const uint2*>(vb + vc * kQ4RowBytes);
        const uint2 v2 = *reinterpret_cast<const uint2*>(vb + (va + 8) * kQ4RowBytes);
        const uint2 v3 = *reinterpret_cast<const uint2*>(vb + (vc + 8) * kQ4RowBytes);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const uint32_t k0 = g ? c0.y : c0.x, k1 = g ? c1.y : c1.x;
          // a weight times its row's scale, rounded to bf16: the tensor cores' operand type
          const uint32_t b0 = movmatrix_trans(cvt_bf16x2(p[0] * lo_f(k0), p[1] * lo_f(k0)));
          const uint32_t b1 = movmatrix_trans(cvt_bf16x2(p[2] * lo_f(k1), p[3] * lo_f(k1)));
          st.mn[g][0] = fmaf(p[0], hi_f(k0), fmaf(p[2], hi_f(k1), st.mn[g][0]));
          st.mn[g][1] = fmaf(p[1], hi_f(k0), fmaf(p[3], hi_f(k1), st.mn[g][1]));
          const uint32_t m128 = 0xc300c300u;  // -128, -128
          mma_bf16_16816(st.off[g], m128, m128, m128, m128, b0, b1);
          const uint32_t x0 = g ? v0.y : v0.x, x1 = g ? v1.y : v1.x;
          const uint32_t x2 = g ? v2.y : v2.x, x3 = g ? v3.y : v3.x;
          const uint32_t e0 = __byte_perm(x0, x1, 0x5410), f0 = __byte_perm(x0, x1, 0x7632);
          const uint32_t e1 = __byte_perm(x2, x3, 0x5410), f1 = __byte_perm(x2, x3, 0x7632);
          mma_bf16_16816(st.o[4 * g + 0], code_pair<0>(e0), code_pair<0>(f0), code_pair<0>(e1),
                         code_pair<0>(f1), b0, b1);
          mma_bf16_16816(st.o[4 * g + 1], code_pair<1>(e0), code_pair<1>(f0), code_pair<1>(e1),
                         code_pair<1>(f1), b0, b1);
          mma_bf16_16816(st.o[4 * g + 2], code_pair<2>(e0), code_pair<2>(f0), code_pair<2>(e1),
                         code_pair<2>(f1), b0, b1);
          mma_bf16_16816(st.o[4 * g + 3], code_pair<3>(e0), code_pair<3>(f0), code_pair<3>(e1),
                         code_pair<3>(f1), b0, b1);
        }
      }
      __syncwarp();  // every lane has read the stage
      if (i + kStages < my_tiles) issue(i + kStages);
    }

    // ------------------------------------------------ combine the warps, write the piece
    // every copy of this warp has landed and been read (or given up on): its stages hold its
    // result now, [8 heads][128], then m[8], l[8]
    float* res = reinterpret_cast<float*>(mine);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        st.l[e] += __shfl_xor_sync(0xffffffffu, st.l[e], o);
        st.mn[0][e] += __shfl_xor_sync(0xffffffffu, st.mn[0][e], o);
        st.mn[1][e] += __shfl_xor_sync(0xffffffffu, st.mn[1][e], o);
      }
      float* dst = res + (2 * t4 + e) * kHeadDim + 8 * g8;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const float add = st.off[g][e] + st.mn[g][e];
        float4 y0, y1;
        y0.x = st.o[4 * g + 0][e] + add, y0.y = st.o[4 * g + 0][2 + e] + add;
        y0.z = st.o[4 * g + 1][e] + add, y0.w = st.o[4 * g + 1][2 + e] + add;
        y1.x = st.o[4 * g + 2][e] + add, y1.y = st.o[4 * g + 2][2 + e] + add;
        y1.z = st.o[4 * g + 3][e] + add, y1.w = st.o[4 * g + 3][2 + e] + add;
        reinterpret_cast<float4*>(dst + 64 * g)[0] = y0;
        reinterpret_cast<float4*>(dst + 64 * g)[1] = y1;
      }
      if (g8 == 0) {
        res[kMaxGroup * kHeadDim + 2 * t4 + e] = st.m[e];
        res[kMaxGroup * kHeadDim + kMaxGroup + 2 * t4 + e] = st.l[e];
      }
    }
    __syncthreads();
    {
      const int head = warp;  // eight warps, eight heads; lane: dims 4 lane .. 4 lane + 3
      if (head < a.group) {
        float ml[kWarps], M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          ml[w] = reinterpret_cast<float*>(smem + w * kWarpBytes)[kMaxGroup * kHeadDim + head];
          M = fmaxf(M, ml[w]);
        }
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float* r = reinterpret_cast<float*>(smem + w * kWarpBytes);
          const float f = ml[w] == -INFINITY ? 0.f : fast_exp2(ml[w] - M);
          const float lw = r[kMaxGroup * kHeadDim + kMaxGroup + head];
          if (lw == 0.f) continue;  // no row of this warp counted
          const float4 y = reinterpret_cast<const float4*>(r + head * kHeadDim)[lane];
          L = fmaf(f, lw, L);
          acc.x = fmaf(f, y.x, acc.x);
          acc.y = fmaf(f, y.y, acc.y);
          acc.z = fmaf(f, y.z, acc.z);
          acc.w = fmaf(f, y.w, acc.w);
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        const float lse2 = L == 0.f ? -INFINITY : M + log2f(L);
        acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
        if (a.ws_o) {
          // unique per (unit, block): both only grow along the rows
          const int64_t slot = ((int64_t)sq.b * a.hkv + sq.h + blockIdx.x) * kMaxGroup + head;
          reinterpret_cast<float4*>(a.ws_o + slot * kHeadDim)[lane] = acc;
          if (lane == 0) a.ws_lse[slot] = lse2;
        } else {
          const int64_t row = (int64_t)sq.b * a.hq + sq.h * a.group + head;
          reinterpret_cast<uint2*>(a.out + row * kHeadDim)[lane] =
              make_uint2(cvt_bf16x2(acc.x, acc.y), cvt_bf16x2(acc.z, acc.w));
          if (a.lse && lane == 0) a.lse[row] = lse2 * kLn2;
        }
      }
    }
    left -= piece;
    if (left <= 0) break;
    // next unit that has rows; its copies overwrite the results just read
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    off = 0;
    if (++sq.h == a.hkv) {
      sq.h = 0;
      do {
        sq.p = a.pos[++sq.b];
        sq.n = visible_rows(a, sq.p);
      } while (sq.n == 0);
    }
  }
}

// Combines the pieces of one (sequence, query head), one warp each: block c of the decode owned
// the rows [total c / grid, total (c + 1) / grid) and stored its piece of unit u at slot u + c, so
// which pieces exist follows from the positions alone.  Lane i owns dims 4 i .. 4 i + 3.
__global__ void __launch_bounds__(128)
    merge_q4_kernel(const DecodeQ4Args a, int32_t grid) {
  const int lane = threadIdx.x & 31;
  const int64_t bh = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const bool live = bh < (int64_t)a.batch * a.hq;
  const int b = live ? static_cast<int>(bh / a.hq) : 0;
  const int head = live ? static_cast<int>(bh % a.hq) : 0;
  const int h = head / a.group, hh = head % a.group;
  const RowScan sc = scan_rows(a, lane, false);
  const int64_t total = sc.total * a.hkv;
  const int src = b / sc.per;
  int64_t first = __shfl_sync(0xffffffffu, sc.before, src);
  for (int i = src * sc.per; i < b; ++i) first += visible_rows(a, a.pos[i]);
  const int64_t n = visible_rows(a, a.pos[b]);
  const int64_t unit = (int64_t)b * a.hkv + h;
  int c_lo = 1, c_hi = 0;
  if (n > 0) {
    const int64_t pu = a.hkv * first + h * n;
    c_lo = static_cast<int>(div_nonneg((pu + 1) * grid - 1, total));
    c_hi = static_cast<int>(div_nonneg((pu + n) * grid - 1, total));
  }
  pdl_trigger();
  pdl_wait();
  if (!live) return;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float M = -INFINITY, L = 0.f;
  for (int c0 = c_lo; c0 <= c_hi; c0 += 4) {
    float lv[4];
    float4 ov[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = c0 + k;
      lv[k] = -INFINITY;
      ov[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      // with fewer rows than blocks some blocks own none and wrote no piece
      if (c <= c_hi && (total >= grid || total * c / grid != total * (c + 1) / grid)) {
        const int64_t slot = (unit + c) * kMaxGroup + hh;
        lv[k] = a.ws_lse[slot];
        ov[k] = reinterpret_cast<const float4*>(a.ws_o + slot * kHeadDim)[lane];
      }
    }
    const float Mn = fmaxf(M, fmaxf(fmaxf(lv[0], lv[1]), fmaxf(lv[2], lv[3])));
    const float ref = Mn == -INFINITY ? 0.f : Mn;
    const float f = fast_exp2(M - ref);
    L *= f;
    acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float e = fast_exp2(lv[k] - ref);
      L += e;
      acc.x = fmaf(e, ov[k].x, acc.x);
      acc.y = fmaf(e, ov[k].y, acc.y);
      acc.z = fmaf(e, ov[k].z, acc.z);
      acc.w = fmaf(e, ov[k].w, acc.w);
    }
    M = Mn;
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  reinterpret_cast<uint2*>(a.out + bh * kHeadDim)[lane] =
      make_uint2(cvt_bf16x2(acc.x * inv, acc.y * inv), cvt_bf16x2(acc.z * inv, acc.w * inv));
  if (a.lse && lane == 0) a.lse[bh] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

int blocks_per_sm() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  if (cached[dev] == 0) {
    int occ = 0;
    if (cudaFuncSetAttribute(decode_q4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmemBytes) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, decode_q4_kernel, kThreads,
                                                      kSmemBytes) != cudaSuccess ||
        occ < 1)
      occ = 1;
    cached[dev] = occ < kBlocksPerSm ? occ : kBlocksPerSm;
  }
  return cached[dev];
}

// Blocks of the one-wave schedule, or 0 for one block a unit.
int64_t share_grid(int64_t batch, int32_t hkv, int64_t max_keys) {
  const int64_t units = batch * hkv;
  const int64_t slots = (int64_t)sm_count() * blocks_per_sm();
  if (units >= slots) return 0;
  int64_t g = units * ((max_keys + kMinRowsPerBlock - 1) / kMinRowsPerBlock);
  if (g >= slots) {
    g = slots;
    // a multiple of the unit count that fills 5/6 of the slots: equally long units then split on
    // their own borders, and no block changes unit midway
    const int64_t even = units * (slots / units);
    if (even * 6 >= slots * 5) g = even;
  }
  return g < 1 ? 1 : g;
}

}  // namespace

size_t decode_q4_workspace_bytes(int64_t batch, int32_t hkv, int64_t max_keys) {
  const int64_t g = share_grid(batch, hkv, max_keys);
  if (g == 0 || batch == 0) return 0;
  const size_t slots = size_t(batch * hkv + g) * kMaxGroup;
  return slots * (kHeadDim + 1) * sizeof(float);
}

int launch_decode_q4(const DecodeQ4Launch& l, cudaStream_t stream) {
  const int64_t units = l.batch * l.hkv;
  const int64_t g = share_grid(l.batch, l.hkv, (int64_t)l.store.lp + l.store.w);
  const int64_t grid = g ? g : units;
  if (grid > 0x7fffffff) return fail(PS_ERR_UNSUPPORTED, "decode grid too large");
  DecodeQ4Args a;
  a.q = static_cast<const __nv_bfloat16*>(l.q);
  a.pos = l.pos;
  a.out = static_cast<__nv_bfloat16*>(l.out);
  a.lse = l.lse;
  a.ws_o = g ? static_cast<float*>(l.workspace) : nullptr;
  a.ws_lse = g ? a.ws_o + size_t(units + g) * kMaxGroup * kHeadDim : nullptr;
  a.status = l.status;
  a.batch = static_cast<int32_t>(l.batch);
  a.hq = l.hq;
  a.hkv = l.hkv;
  a.group = l.hq / l.hkv;
  a.scale_log2 = l.scale * kLog2e;
  a.store = l.store;
  PS_TRY(check_cuda(launch_pdl(decode_q4_kernel, dim3(static_cast<unsigned>(grid)),
                               dim3(kThreads), kSmemBytes, stream, a),
                    "decode_q4_kernel launch"));
  if (!g) return PS_OK;
  return check_cuda(
      launch_pdl(merge_q4_kernel, dim3(static_cast<unsigned>((l.batch * l.hq + 3) / 4)), dim3(128),
                 0, stream, a, static_cast<int32_t>(g)),
      "merge_q4_kernel launch");
}

}  // namespace ps
