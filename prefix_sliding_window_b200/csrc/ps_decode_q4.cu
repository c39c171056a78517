// Decode attention over the 4-bit store, sm_100a.
//
// The query of sequence b at position p attends its visible rows (prefix rows, then the window's
// ring slots), each standing for m_g + s_g u_d in its two groups g of 64 dims:
//   S_k = sum_g s_kg (sum_{d in g} q_d u_kd) + m_kg sum_{d in g} q_d
//   o_d = sum_k p_k m_kg + sum_k (p_k s_kg) u_kd,  p = softmax(scale S)
// A row is 144 bytes (64 of K, 64 of V, 16 of scales and minima), so the kernel is bound by HBM
// once the codes can be fed to the tensor cores cheaply:
//  * a code u enters the matrix products as a subnormal: four bits at the bottom of a half word
//    are u 2^-133 as bf16 and u 2^-24 as fp16, the next four, masked in place, 16 times that
//    (exactly: the codes stay where the spacing is the subnormals'; the tensor cores take
//    subnormals in full).  A word of eight codes costs one shift and four ands, V's one byte move
//    more to bring two rows together.  (As e4m3 bytes a word would cost three operations, but there is no
//    such warp product in hardware: it is unpacked to halves, 186 us where this takes 139 at 256
//    sequences of 28 / 4 heads)
//  * queries are bf16 as given, times 2^64 against the small codes; weights are fp16, on a scale
//    that keeps the greatest weight times V scale in [2^6, 2^14): 11 bits down to 2^-20 of the
//    greatest.  (As bf16 their 8 bits tripled the output's error, since codes are not centred)
//  * the dims of a row are stored so that one 16-byte load gives a lane the words of a whole
//    K fragment row; which dim goes to which position of the product does not matter as long as
//    the query's fragment agrees
//  * scales multiply scores (K) and weights (V), never the 128 codes of a row
// Eight query heads of a KV head share a row's bytes (the columns of the products).
//
// Work: a unit is (sequence, KV head).  One wave of blocks takes equal shares of all units' visible
// rows back to back; a share may span units, and a unit's pieces are combined by merge_q4_kernel
// (above kMaxBatch sequences, whose lengths would take long to scan: one block a unit).  Inside a
// block every warp streams its own 32-row tiles (every eighth of a piece) through three stages of
// shared memory, on into the next piece: warps meet only where a piece ends.  The copies are
// 16-byte asynchronous loads, nine a lane and tile.  (One lane's bulk copies cost a hundred
// instructions a tile in setting up their uniform operands, a fifth of all; tiles of 256 rows for
// the whole block amortised that, but had to land whole before any warp could start.)
#include <cuda_bf16.h>
#include <math.h>

#include "ps_device.cuh"
#include "ps_internal.h"
#include "ps_ranges.cuh"
#include "ps_store.cuh"

namespace ps {
namespace {

// Sixteen warps an SM either way (128 registers a thread): two blocks of eight, or one of sixteen.
constexpr int kSmWarps = 16;
constexpr int kTile = 32;  // rows of a warp's tile
constexpr int kStages = 3;
constexpr int kRowBytes = 2 * kQ4RowBytes + kQ4RecordBytes;
constexpr int kStageBytes = kTile * kRowBytes;
constexpr int kWarpBytes = kStages * kStageBytes;
static_assert(kStageBytes >= (kHeadDim + 2) * kMaxGroup * 4, "a warp's result fits a stage");
// Rows of a block where a few units are split further than the SMs ask for: a tile a warp.  (One
// sequence of 4196 rows: 128 rows a block 12.7 us, 256 11.0, 512 10.9.)
constexpr int kMinRowsPerBlock = kSmWarps * kTile;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxBatch = 1024;
constexpr float kLift = 18446744073709551616.f;     // 2^64: queries, against the codes' 2^-133
constexpr float kUncode = 590295810358705651712.f;  // 2^69 = 2^133 / 2^64
constexpr float kUncodeV = 16777216.f;              // 2^24
// A weight times its row's V scale is below 2^(kWeightLog2 + kMaxSlack) = 2^14 < 65504.
constexpr int kWeightLog2 = 6;
// V scales below 2^kLeastScale are taken as that (fp32 sums of weights over them stay finite).
constexpr int kLeastScale = -90;
// A running maximum is moved only when a score passes it by more than this (in log2): weights
// then stay below 2^8, and a row of tiles rarely rescales its accumulators.
constexpr float kMaxSlack = 8.f;

struct DecodeQ4Args {
  const __nv_bfloat16* q;
  const int64_t* pos;
  __nv_bfloat16* out;
  float* lse;
  float* ws_o;    // [grid, 2, 8, D] a block's first and last piece where they are not whole units,
                  // normalised; NULL: one block a unit
  float* ws_lse;  // [grid, 2, 8] base-2 lse of each
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

// A unit, and the rows [off, off + rows) of it that a block works on.
struct Unit {
  int64_t p;       // position
  uint32_t n, pre; // visible rows, visible prefix rows
  uint32_t slot0;  // ring slot of the oldest window row
  int32_t b, h;
  uint32_t off, rows;
};

__device__ __forceinline__ void enter(const DecodeQ4Args& a, Unit& u) {
  u.pre = min(u.n, static_cast<uint32_t>(a.store.lp));
  u.slot0 = u.n > u.pre ? static_cast<uint32_t>(mod_nonneg(
                              u.p + 1 - (u.n - u.pre) - a.store.lp, a.store.w))
                        : 0;
}

// A run of rows that are contiguous in their array; ok: false where a block table entry is bad.
struct Rows {
  int64_t at;
  uint32_t run;
  bool ring, ok;  // ring: in the ring's array (never for a paged store: one pool)
};

// The run that visible row x starts.
__device__ __forceinline__ Rows locate(const DecodeQ4Args& a, const Unit& u, uint32_t x) {
  const StoreArgs& st = a.store;
  // prefix position x, or the window's (x - pre)-th oldest row
  const bool ring = x >= u.pre;
  uint32_t row = ring ? u.slot0 + (x - u.pre) : x;
  if (ring && row >= static_cast<uint32_t>(st.w)) row -= st.w;
  Rows r;
  r.run = ring ? min(st.w - row, u.n - x) : u.pre - x;
  r.ring = ring && !st.table;
  r.ok = true;
  if (st.table) {
    r.run = min(r.run, 64 - (row & 63));
    const int32_t blk =
        st.table[(int64_t)u.b * st.table_stride + (ring ? st.pre_blocks : 0) + (row >> 6)];
    r.ok = blk >= 0 && blk < st.n_blocks;
    r.at = ((int64_t)blk * a.hkv + u.h) * 64 + (row & 63);
  } else {
    r.at = ((int64_t)u.b * a.hkv + u.h) * (ring ? st.w : st.lp) + row;
  }
  return r;
}

// A lane's place in a piece: where its 16 bytes of the warp's next tile are, if that is one of
// `more` tiles that follow in the same run of rows.
struct Cursor {
  const uint8_t *k, *v, *s;
  int32_t more;
};

// Copies the tile at the cursor, 16 bytes a lane and load, and moves on to the warp's next.
template <int kWarps>
__device__ __forceinline__ void copy_tile(Cursor& c, uint32_t dst) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    copy16(dst + 512 * j, c.k + 512 * j);
    copy16(dst + kTile * kQ4RowBytes + 512 * j, c.v + 512 * j);
  }
  copy16(dst + 2 * kTile * kQ4RowBytes, c.s);
  c.k += kWarps * kTile * kQ4RowBytes;
  c.v += kWarps * kTile * kQ4RowBytes;
  c.s += kWarps * kTile * kQ4RecordBytes;
}

// Copies the tile from row row0 of a piece into a stage (all lanes).  Rows past the piece's end
// and rows that a bad block table entry leaves out become zeros; `absent` gets the latter.
template <int kWarps>
__device__ __forceinline__ void load_tile(const DecodeQ4Args& a, const Unit& u, uint32_t row0,
                                          int lane, Cursor& c, uint32_t dst, uint32_t* absent) {
  const StoreArgs& st = a.store;
  const uint32_t cnt = u.rows - row0;  // a tile or more, or the last rows
  const Rows f = locate(a, u, u.off + row0);
  if (st.table && lane == 0) *absent = 0;
  c.more = 0;
  if (f.ok && min(f.run, cnt) >= kTile) {
    const int64_t at = f.at * kQ4RowBytes + lane * 16;
    c.k = (f.ring ? st.k[1] : st.k[0]) + at;
    c.v = (f.ring ? st.v[1] : st.v[0]) + at;
    c.s = (f.ring ? st.s[1] : st.s[0]) + f.at * kQ4RecordBytes + lane * 16;
    c.more = static_cast<int32_t>((min(f.run, cnt) - kTile) / (kWarps * kTile));
    copy_tile<kWarps>(c, dst);
    return;
  }
  // row by row: lane l copies a quarter of rows 8 j + l / 4, and row l's record
#pragma unroll 1
  for (int j = 0; j < 5; ++j) {
    const uint32_t r = j < 4 ? 8 * j + (lane >> 2) : lane;
    Rows x{0, 0, !st.k[0], false};
    if (r < cnt) x = locate(a, u, u.off + row0 + r);
    if (!x.ok) x.at = 0;
    if (j < 4) {
      const int64_t at = x.at * kQ4RowBytes + (lane & 3) * 16;
      copy16_if(dst + 512 * j, (x.ring ? st.k[1] : st.k[0]) + at, x.ok);
      copy16_if(dst + kTile * kQ4RowBytes + 512 * j, (x.ring ? st.v[1] : st.v[0]) + at, x.ok);
    } else {
      copy16_if(dst + 2 * kTile * kQ4RowBytes,
                (x.ring ? st.s[1] : st.s[0]) + x.at * kQ4RecordBytes, x.ok);
      const uint32_t gone = __ballot_sync(0xffffffffu, r < cnt && !x.ok);
      if (gone && lane == 0) {  // (only a paged store has any)
        if (a.status) atomicOr(a.status, PS_DEV_POS_RANGE);
        *absent = gone;
      }
    }
  }
}

// The warp products and the 8 x 8 transpose as pure functions (not volatile), so that the
// compiler may interleave independent chains.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two floats as an fp16 pair, the first in the low half.
__device__ __forceinline__ uint32_t cvt_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// The greater of each 16-bit half.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Codes as pairs of small floats, one from each half word, of the low byte's two: the lower one,
// and the upper one (16 u).
__device__ __forceinline__ uint32_t pair_lo(uint32_t w) { return w & 0x000f000fu; }
__device__ __forceinline__ uint32_t pair_hi(uint32_t w) { return w & 0x00f000f0u; }

// The halves of a word of two bf16 as floats: adding -0 in mixed precision, which the FMA pipe
// does, where a shift or a mask would take the integer pipe that the codes are unpacked on.
__device__ __forceinline__ float lo_f(uint32_t w) {
  float y;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tadd.rn.f32.bf16 %0, l, 0f80000000;\n\t}"
      : "=f"(y)
      : "r"(w));
  return y;
}
__device__ __forceinline__ float hi_f(uint32_t w) {
  float y;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tadd.rn.f32.bf16 %0, h, 0f80000000;\n\t}"
      : "=f"(y)
      : "r"(w));
  return y;
}

// One warp's running softmax and accumulators over the heads (2 t, 2 t + 1) of its lane's t.
struct State {
  float l[2];
  float o[8][4];   // tile 4 g + i: dims 64 g + 8 (lane / 4) + 2 i + {0, 1}, heads 2 t + {0, 1}
  float mn[2][2];  // sum p m of a group, over this lane's rows
};

// The tile row of product row r (0..7): even rows first, so that the four rows a lane's V words
// come from fall into different halves of the shared memory banks.
__device__ __forceinline__ int tile_row(int r) { return (r & 1) ? 4 + ((r >> 1) ^ 1) : r >> 1; }

template <int kWarps>
__global__ void __launch_bounds__(kWarps * 32, kSmWarps / kWarps)
    decode_q4_kernel(const DecodeQ4Args a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t s_absent[kWarps][kStages];
  __shared__ float* s_result[kWarps];
  // this piece and the next, a copy a warp: only the lane that issues copies reads most of it
  __shared__ Unit s_piece[kWarps][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g8 = lane >> 2, t4 = lane & 3;
  pdl_wait();
  pdl_trigger();

  // ------------------------------------------------ this block's share of the rows
  Unit u;
  int64_t left;  // rows of the share still to do
  u.off = 0;
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
    u.b = src * sc.per;
    int64_t n;
    while (true) {
      u.p = a.pos[u.b];
      n = visible_rows(a, u.p);
      if (rest < a.hkv * n) break;
      rest -= a.hkv * n;
      ++u.b;
    }
    u.n = static_cast<uint32_t>(n);
    u.h = static_cast<int32_t>(div_nonneg(rest, n));
    u.off = static_cast<uint32_t>(rest - u.h * n);
  } else {
    u.b = blockIdx.x / a.hkv;
    u.h = blockIdx.x % a.hkv;
    u.p = a.pos[u.b];
    left = visible_rows(a, u.p);
    u.n = static_cast<uint32_t>(left);
    if (left == 0 && threadIdx.x == 0 && a.status)
      atomicOr(a.status, u.p < 0 ? PS_DEV_BAD_POS : PS_DEV_POS_RANGE);
  }

  // scores come out of the products times 2^(64 - 133); c takes that off and scales to base 2
  const float c = a.scale_log2 * kUncode;
  uint32_t in = 0, at = 0;  // stages the next tile goes to and the next tile comes from, in bytes
  int flying = 0;           // tiles issued and not yet used
  uint32_t row = warp * kTile;  // the next tile to issue: its row, and whether in the next piece
  bool next = false;
  Cursor cursor{nullptr, nullptr, nullptr, 0};
  const uint32_t mine = smem_u32(smem) + warp * kWarpBytes;
  int cur = 0;        // which of s_piece is this one
  enter(a, u);
  u.rows = static_cast<uint32_t>(left < u.n - u.off ? left : u.n - u.off);
  if (lane == 0) s_piece[warp][0] = u;
  __syncwarp();
  for (bool first_piece = true;; first_piece = false) {
    const uint32_t piece = s_piece[warp][cur].rows;
    left -= piece;
    if (lane == 0) {  // the next piece: the next unit that has rows, from its first row
      Unit v = s_piece[warp][cur];
      v.off = v.rows = 0;
      if (left > 0) {
        if (++v.h == a.hkv) {
          v.h = 0;
          do {
            v.p = a.pos[++v.b];
            v.n = static_cast<uint32_t>(visible_rows(a, v.p));
          } while (v.n == 0);
          enter(a, v);
        }
        v.rows = static_cast<uint32_t>(left < v.n ? left : v.n);
      }
      s_piece[warp][cur ^ 1] = v;
    }
    __syncwarp();
    // Issues the warp's next tile, of this piece or the next.  One stage stays free while a tile of
    // the next piece would take it: the warp's result goes there.
    // Every call commits a group of copies, empty or not: when a tile is used, two groups at least
    // have been committed after its own.
    auto issue = [&]() {
      if (!next && row >= piece) {
        next = true;
        row = warp * kTile;
        cursor.more = 0;
      }
      const Unit& from = s_piece[warp][next ? cur ^ 1 : cur];
      if (flying < (next ? kStages - 1 : kStages) && row < from.rows) {
        const uint32_t dst = mine + in + lane * 16;
        if (cursor.more > 0) {
          --cursor.more;
          copy_tile<kWarps>(cursor, dst);
        } else {
          load_tile<kWarps>(a, from, row, lane, cursor, dst, &s_absent[warp][in / kStageBytes]);
        }
        in = in == (kStages - 1) * kStageBytes ? 0 : in + kStageBytes;
        row += kWarps * kTile;
        ++flying;
      }
      copies_commit();
    };
    // the query's fragments: head g8, blocks 2 t and 2 t + 1 of both groups, times 2^64 (2^60
    // where the codes come out 16 times as large); and each group's sum of query dims
    uint32_t qf[2][2][4];
    float Q[2][2];  // of heads 2 t + e, on the products' scale
    {
      const int head0 = s_piece[warp][cur].b * a.hq + s_piece[warp][cur].h * a.group;
      uint4 w[2][2];
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          w[g][j] = make_uint4(0, 0, 0, 0);
          if (g8 < a.group)
            w[g][j] = *reinterpret_cast<const uint4*>(a.q + (int64_t)(head0 + g8) * kHeadDim +
                                                      64 * g + 16 * t4 + 8 * j);
        }
      // the query, then every block's first tile, then the rest: behind 28 MB of everybody's
      // third tiles the query would arrive 5 us later
      issue();
      float qs[2];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        qs[g] = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t ww[4] = {w[g][j].x, w[g][j].y, w[g][j].z, w[g][j].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float f = (i & 1) ? kLift / 16.f : kLift;
            qs[g] += lo_f(ww[i]) + hi_f(ww[i]);
            qf[g][j][i] = cvt_bf16x2(lo_f(ww[i]) * f, hi_f(ww[i]) * f);
          }
        }
        qs[g] += __shfl_xor_sync(0xffffffffu, qs[g], 1);
        qs[g] = (qs[g] + __shfl_xor_sync(0xffffffffu, qs[g], 2)) * (1.f / kUncode);
      }
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int e = 0; e < 2; ++e) Q[g][e] = __shfl_sync(0xffffffffu, qs[g], 4 * (2 * t4 + e));
    }

#pragma unroll 1
    for (int i = 1; i < kStages; ++i) issue();

    State st;
    st.l[0] = st.l[1] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) st.o[i][0] = st.o[i][1] = st.o[i][2] = st.o[i][3] = 0.f;
    st.mn[0][0] = st.mn[0][1] = st.mn[1][0] = st.mn[1][1] = 0.f;
    // a score (before c) above this moves the running maximum m
    float above[2] = {-INFINITY, -INFINITY};
    // weights are 2^(c x + shift), shift = kWeightLog2 - m - log2 of the least power of two above
    // every V scale so far (while there is no m, no score counts)
    float shift[2] = {INFINITY, INFINITY};
    int scale_exp = kLeastScale;

    const int kr = tile_row(g8);  // this lane's K rows: kr, kr + 8
    for (uint32_t first = warp * kTile; first < piece; first += kWarps * kTile) {
      copies_wait<kStages - 1>();
      __syncwarp();  // every lane's copies
      const uint8_t* stage = smem + warp * kWarpBytes + at;
      const uint8_t* kst = stage + kr * kQ4RowBytes + 16 * t4;
      const uint8_t* va = stage + (kTile + t4) * kQ4RowBytes + 8 * g8;
      const uint8_t* vc = stage + (kTile + 4 + (t4 ^ 1)) * kQ4RowBytes + 8 * g8;
      const uint8_t* rec = stage + 2 * kTile * kQ4RowBytes + kr * kQ4RecordBytes;
      // rows that are there; all but where the piece ends or a block table entry is bad
      uint32_t mask = 0xffffffffu;
      if (piece - first < kTile) mask = (1u << (piece - first)) - 1u;
      if (a.store.table) mask &= ~s_absent[warp][at / kStageBytes];
      // ---------------------------------------- scores of 2 x 16 rows
      float x[2][4];
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        const int r0 = 16 * blk, r1 = r0 + 8;
        const uint4 w0 = *reinterpret_cast<const uint4*>(kst + r0 * kQ4RowBytes);
        const uint4 w1 = *reinterpret_cast<const uint4*>(kst + r1 * kQ4RowBytes);
        const uint2 c0 = *reinterpret_cast<const uint2*>(rec + r0 * kQ4RecordBytes);
        const uint2 c1 = *reinterpret_cast<const uint2*>(rec + r1 * kQ4RecordBytes);
        float acc[2][4];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          acc[g][0] = acc[g][1] = acc[g][2] = acc[g][3] = 0.f;
#pragma unroll
          for (int j = 0; j < 2; ++j) {  // words 2 j + g of the lane's four
            const uint32_t a0 = j ? (g ? w0.w : w0.z) : (g ? w0.y : w0.x);
            const uint32_t a1 = j ? (g ? w1.w : w1.z) : (g ? w1.y : w1.x);
            const uint32_t b0 = a0 >> 8, b1 = a1 >> 8;
            mma(acc[g], pair_lo(a0), pair_lo(a1), pair_hi(a0), pair_hi(a1), qf[g][j][0],
                qf[g][j][1]);
            mma(acc[g], pair_lo(b0), pair_lo(b1), pair_hi(b0), pair_hi(b1), qf[g][j][2],
                qf[g][j][3]);
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float s0 = lo_f(c0.x) * acc[0][e], s1 = lo_f(c1.x) * acc[0][2 + e];
          s0 = fmaf(lo_f(c0.y), acc[1][e], s0);
          s1 = fmaf(lo_f(c1.y), acc[1][2 + e], s1);
          s0 = fmaf(hi_f(c0.x), Q[0][e], s0);
          s1 = fmaf(hi_f(c1.x), Q[0][e], s1);
          x[blk][e] = fmaf(hi_f(c0.y), Q[1][e], s0);
          x[blk][2 + e] = fmaf(hi_f(c1.y), Q[1][e], s1);
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
      for (int e = 0; e < 2; ++e)
        mx[e] = fmaxf(max3f(x[0][e], x[0][2 + e], x[1][e]), x[1][2 + e]);
      // this lane looks at row `lane`'s V scales (bf16, not negative: they compare as integers)
      const uint2 own = *reinterpret_cast<const uint2*>(stage + 2 * kTile * kQ4RowBytes +
                                                        lane * kQ4RecordBytes + 8);
      const uint32_t top = max_u16x2(own.x, own.y) & 0xffffu;
      if (__any_sync(0xffffffffu, mx[0] > above[0] || mx[1] > above[1] ||
                                      top >= static_cast<uint32_t>(scale_exp + 127) << 7)) {
        // (a scale that is not finite makes its products NaN whatever the exponent)
        const uint32_t most = __reduce_max_sync(0xffffffffu, top < 0x7f80u ? top : 0u);
        const int was = scale_exp;
        scale_exp = max(scale_exp, static_cast<int>(most >> 7) - 126);
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1)
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], o));
          // the old m, from the old shift (-inf where there is none)
          const float m = fmaxf(static_cast<float>(kWeightLog2 - was) - shift[e], mx[e] * c);
          const float to = static_cast<float>(kWeightLog2 - scale_exp) - m;
          f[e] = shift[e] == INFINITY ? 0.f : fast_exp2(to - shift[e]);
          if (m != -INFINITY) above[e] = (m + kMaxSlack) / c;
          shift[e] = to;
          st.l[e] *= f[e];
          st.mn[0][e] *= f[e];
          st.mn[1][e] *= f[e];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          st.o[j][0] *= f[0];
          st.o[j][1] *= f[1];
          st.o[j][2] *= f[0];
          st.o[j][3] *= f[1];
        }
      }
      const float sh[2] = {shift[0] == INFINITY ? 0.f : shift[0],
                           shift[1] == INFINITY ? 0.f : shift[1]};
      // ---------------------------------------- weights and values
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        const int r0 = 16 * blk, r1 = r0 + 8;
        const uint2 c0 = *reinterpret_cast<const uint2*>(rec + r0 * kQ4RecordBytes + 8);
        const uint2 c1 = *reinterpret_cast<const uint2*>(rec + r1 * kQ4RecordBytes + 8);
        float p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] = fast_exp2(fmaf(x[blk][j], c, sh[j & 1]));
        st.l[0] += p[0] + p[2];
        st.l[1] += p[1] + p[3];
        // this lane's V words: rows of the product's k = 2 t, 2 t + 1, 2 t + 8, 2 t + 9
        const uint2 v0 = *reinterpret_cast<const uint2*>(va + r0 * kQ4RowBytes);
        const uint2 v1 = *reinterpret_cast<const uint2*>(vc + r0 * kQ4RowBytes);
        const uint2 v2 = *reinterpret_cast<const uint2*>(va + r1 * kQ4RowBytes);
        const uint2 v3 = *reinterpret_cast<const uint2*>(vc + r1 * kQ4RowBytes);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const uint32_t k0 = g ? c0.y : c0.x, k1 = g ? c1.y : c1.x;
          // a weight times its row's scale, rounded to fp16: the tensor cores' operand type
          const uint32_t b0 = transpose8(cvt_f16x2(p[0] * lo_f(k0), p[1] * lo_f(k0)));
          const uint32_t b1 = transpose8(cvt_f16x2(p[2] * lo_f(k1), p[3] * lo_f(k1)));
          st.mn[g][0] = fmaf(p[0], hi_f(k0), fmaf(p[2], hi_f(k1), st.mn[g][0]));
          st.mn[g][1] = fmaf(p[1], hi_f(k0), fmaf(p[3], hi_f(k1), st.mn[g][1]));
          const uint32_t x0 = g ? v0.y : v0.x, x1 = g ? v1.y : v1.x;
          const uint32_t x2 = g ? v2.y : v2.x, x3 = g ? v3.y : v3.x;
          const uint32_t e0 = __byte_perm(x0, x1, 0x5410), f0 = __byte_perm(x0, x1, 0x7632);
          const uint32_t e1 = __byte_perm(x2, x3, 0x5410), f1 = __byte_perm(x2, x3, 0x7632);
          mma_f16(st.o[4 * g + 0], pair_lo(e0), pair_lo(f0), pair_lo(e1), pair_lo(f1), b0, b1);
          mma_f16(st.o[4 * g + 1], pair_hi(e0), pair_hi(f0), pair_hi(e1), pair_hi(f1), b0, b1);
          const uint32_t e2 = e0 >> 8, f2 = f0 >> 8, e3 = e1 >> 8, f3 = f1 >> 8;
          mma_f16(st.o[4 * g + 2], pair_lo(e2), pair_lo(f2), pair_lo(e3), pair_lo(f3), b0, b1);
          mma_f16(st.o[4 * g + 3], pair_hi(e2), pair_hi(f2), pair_hi(e3), pair_hi(f3), b0, b1);
        }
      }
      __syncwarp();  // every lane has read the stage
      if (cursor.more > 0 && !next) {
        // the common case, with all stages in flight: the next tile goes where this one was
        --cursor.more;
        copy_tile<kWarps>(cursor, mine + at + lane * 16);
        copies_commit();
        row += kWarps * kTile;
        in = at == (kStages - 1) * kStageBytes ? 0 : at + kStageBytes;
      } else {
        --flying;
        issue();
      }
      at = at == (kStages - 1) * kStageBytes ? 0 : at + kStageBytes;
    }

    // ------------------------------------------------ combine the warps, write the piece
    // the stage to be filled next holds the warp's result now, [8 heads][128], then m[8], l[8], o
    // and l to be taken times 2^m; the other stages may hold the next piece's first tiles
    float* res = reinterpret_cast<float*>(smem + warp * kWarpBytes + in);
    if (lane == 0) s_result[warp] = res;
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
        float y[8];
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          const int i = 4 * g + (d >> 1), j = 2 * (d & 1) + e;
          y[d] = fmaf(st.o[i][j], (d & 2) ? kUncodeV / 16.f : kUncodeV, st.mn[g][e]);
        }
        reinterpret_cast<float4*>(dst + 64 * g)[0] = make_float4(y[0], y[1], y[2], y[3]);
        reinterpret_cast<float4*>(dst + 64 * g)[1] = make_float4(y[4], y[5], y[6], y[7]);
      }
      if (g8 == 0) {
        res[kMaxGroup * kHeadDim + 2 * t4 + e] = -shift[e];
        res[kMaxGroup * kHeadDim + kMaxGroup + 2 * t4 + e] = st.l[e];
      }
    }
    __syncthreads();
    // one warp a head, dims 4 lane .. 4 lane + 3.  (Spread over all sixteen warps and unrolled it
    // took half a microsecond longer: this runs once a piece, from a cold instruction cache.)
    if (warp < a.group) {
      const int head = warp;
      float M = -INFINITY, L = 0.f;
#pragma unroll 4
      for (int w = 0; w < kWarps; ++w)
        M = fmaxf(M, s_result[w][kMaxGroup * kHeadDim + head]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int w = 0; w < kWarps; ++w) {
        const float* r = s_result[w];
        const float m = r[kMaxGroup * kHeadDim + head];
        const float f = m == -INFINITY ? 0.f : fast_exp2(m - M);  // (such a warp left zeros)
        const float4 y = reinterpret_cast<const float4*>(r + head * kHeadDim)[lane];
        L = fmaf(f, r[kMaxGroup * kHeadDim + kMaxGroup + head], L);
        acc.x = fmaf(f, y.x, acc.x);
        acc.y = fmaf(f, y.y, acc.y);
        acc.z = fmaf(f, y.z, acc.z);
        acc.w = fmaf(f, y.w, acc.w);
      }
      const float inv = L == 0.f ? 0.f : 1.f / L;
      const float lse2 = L == 0.f ? -INFINITY : M + log2f(L);
      acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
      if (piece < s_piece[warp][cur].n) {
        const int64_t slot = (2 * (int64_t)blockIdx.x + (first_piece ? 0 : 1)) * kMaxGroup + head;
        reinterpret_cast<float4*>(a.ws_o + slot * kHeadDim)[lane] = acc;
        if (lane == 0) a.ws_lse[slot] = lse2;
      } else {
        const int64_t row = (int64_t)s_piece[warp][cur].b * a.hq +
                            s_piece[warp][cur].h * a.group + head;
        reinterpret_cast<uint2*>(a.out + row * kHeadDim)[lane] =
            make_uint2(cvt_bf16x2(acc.x, acc.y), cvt_bf16x2(acc.z, acc.w));
        if (a.lse && lane == 0) a.lse[row] = lse2 * kLn2;
      }
    }
    if (left <= 0) break;
    __syncthreads();  // the next piece's tiles overwrite the results just read
    cur ^= 1;
    next = false;  // `row` is a row of the next piece already
  }
}

// Combines the pieces of one (sequence, query head), one block each, where its unit was split:
// block c of the decode owned the rows [total c / grid, total (c + 1) / grid), so which blocks hold
// pieces follows from the positions alone.  A unit's later pieces are their blocks' first ones, its
// earliest is its block's first or last.  Each warp takes every fourth piece, eight in flight (a
// long row has dozens, and each round is a trip to L2: four cost 1.5 us more at 33 pieces); lane i
// owns dims 4 i .. 4 i + 3.
constexpr int kMergeWarps = 4;
constexpr int kMergeBatch = 8;
__global__ void __launch_bounds__(kMergeWarps * 32)
    merge_q4_kernel(const DecodeQ4Args a, int32_t grid) {
  __shared__ float4 s_acc[kMergeWarps][32];
  __shared__ float2 s_ml[kMergeWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t bh = blockIdx.x;
  const int b = static_cast<int>(bh / a.hq), head = static_cast<int>(bh % a.hq);
  const int h = head / a.group, hh = head % a.group;
  const RowScan sc = scan_rows(a, lane, false);
  const int64_t total = sc.total * a.hkv;
  const int src = b / sc.per;
  int64_t first = __shfl_sync(0xffffffffu, sc.before, src);
  for (int i = src * sc.per; i < b; ++i) first += visible_rows(a, a.pos[i]);
  const int64_t n = visible_rows(a, a.pos[b]);
  int c_lo = 1, c_hi = 0, late = 0;  // late: the piece in c_lo is that block's last
  if (n > 0) {
    const int64_t pu = a.hkv * first + h * n;
    c_lo = static_cast<int>(div_nonneg((pu + 1) * grid - 1, total));
    c_hi = static_cast<int>(div_nonneg((pu + n) * grid - 1, total));
    late = div_nonneg(total * c_lo, grid) < pu;
  }
  pdl_trigger();
  pdl_wait();
  if (n > 0 && c_lo == c_hi) return;  // a whole unit is written already
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float M = -INFINITY, L = 0.f;
  for (int c0 = c_lo + warp; c0 <= c_hi; c0 += kMergeWarps * kMergeBatch) {
    float lv[kMergeBatch];
    float4 ov[kMergeBatch];
    float Mn = M;
#pragma unroll
    for (int k = 0; k < kMergeBatch; ++k) {
      const int c = c0 + k * kMergeWarps;
      lv[k] = -INFINITY;
      ov[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      // with fewer rows than blocks some blocks own none and wrote no piece
      if (c <= c_hi && (total >= grid || total * c / grid != total * (c + 1) / grid)) {
        const int64_t slot = (2 * (int64_t)c + (c == c_lo ? late : 0)) * kMaxGroup + hh;
        lv[k] = a.ws_lse[slot];
        ov[k] = reinterpret_cast<const float4*>(a.ws_o + slot * kHeadDim)[lane];
      }
    }
#pragma unroll
    for (int k = 0; k < kMergeBatch; ++k) Mn = fmaxf(Mn, lv[k]);
    const float ref = Mn == -INFINITY ? 0.f : Mn;
    const float f = fast_exp2(M - ref);
    L *= f;
    acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
#pragma unroll
    for (int k = 0; k < kMergeBatch; ++k) {
      const float e = fast_exp2(lv[k] - ref);
      L += e;
      acc.x = fmaf(e, ov[k].x, acc.x);
      acc.y = fmaf(e, ov[k].y, acc.y);
      acc.z = fmaf(e, ov[k].z, acc.z);
      acc.w = fmaf(e, ov[k].w, acc.w);
    }
    M = Mn;
  }
  s_acc[warp][lane] = acc;
  if (lane == 0) s_ml[warp] = make_float2(M, L);
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int w = 1; w < kMergeWarps; ++w) {
    const float2 ml = s_ml[w];
    const float4 y = s_acc[w][lane];
    const float Mn = fmaxf(M, ml.x), ref = Mn == -INFINITY ? 0.f : Mn;
    const float f = fast_exp2(M - ref), e = fast_exp2(ml.x - ref);
    L = L * f + ml.y * e;
    acc.x = acc.x * f + y.x * e;
    acc.y = acc.y * f + y.y * e;
    acc.z = acc.z * f + y.z * e;
    acc.w = acc.w * f + y.w * e;
    M = Mn;
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  reinterpret_cast<uint2*>(a.out + bh * kHeadDim)[lane] =
      make_uint2(cvt_bf16x2(acc.x * inv, acc.y * inv), cvt_bf16x2(acc.z * inv, acc.w * inv));
  if (a.lse && lane == 0) a.lse[bh] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

// How a decode is laid out: blocks of `warps` warps, `grid` of them, sharing the rows or one a unit.
struct Plan {
  int64_t grid;
  int warps;
  bool share;
};
Plan plan_decode(int64_t batch, int32_t hkv, int64_t max_keys) {
  const int64_t units = batch * hkv, sms = sm_count();
  // two blocks an SM overlap one's start and end with the other's stream
  if (units >= 2 * sms || batch > kMaxBatch) return {units, kSmWarps / 2, false};
  if (units > sms) return {2 * sms, kSmWarps / 2, true};
  // few units: one block an SM, a whole number of blocks a unit if that fills 5/6 of the SMs, so
  // that equally long units split on their own borders
  int64_t g = units * ((max_keys + kMinRowsPerBlock - 1) / kMinRowsPerBlock);
  if (g >= sms) {
    const int64_t even = units * (sms / units);
    g = even * 6 >= sms * 5 ? even : sms;
  }
  if (g < 1) g = 1;
  return {g, kSmWarps, g != units};
}

}  // namespace

size_t decode_q4_workspace_bytes(int64_t batch, int32_t hkv, int64_t max_keys) {
  const Plan p = plan_decode(batch, hkv, max_keys);
  if (!p.share || batch == 0) return 0;
  return size_t(2 * p.grid) * kMaxGroup * (kHeadDim + 1) * sizeof(float);
}

int launch_decode_q4(const DecodeQ4Launch& l, cudaStream_t stream) {
  const Plan p = plan_decode(l.batch, l.hkv, (int64_t)l.store.lp + l.store.w);
  if (p.grid > 0x7fffffff) return fail(PS_ERR_UNSUPPORTED, "decode grid too large");
  DecodeQ4Args a;
  a.q = static_cast<const __nv_bfloat16*>(l.q);
  a.pos = l.pos;
  a.out = static_cast<__nv_bfloat16*>(l.out);
  a.lse = l.lse;
  a.ws_o = p.share ? static_cast<float*>(l.workspace) : nullptr;
  a.ws_lse = p.share ? a.ws_o + size_t(2 * p.grid) * kMaxGroup * kHeadDim : nullptr;
  a.status = l.status;
  a.batch = static_cast<int32_t>(l.batch);
  a.hq = l.hq;
  a.hkv = l.hkv;
  a.group = l.hq / l.hkv;
  a.scale_log2 = l.scale * kLog2e;
  a.store = l.store;
  const bool one = p.warps == kSmWarps;
  const size_t smem = size_t(p.warps) * kWarpBytes;
  PS_TRY(one ? allow_smem<decode_q4_kernel<kSmWarps>>(smem)
             : allow_smem<decode_q4_kernel<kSmWarps / 2>>(smem));
  PS_TRY(check_cuda(
      launch_pdl(one ? decode_q4_kernel<kSmWarps> : decode_q4_kernel<kSmWarps / 2>,
                 dim3(static_cast<unsigned>(p.grid)), dim3(p.warps * 32), smem, stream, a),
      "decode_q4_kernel launch"));
  if (!p.share) return PS_OK;
  return check_cuda(
      launch_pdl(merge_q4_kernel, dim3(static_cast<unsigned>(l.batch * l.hq)),
                 dim3(kMergeWarps * 32), 0, stream, a, static_cast<int32_t>(p.grid)),
      "merge_q4_kernel launch");
}

}  // namespace ps
