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
//    more to bring two rows together.  (As e4m3 bytes a word would cost three operations, but there
//    is no such warp product in hardware: it is unpacked to halves, 186 us where this took 139 at
//    256 sequences of 28 / 4 heads and 4196 rows)
//  * queries are bf16 as given, times 2^48 against the small codes
//  * a weight times its row's V scale is rounded to fp16, on a power of two of its own for every
//    query head and group that follows the greatest such product: 11 bits down to 2^-10 of the
//    greatest at least, off by 2^-21 of it at most below.  (On one scale for all, set by the
//    greatest V scale, a group whose scales are 2^-24 of the other's lost bits, one of 2^-32 all of
//    them.  As bf16 the products' 8 bits tripled the output's error, since codes are not centred;
//    centring them, by a product with a constant 8 a group, takes 13 % more time)
//  * the dims of a row are stored so that one 16-byte load gives a lane the words of a whole
//    K fragment row; which dim goes to which position of the product does not matter as long as
//    the query's fragment agrees
//  * scales multiply scores (K) and weights (V), never the 128 codes of a row
// Eight query heads of a KV head share a row's bytes (the columns of the products).
//
// Work: a unit is (sequence, KV head), worked on in one block of eight warps or in pieces that
// merge_q4_kernel combines.  Every warp streams its own tiles of up to 32 rows (every eighth of the
// piece) through three stages of shared memory; warps meet where the piece ends.  The copies are
// 16-byte asynchronous loads, nine a lane and tile.  (One lane's bulk copies cost a hundred
// instructions a tile in setting up their uniform operands, a fifth of all; tiles of 256 rows for
// the whole block amortised that, but had to land whole before any warp could start.)
//
// Measured back to back in a graph, 28 / 4 heads or 16 / 2: 296 units of 32768 rows 220 us, as fast
// as a copy of the same bytes; 1024 of 4196 rows 110 us (5.6 TB/s), 128 of them 21 us (12 us at a
// copy's rate, the rest start and end), 8 of 131072 rows 34 us, 2 of 612 rows 7.3 us.  Equal shares
// of all rows for one wave of blocks, whatever units they span, balance better on paper, but
// finding a share took 5 us of scanning positions, each border a start, an end and a merge, and the
// SMs do not run equally fast: 134 us for the 1024, 49 us where 280 units take 35 one by one.
#include <cuda_bf16.h>
#include <math.h>

#include "ps_device.cuh"
#include "ps_internal.h"
#include "ps_ranges.cuh"
#include "ps_store.cuh"

namespace ps {
namespace {

// Two blocks of eight warps an SM (128 registers a thread) overlap one's start and end with the
// other's stream.
constexpr int kWarps = 8;
constexpr int kBlocksPerSm = 2;
constexpr int kTile = 32;  // rows of a warp's tile
constexpr int kStages = 3;
constexpr int kRowBytes = 2 * kQ4RowBytes + kQ4RecordBytes;
constexpr int kMaskAt = kTile * kRowBytes;  // in a stage, behind the rows: which of them are there
constexpr int kStageBytes = kMaskAt + 128;
constexpr int kWarpBytes = kStages * kStageBytes;
static_assert(kStageBytes >= (kHeadDim + 2) * kMaxGroup * 4, "a warp's result fits a stage");
constexpr int kGrain = kWarps;  // least tiles of a piece, on average
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Queries times this, against the codes' 2^-133: queries below 2^79 stay finite, and a product's
// place below the normal numbers, 2^-149, is 2^-64 of a query times a code.
constexpr float kLift = 281474976710656.f;                  // 2^48
constexpr float kUncode = 38685626227668133590597632.f;     // 2^85 = 2^133 / 2^48
constexpr float kUncodeV = 16777216.f;                      // 2^24
// A running maximum is moved only when a score passes it by more than this (in log2): weights
// then stay below 2^8, and a row of tiles rarely rescales its accumulators.
constexpr int kMaxSlack = 8;
// Of a head and group, products of a weight and a V scale go to fp16 times 2^e.  Where e is set, R
// being the greatest product so far (or a bound below it), R 2^e is in [2^(kProductLeast - 1),
// 2^kProductMost).  Until it is set again products stay below 2^kOperandMost: weights are below
// 2^kMaxSlack, and a V scale of 2^(kOperandMost - kMaxSlack - e) or more sets it again, low enough
// for that scale if the range allows it.  (Low only then: what is below 2^-14 loses bits.)
constexpr int kOperandMost = 15, kProductMost = 4, kProductLeast = -3;
// |e| is at most this: a weight times 2^e stays finite, 2^-e normal.
constexpr int kExpMost = 116;

struct DecodeQ4Args {
  const __nv_bfloat16* q;
  const int64_t* pos;
  __nv_bfloat16* out;
  float* lse;
  float* ws_o;    // [units, pieces, 8, D] the pieces of units that are split, normalised
  float* ws_lse;  // [units, pieces, 8] base-2 lse of each
  int32_t pieces;  // a unit has one for every kGrain tiles, up to this many
  int32_t* status;
  int32_t hq, hkv, group;
  float scale_log2;
  StoreArgs store;
};

__device__ __forceinline__ int64_t visible_rows(const DecodeQ4Args& a, int64_t p) {
  if (p < 0 || p >= (1ll << 31) || (a.store.linear && p >= a.store.lp)) return 0;
  const int64_t n = p + 1, cap = (int64_t)a.store.lp + (a.store.linear ? 0 : a.store.w);
  return n < cap ? n : cap;
}

// The rows a position sees, as tiles of up to 32: a tile is an aligned group of 32 rows of the
// prefix or of the ring, as far as its rows are visible.  Tiles are in up to three runs: the
// prefix, the ring from the oldest row's slot up, the ring from slot 0.  (Groups of 32 visible rows
// that straddle a border, loaded row by row, cost 5 us of 41 at 296 units of 100 + 4096 rows.)
struct Span {
  uint32_t pre, slot0, end;  // prefix rows; ring slots [slot0, end), from w on they are slot - w
  uint32_t n0, n1, n;        // tiles of the prefix, of the ring up to w, in all
};
__device__ __forceinline__ Span span_of(const DecodeQ4Args& a, int64_t p) {
  Span s;
  const uint32_t rows = static_cast<uint32_t>(visible_rows(a, p)), w = a.store.w;
  s.pre = min(rows, static_cast<uint32_t>(a.store.lp));
  const uint32_t ring = rows - s.pre;
  s.slot0 = 0;
  if (ring == w && ring) s.slot0 = static_cast<uint32_t>(mod_nonneg(p + 1 - a.store.lp, w));
  s.end = s.slot0 + ring;
  s.n0 = (s.pre + kTile - 1) / kTile;
  s.n1 = ring ? (min(s.end, w) + kTile - 1) / kTile - s.slot0 / kTile : 0;
  s.n = s.n0 + s.n1 + (s.end > w ? (s.end - w + kTile - 1) / kTile : 0);
  return s;
}

// How many pieces a unit of n tiles is worked on in.
__device__ __forceinline__ uint32_t pieces_of(const DecodeQ4Args& a, uint32_t n) {
  const uint32_t k = (n + kGrain - 1) / kGrain;
  return max(1u, min(k, static_cast<uint32_t>(a.pieces)));
}

// A unit, and the tiles [off, off + tiles) of it that a block has.
struct Unit {
  Span span;
  int32_t b, h;
  uint32_t off, tiles;
};

// Tile i of a unit: where its group of 32 rows starts, which of them are visible (none where a
// block table entry is bad), and how many tiles that are full follow in the same array.
struct Tile {
  int64_t at;
  uint32_t mask, full;
  bool ring, ok;  // ring: in the ring's array (never for a paged store: one pool)
};
__device__ __forceinline__ Tile locate(const DecodeQ4Args& a, const Unit& u, uint32_t i) {
  const StoreArgs& st = a.store;
  const Span& s = u.span;
  const uint32_t w = st.w;
  const bool ring = i >= s.n0;
  uint32_t g = i, lo = 0, hi = s.pre;  // the group, and the run's rows
  if (ring) {
    g -= s.n0;
    if (g < s.n1) {
      g += s.slot0 / kTile;
      lo = s.slot0;
      hi = min(s.end, w);
    } else {
      g -= s.n1;
      hi = s.end - w;
    }
  }
  const uint32_t row = g * kTile;
  Tile t;
  t.full = hi / kTile > g ? hi / kTile - g - 1 : 0;
  t.mask = 0xffffffffu;
  if (lo > row) t.mask <<= lo - row;
  if (hi - row < kTile) t.mask &= (1u << (hi - row)) - 1u;
  t.ring = ring && !st.table;
  t.ok = true;
  if (st.table) {
    const int32_t blk =
        st.table[(int64_t)u.b * st.table_stride + (ring ? st.pre_blocks : 0) + (row >> 6)];
    t.ok = blk >= 0 && blk < st.n_blocks;
    t.at = ((int64_t)blk * a.hkv + u.h) * 64 + (row & 63);
    t.full = 0;
    if (!t.ok) t.at = t.mask = 0;
  } else {
    t.at = ((int64_t)u.b * a.hkv + u.h) * (ring ? st.w : st.lp) + row;
  }
  return t;
}

// A lane's place in a piece: where its 16 bytes of the warp's next tile are, if that is one of
// `more` full tiles that follow in the same array.
struct Cursor {
  const uint8_t *k, *v, *s;
  int32_t more;
};

// Copies the tile at the cursor, 16 bytes a lane and load, and moves on to the warp's next.
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

// Copies the unit's tile i, one of `left` that its piece still has, into a stage (all lanes).  Rows
// that are not visible become zeros; `mask` gets those that are.
__device__ __forceinline__ void load_tile(const DecodeQ4Args& a, const Unit& u, uint32_t i,
                                          uint32_t left, int lane, Cursor& c, uint32_t dst,
                                          uint32_t* mask) {
  const StoreArgs& st = a.store;
  const Tile f = locate(a, u, i);
  if (lane == 0) {
    *mask = f.mask;
    if (!f.ok && a.status) atomicOr(a.status, PS_DEV_POS_RANGE);
  }
  c.k = (f.ring ? st.k[1] : st.k[0]) + f.at * kQ4RowBytes + lane * 16;
  c.v = (f.ring ? st.v[1] : st.v[0]) + f.at * kQ4RowBytes + lane * 16;
  c.s = (f.ring ? st.s[1] : st.s[0]) + f.at * kQ4RecordBytes + lane * 16;
  c.more = 0;
  if (f.mask == 0xffffffffu) {
    c.more = static_cast<int32_t>(min(f.full, left - 1) / kWarps);
    copy_tile(c, dst);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const bool there = (f.mask >> (8 * j + (lane >> 2))) & 1u;
    copy16_if(dst + 512 * j, there ? c.k + 512 * j : st.k[f.ring], there);
    copy16_if(dst + kTile * kQ4RowBytes + 512 * j, there ? c.v + 512 * j : st.v[f.ring], there);
  }
  const bool there = (f.mask >> lane) & 1u;
  copy16_if(dst + 2 * kTile * kQ4RowBytes, there ? c.s : st.s[f.ring], there);
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
// Products of two bf16 pairs, and the greater sizes of each half (a NaN counts for nothing).
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b & 0x7fff7fffu));
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

// 2^e, |e| <= 126, and back.
__device__ __forceinline__ float exp2_of(int e) { return __int_as_float((e + 127) << 23); }
__device__ __forceinline__ int exp_of(float x) {
  return static_cast<int>(__float_as_uint(x) >> 23) - 127;
}

// One warp's running softmax and accumulators over the heads (2 t, 2 t + 1) of its lane's t.
struct State {
  float l[2];
  float o[8][4];   // tile 4 g + i: dims 64 g + 8 (lane / 4) + 2 i + {0, 1}, heads 2 t + {0, 1};
                   // times 2^e of the group and head
  float mn[2][2];  // sum p m of a group, over this lane's rows
};

// The tile row of product row r (0..7): even rows first, so that the four rows a lane's V words
// come from fall into different halves of the shared memory banks.
__device__ __forceinline__ int tile_row(int r) { return (r & 1) ? 4 + ((r >> 1) ^ 1) : r >> 1; }

__global__ void __launch_bounds__(kWarps * 32, kBlocksPerSm)
    decode_q4_kernel(const DecodeQ4Args a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Unit s_unit[kWarps];  // a copy a warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g8 = lane >> 2, t4 = lane & 3;
  const uint32_t unit = blockIdx.x / a.pieces, j = blockIdx.x % a.pieces;
  const int b = unit / a.hkv, h = unit % a.hkv;
  pdl_wait();
  pdl_trigger();

  uint8_t* const stages = smem + warp * kWarpBytes;
  const int64_t pos = a.pos[b];
  uint32_t tiles, pieces;  // of this piece, of the unit
  {
    Unit u;
    u.span = span_of(a, pos);
    u.b = b;
    u.h = h;
    const uint32_t n = u.span.n;
    if (n == 0 && threadIdx.x == 0 && j == 0 && a.status)
      atomicOr(a.status, pos < 0 ? PS_DEV_BAD_POS : PS_DEV_POS_RANGE);
    pieces = pieces_of(a, n);
    if (j >= pieces) return;
    const uint32_t q = n / pieces, r = n % pieces;
    u.off = j * q + min(j, r);
    u.tiles = tiles = q + (j < r ? 1 : 0);
    if (lane < kStages)
      *reinterpret_cast<uint32_t*>(stages + lane * kStageBytes + kMaskAt) = 0xffffffffu;
    if (lane == 0) s_unit[warp] = u;
    __syncwarp();
  }
  const int head0 = b * a.hq + h * a.group;

  // scores come out of the products times 2^(48 - 133); c takes that off and scales to base 2
  const float c = a.scale_log2 * kUncode, to_x = 1.f / c;
  Cursor cursor{nullptr, nullptr, nullptr, 0};
  const uint32_t mine = smem_u32(stages) + lane * 16;
  uint32_t tile = warp;  // the warp's next to load
  // Loads that into the stage at `at`.  Every call commits a group of copies, empty or not: when a
  // tile is used, two groups have been committed after its own.
  auto load = [&](uint32_t at) {
    if (cursor.more > 0) {
      --cursor.more;
      copy_tile(cursor, mine + at);
    } else if (tile < tiles) {
      const Unit& u = s_unit[warp];
      load_tile(a, u, u.off + tile, tiles - tile, lane, cursor, mine + at,
                reinterpret_cast<uint32_t*>(stages + at + kMaskAt));
    }
    tile += kWarps;
    copies_commit();
  };

  // the query's fragments: head g8, blocks 2 t and 2 t + 1 of both groups, times 2^48 (2^44
  // where the codes come out 16 times as large); and each group's sum of query dims
  uint32_t qf[2][2][4];
  float Q[2][2];  // of heads 2 t + e, on the products' scale
  {
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
    load(0);
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
  for (int i = 1; i < kStages; ++i) load(i * kStageBytes);

  State st;
  st.l[0] = st.l[1] = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) st.o[i][0] = st.o[i][1] = st.o[i][2] = st.o[i][3] = 0.f;
  st.mn[0][0] = st.mn[0][1] = st.mn[1][0] = st.mn[1][1] = 0.f;
  // a score (before c) above this moves the running maximum m
  float above[2] = {-INFINITY, -INFINITY};
  // weights are 2^(c x + shift), shift = -m, m whole (while there is no m, no score counts)
  float shift[2] = {INFINITY, INFINITY};
  // 2^e of both groups, of the two heads as a pair, and the greatest V scales of the two groups
  // that do not set it again, as bf16 side by side
  uint64_t lift[2];
  lift[0] = lift[1] = pack_f32x2(exp2_of(kExpMost), exp2_of(kExpMost));
  uint32_t scales_below = 0;

  const int kr = tile_row(g8);  // this lane's K rows: kr, kr + 8
  uint32_t at = 0;  // the stage of the tile in hand
  for (uint32_t i = warp; i < tiles; i += kWarps) {
    copies_wait<kStages - 1>();
    __syncwarp();  // every lane's copies
    const uint8_t* stage = stages + at;
    const uint8_t* kst = stage + kr * kQ4RowBytes + 16 * t4;
    const uint8_t* va = stage + (kTile + t4) * kQ4RowBytes + 8 * g8;
    const uint8_t* vc = stage + (kTile + 4 + (t4 ^ 1)) * kQ4RowBytes + 8 * g8;
    const uint8_t* rec = stage + 2 * kTile * kQ4RowBytes + kr * kQ4RecordBytes;
    const uint32_t mask = *reinterpret_cast<const uint32_t*>(stage + kMaskAt);
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
      __syncwarp();  // (all have read the mask)
      if (lane == 0) *reinterpret_cast<uint32_t*>(stages + at + kMaskAt) = 0xffffffffu;
    }
    // ---------------------------------------- running maximum
    float mx[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      mx[e] = fmaxf(max3f(x[0][e], x[0][2 + e], x[1][e]), x[1][2 + e]);
    // this lane looks at row `lane`'s V scales (bf16: not negative, they compare as integers)
    const uint2 own = *reinterpret_cast<const uint2*>(stage + 2 * kTile * kQ4RowBytes +
                                                      lane * kQ4RecordBytes + 8);
    const uint32_t scales = __byte_perm(own.x, own.y, 0x5410);
    if (__any_sync(0xffffffffu, mx[0] > above[0] || mx[1] > above[1] ||
                                    max_u16x2(scales, scales_below) != scales_below)) {
      int fall[2];  // log2 of what weights so far shrink by
      float sh[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1)
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], o));
        const float m = fmaxf(-shift[e], ceilf(mx[e] * c));  // (-inf where there is none)
        fall[e] = 0;
        sh[e] = 0.f;
        if (m != -INFINITY) {
          const float x_most = (m + kMaxSlack) * to_x;
          above[e] = fmaf(-0x1p-20f, fabsf(x_most), x_most);  // (less what its roundings may add)
          fall[e] = static_cast<int>(fminf(m + shift[e], 1000.f));
          sh[e] = -m;
        }
        shift[e] = -m;
        const float f = fast_exp2(static_cast<float>(-fall[e]));
        st.l[e] *= f;
        st.mn[0][e] *= f;
        st.mn[1][e] *= f;
      }
      // each group's greatest products of both heads, as bf16
      uint32_t most[2] = {0, 0};
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float* y = &x[r >> 1][2 * (r & 1)];
        const uint32_t p = cvt_bf16x2(fast_exp2(fmaf(y[0], c, sh[0])),
                                      fast_exp2(fmaf(y[1], c, sh[1])));
        const uint2 k = *reinterpret_cast<const uint2*>(rec + 8 * r * kQ4RecordBytes + 8);
        most[0] = max_abs_bf16x2(most[0], mul_bf16x2(p, __byte_perm(k.x, 0, 0x1010)));
        most[1] = max_abs_bf16x2(most[1], mul_bf16x2(p, __byte_perm(k.y, 0, 0x1010)));
      }
      scales_below = 0;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1)
          most[g] = max_u16x2(most[g], __shfl_xor_sync(0xffffffffu, most[g], o));
        // this tile's V scales are below 2^(top - 126)
        const uint32_t top =
            __reduce_max_sync(0xffffffffu, (g ? own.y : own.x) & 0x7fffu) >> 7;
        const float2 lifts = unpack_f32x2(lift[g]);
        int n[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // the range of e: R is below 2^(b - 126) of this tile's b, and of earlier products one is
          // 2^(kProductLeast - 1 - was) at least; it rises only as far as weights fall.  (Numbers
          // that are not finite stay so whatever e is)
          const int was = exp_of(e ? lifts.y : lifts.x) + fall[e];
          const int b = (e ? most[g] >> 16 : most[g] & 0xffffu) >> 7;
          const int least = min(kProductLeast + 126 - b, was);
          n[e] = max(kOperandMost - kMaxSlack + 126 - static_cast<int>(top), least);
          n[e] = min(min(n[e], least + kProductMost - kProductLeast), was);
          n[e] = min(max(n[e], -kExpMost), kExpMost);
          const float f = fast_exp2(static_cast<float>(n[e] - was));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            st.o[4 * g + i][e] *= f;
            st.o[4 * g + i][2 + e] *= f;
          }
        }
        lift[g] = pack_f32x2(exp2_of(n[0]), exp2_of(n[1]));
        // bf16 numbers below 2^(kOperandMost - kMaxSlack - e)
        const int highest = __reduce_max_sync(0xffffffffu, max(n[0], n[1]));
        scales_below |= ((min(127 + kOperandMost - kMaxSlack - highest, 254) << 7) - 1) << (16 * g);
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
        // a weight times its row's scale and 2^e, rounded to fp16: the tensor cores' operand type
        const float2 w0 = unpack_f32x2(fmul2(pack_f32x2(p[0], p[1]), lift[g]));
        const float2 w1 = unpack_f32x2(fmul2(pack_f32x2(p[2], p[3]), lift[g]));
        const uint32_t b0 = transpose8(cvt_f16x2(w0.x * lo_f(k0), w0.y * lo_f(k0)));
        const uint32_t b1 = transpose8(cvt_f16x2(w1.x * lo_f(k1), w1.y * lo_f(k1)));
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
    load(at);
    at = at == (kStages - 1) * kStageBytes ? 0 : at + kStageBytes;
  }

  // ------------------------------------------------ combine the warps, write the piece
  // the warp's first stage takes its result, [8 heads][128], then m[8], l[8], o and l to be taken
  // times 2^m
  const auto result_of = [&](int w) { return reinterpret_cast<float*>(smem + w * kWarpBytes); };
  float* res = result_of(warp);
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
      const float2 up = unpack_f32x2(lift[g]);
      const float down = exp2_of(-exp_of(e ? up.y : up.x));
      float y[8];
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        const int i = 4 * g + (d >> 1), j = 2 * (d & 1) + e;
        y[d] = fmaf(st.o[i][j] * ((d & 2) ? kUncodeV / 16.f : kUncodeV), down, st.mn[g][e]);
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
  // one warp a head, dims 4 lane .. 4 lane + 3.  (Spread over all warps and unrolled it
  // took half a microsecond longer: this runs once a piece, from a cold instruction cache.)
  if (warp < a.group) {
    const int head = warp;
    float M = -INFINITY, L = 0.f;
#pragma unroll 4
    for (int w = 0; w < kWarps; ++w)
      M = fmaxf(M, result_of(w)[kMaxGroup * kHeadDim + head]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int w = 0; w < kWarps; ++w) {
      const float* r = result_of(w);
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
    if (pieces > 1) {
      const int64_t slot = (int64_t)blockIdx.x * kMaxGroup + head;
      reinterpret_cast<float4*>(a.ws_o + slot * kHeadDim)[lane] = acc;
      if (lane == 0) a.ws_lse[slot] = lse2;
    } else {
      const int64_t row = head0 + head;
      reinterpret_cast<uint2*>(a.out + row * kHeadDim)[lane] =
          make_uint2(cvt_bf16x2(acc.x, acc.y), cvt_bf16x2(acc.z, acc.w));
      if (a.lse && lane == 0) a.lse[row] = lse2 * kLn2;
    }
  }
}

// Combines the pieces of units that were split, a warp (SPLIT 1) or a block (SPLIT 8, for many
// pieces) a query head, each warp eight pieces in flight (each round is a trip to L2); lane i owns
// dims 4 i .. 4 i + 3.
constexpr int kMergeBatch = 8;
template <int SPLIT>
__global__ void __launch_bounds__(kMaxGroup * 32) merge_q4_kernel(const DecodeQ4Args a) {
  static_assert(SPLIT == 1 || SPLIT == kMaxGroup, "warps a head");
  __shared__ float4 s_acc[SPLIT][32];
  __shared__ float2 s_ml[SPLIT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = SPLIT == 1 ? blockIdx.x : blockIdx.x / a.group;
  const int hh = SPLIT == 1 ? warp : blockIdx.x % a.group;
  const int part = SPLIT == 1 ? 0 : warp;
  const int b = unit / a.hkv, h = unit % a.hkv;
  const int64_t bh = (int64_t)b * a.hq + h * a.group + hh;
  pdl_trigger();
  // (the positions are from before the kernel that this one follows, which waited for them)
  const int n = static_cast<int>(pieces_of(a, span_of(a, a.pos[b]).n));
  pdl_wait();
  if (n == 1 || hh >= a.group) return;  // (a whole unit is written already)
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float M = -INFINITY, L = 0.f;
  for (int c0 = part; c0 < n; c0 += SPLIT * kMergeBatch) {
    float lv[kMergeBatch];
    float4 ov[kMergeBatch];
    float Mn = M;
#pragma unroll
    for (int k = 0; k < kMergeBatch; ++k) {
      const int c = c0 + k * SPLIT;
      lv[k] = -INFINITY;
      ov[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c < n) {
        const int64_t slot = ((int64_t)unit * a.pieces + c) * kMaxGroup + hh;
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
  if (SPLIT > 1) {
    s_acc[part][lane] = acc;
    if (lane == 0) s_ml[part] = make_float2(M, L);
    __syncthreads();
    if (part != 0) return;
#pragma unroll
    for (int w = 1; w < SPLIT; ++w) {
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
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  reinterpret_cast<uint2*>(a.out + bh * kHeadDim)[lane] =
      make_uint2(cvt_bf16x2(acc.x * inv, acc.y * inv), cvt_bf16x2(acc.z * inv, acc.w * inv));
  if (a.lse && lane == 0) a.lse[bh] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

// In how many blocks a unit is worked on, at most.  Pieces fill the SMs and even out the last wave
// of blocks, but each starts and ends on its own and has to be merged.  Of the numbers that fill
// one to eight halves of a wave, the one of least time is taken, with 0.1 us for a tile of each of
// an SM's two blocks (46 GB/s an SM: HBM's rate over all of them), 4 us for a block's start and end
// and 2 us for a merge.  Half a wave of pieces counts as a whole one: behind another kernel some
// SMs get two of its blocks (74 units of 4196 rows: 21.4 us in two pieces, 16.0 in four).  Whole
// units: 40 of 32768 rows take 110.9 us in one piece, 77.3 in seven; 1024 of 8448 rows 200 in one,
// 218 in two.
int64_t plan_decode(int64_t batch, int32_t hkv, int64_t max_keys) {
  const int64_t units = batch * hkv, sms = sm_count();
  const int64_t tiles = max_keys / kTile + 3;  // (a partial one at the end of each run)
  int64_t best = 1;
  float least = INFINITY;
  for (int64_t half = 0; half <= 8; ++half) {
    int64_t k = units > 0 ? half * sms / units : 0;
    if (k > tiles / kGrain) k = tiles / kGrain;
    if (k < 1) k = 1;
    int64_t halves = (units * k + sms - 1) / sms;
    if (k > 1 && halves < 2) halves = 2;
    const float us = 0.1f * halves * ((tiles + k - 1) / k) + 4.f * ((halves + 1) / 2) +
                     (k > 1 ? 2.f : 0.f);
    if (us < least) {
      least = us;
      best = k;
    }
  }
  return best;
}

}  // namespace

size_t decode_q4_workspace_bytes(int64_t batch, int32_t hkv, int64_t max_keys) {
  const int64_t pieces = plan_decode(batch, hkv, max_keys);
  if (pieces == 1) return 0;
  return size_t(batch * hkv * pieces) * kMaxGroup * (kHeadDim + 1) * sizeof(float);
}

int launch_decode_q4(const DecodeQ4Launch& l, cudaStream_t stream) {
  const int64_t pieces = plan_decode(l.batch, l.hkv, (int64_t)l.store.lp + l.store.w);
  const int64_t grid = l.batch * l.hkv * pieces;
  if (grid > 0x7fffffff) return fail(PS_ERR_UNSUPPORTED, "decode grid too large");
  DecodeQ4Args a;
  a.q = static_cast<const __nv_bfloat16*>(l.q);
  a.pos = l.pos;
  a.out = static_cast<__nv_bfloat16*>(l.out);
  a.lse = l.lse;
  a.pieces = static_cast<int32_t>(pieces);
  a.ws_o = static_cast<float*>(l.workspace);
  a.ws_lse = pieces > 1 ? a.ws_o + size_t(grid) * kMaxGroup * kHeadDim : nullptr;
  a.status = l.status;
  a.hq = l.hq;
  a.hkv = l.hkv;
  a.group = l.hq / l.hkv;
  a.scale_log2 = l.scale * kLog2e;
  a.store = l.store;
  constexpr size_t smem = size_t(kWarps) * kWarpBytes;
  PS_TRY(allow_smem<decode_q4_kernel>(smem));
  PS_TRY(check_cuda(launch_pdl(decode_q4_kernel, dim3(static_cast<unsigned>(grid)),
                               dim3(kWarps * 32), smem, stream, a),
                    "decode_q4_kernel launch"));
  if (pieces == 1) return PS_OK;
  const bool few = pieces <= kMergeBatch;
  return check_cuda(
      launch_pdl(few ? merge_q4_kernel<1> : merge_q4_kernel<kMaxGroup>,
                 dim3(static_cast<unsigned>(l.batch * l.hkv * (few ? 1 : a.group))),
                 dim3(kMaxGroup * 32), 0, stream, a),
      "merge_q4_kernel launch");
}

}  // namespace ps
