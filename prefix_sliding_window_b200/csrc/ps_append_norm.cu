// Appends that normalise and rotate on the way into the store (bf16, or quantised to 4 bits), and
// the read-back of a 4-bit store, sm_100a.
//
// One pass: a token's packed q, k and v heads are read once; keys are normalised, rotated at the
// token's position and written to their prefix row or ring slot, values go straight there, queries
// to q_out.  Bound by HBM and issue slots for long prompts (4 x 8192 tokens of 28 + 4 heads, half
// of them kept, back to back in a graph: 97 us, 86 % of a copy's rate; into 4 bits 115 us) and by
// latency for a decode step's single tokens.  Of tokens that share a ring slot only the newest of
// the call is written, so the result does not depend on which block runs first.
//
// A warp keeps a token's angles and weights in registers over all of its heads, as in the pass
// without a store; with few tokens eight warps share one.
//
// 4-bit rows: eight lanes hold a row, so the least and greatest value of a group of 64 dims, kept
// in one word, take three shuffles; every lane packs its two 8-dim chunks into two of the row's
// sixteen words.
#include <cuda_bf16.h>

#include "ps_norm_rope.cuh"
#include "ps_store.cuh"

namespace ps {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Least and greatest of two bf16 pairs; a NaN stays one.
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// A chunk's least value and its greatest one's negative, a bf16 each: the least of two such words
// is both again.
__device__ __forceinline__ uint32_t span_word(const uint4& w) {
  const uint32_t lo = min2_nan(min2_nan(w.x, w.y), min2_nan(w.z, w.w));
  const uint32_t hi = max2_nan(max2_nan(w.x, w.y), max2_nan(w.z, w.w));
  return min2_nan(__byte_perm(lo, hi, 0x5410) ^ 0x80000000u,
                  __byte_perm(lo, hi, 0x7632) ^ 0x80000000u);
}
__device__ __forceinline__ uint32_t row_span(uint32_t v) {
  v = min2_nan(v, __shfl_xor_sync(0xffffffffu, v, 1));
  v = min2_nan(v, __shfl_xor_sync(0xffffffffu, v, 2));
  return min2_nan(v, __shfl_xor_sync(0xffffffffu, v, 4));
}

// Quantises a row held by eight lanes (chunks p.c1, p.c2 of a lane, bf16) and writes it: payload
// words at `pay`, (s, m) of both groups at `rec` (8 bytes).  All lanes take part; only `live` ones
// write.
//
// A code is (x - m) / s rounded to nearest even, by a product with 1 / s (within 1e-5 of the
// quotient) and the remainder r = (x - m) - u s, which one fma gives exactly: beyond s / 2, or at
// s / 2 with u odd, the code is one further on.  (On the bf16 grid such ties are common: dividing
// where a product was near one ran for nearly every warp.)
__device__ __forceinline__ void quantise_row(const RopeLane& p, const uint4& r1, const uint4& r2,
                                             bool live, int lane8, uint8_t* pay, uint8_t* rec) {
  const int g1 = p.c1 >> 3, g2 = p.c2 >> 3;
  const uint32_t span1 = span_word(r1), span2 = span_word(r2);
  float m[2], s[2];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    constexpr uint32_t kNone = 0x7f807f80u;  // infinities
    const uint32_t span = row_span(min2_nan(g1 == g ? span1 : kNone, g2 == g ? span2 : kNone));
    m[g] = __uint_as_float(span << 16);
    const float most = -__uint_as_float(span & 0xffff0000u);
    s[g] = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(most - m[g], 15.f)));
    if (!(s[g] < INFINITY)) m[g] = s[g] = __uint_as_float(0x7fc00000u);
  }
  const float round = 12582912.f;  // 1.5 2^23: adding and taking it off rounds to nearest even
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int chunk = c ? p.c2 : p.c1;
    const int g = chunk >> 3, b = chunk & 7;
    const uint4& rw = c ? r2 : r1;
    const uint32_t w[4] = {rw.x, rw.y, rw.z, rw.w};
    const float mm = g ? m[1] : m[0], ss = g ? s[1] : s[0];
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(ss));
    const uint32_t half = __float_as_uint(0.5f * ss);
    float u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // (as packed operations, two values each, it took 6 % longer)
      const float x = __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
      const float d = __fsub_rn(x, mm), t = fmaf(d, inv, round);
      u[i] = t - round;
      const float r = fmaf(-u[i], ss, d);
      // an odd code leaves at the border already: its bound is the float below s / 2
      const float bound = __uint_as_float(half - (__float_as_uint(t) & 1u));
      if (fabsf(r) > bound) u[i] += copysignf(1.f, r);
      u[i] = fminf(u[i], 15.f);
    }
    if (ss > 0.f && ss < 1e-37f) {  // 1 / s overflows below 2^-128
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
        u[i] = fminf(rintf(__fdiv_rn(x - mm, ss)), 15.f);
      }
    }
    // halves of the word as sums of codes times 16^i, exact in fp32; 2^23 puts them into the
    // low mantissa bits
    const float lo16 = fmaf(u[6], 4096.f, fmaf(u[4], 256.f, fmaf(u[2], 16.f, u[0] + 8388608.f)));
    const float hi16 = fmaf(u[7], 4096.f, fmaf(u[5], 256.f, fmaf(u[3], 16.f, u[1] + 8388608.f)));
    const uint32_t word = __byte_perm(__float_as_uint(lo16), __float_as_uint(hi16), 0x5410);
    // (s is 0 or not a number: codes of 0)
    if (live) *reinterpret_cast<uint32_t*>(pay + 4 * (2 * b + g)) = ss > 0.f ? word : 0u;
  }
  if (live && lane8 == 0)
    *reinterpret_cast<uint2*>(rec) =
        make_uint2(cvt_bf16x2(s[0], m[0]), cvt_bf16x2(s[1], m[1]));
}

constexpr int kAhead = 2;  // items in flight a warp (four: 1 % slower)
constexpr int kBlocksPerSm = 2;
// Start positions of up to this many sequences are kept in shared memory (every warp reads its
// tokens' twice; from L2 they cost 1 us of 114 at 4 x 8192 tokens).
constexpr int kHeldBatch = kThreads;

// Warps stride over the call's tokens; SPLIT of them share one (1 or 8).  A token's items are four
// q heads each, then four rows each of its keys and values together (a K row and a V row cost
// little more in one item than apart, and with two KV heads apart would leave half a warp idle).
template <int SPLIT, bool Q4, bool INTER>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    append_norm_kernel(const AppendNormArgs a) {
  extern __shared__ __align__(16) uint4 s_ring[];  // [kWarps][kAhead + 1][2][32]
  __shared__ __align__(16) float s_cos[kWarps][kHalfDim];
  __shared__ __align__(16) float s_sin[kWarps][kHalfDim];
  __shared__ __align__(16) float s_w[2 * kHeadDim];
  __shared__ double s_freq[kHalfDim];
  __shared__ int64_t s_pos0[SPLIT == 1 ? kHeldBatch : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const RopeLane p = rope_lane<INTER>(a.rope, lane & 7);
  const int64_t gw = (int64_t)blockIdx.x * kWarps + warp;
  const Items<SPLIT> items((int64_t)gridDim.x * kWarps / SPLIT, static_cast<int>(gw % SPLIT),
                           a.q ? a.hq : 0, 2 * a.hkv);
  const int row = lane >> 3;  // of an item's four rows
  const int o1 = row * kHeadDim + 8 * p.c1, d2 = 8 * (p.c2 - p.c1);
  pdl_wait();
  pdl_trigger();

  const int64_t* pos0 = a.pos0;
  if (SPLIT == 1 && a.batch <= kHeldBatch) {
    if (threadIdx.x < a.batch) s_pos0[threadIdx.x] = pos0[threadIdx.x];
    __syncthreads();
    pos0 = s_pos0;
  }

  const int64_t end = items.any() ? a.batch * a.T : 0;
  // a token's sequence and place in it move on without divisions
  const int64_t step_b = items.step / a.T;
  const int32_t step_t = static_cast<int32_t>(items.step - step_b * a.T);
  struct Place {
    int64_t b;
    int32_t t;
  };
  auto next_place = [&](Place& g) {
    g.b += step_b;
    g.t += step_t;
    if (g.t >= a.T) g.t -= a.T, ++g.b;
  };
  // what a token's position says (`pos` where it is not `bad`); `none`: the store has no place for
  // it; `kept`: its rows go to the store (a newer token of the call may own the ring slot)
  struct Token {
    int32_t pos;
    bool bad, none, kept;
  };
  const int32_t fresh_from = a.store.linear ? 0 : max(a.T - a.store.w, 0);
  const bool no_prefix = !a.store.linear && !a.store.k[0];
  auto token = [&](const Place& g) {
    const uint64_t p = static_cast<uint64_t>(pos0[g.b] + g.t);
    Token t;
    t.pos = static_cast<int32_t>(p);
    t.bad = p >= (1ull << 31);
    const bool prefix = t.pos < a.store.lp;
    t.none = t.bad | (a.store.linear ? !prefix : prefix & no_prefix);
    t.kept = !t.none & (prefix | (g.t >= fresh_from));
    return t;
  };
  Segment at = items.first(gw / SPLIT), far = at;
  Place at_place, far_place;
  at_place.b = at.tok / a.T;
  at_place.t = static_cast<int32_t>(at.tok - at_place.b * a.T);
  far_place = at_place;
  // moves `far` past the K and V segments of tokens that keep none
  auto settle_far = [&]() {
    while (far.tok < end && far.is_k && !token(far_place).kept) {
      far = items.first(far.tok + items.step);
      next_place(far_place);
    }
  };
  settle_far();
  const __nv_bfloat16* src = nullptr;  // the next q item's
  auto open = [&]() {
    if (!far.is_k) src = a.q + far.tok * a.q_stride + items.q0 * 4 * kHeadDim + o1;
  };
  open();
  const uint4* ring_of = s_ring + warp * (kAhead + 1) * 2 * 32 + lane;
  const uint32_t ring_at = smem_u32(ring_of);
  constexpr uint32_t kItem = 2 * 32 * sizeof(uint4), kRing = (kAhead + 1) * kItem;
  uint32_t in = 0;
  auto load = [&]() {
    if (far.tok < end) {
      const bool there = row < far.rows;
      const __nv_bfloat16* from = src;
      if (far.is_k) {
        const int r = 2 * a.hkv - far.rows + row;
        from = r < a.hkv ? a.k + far.tok * a.k_stride + r * kHeadDim
                         : a.v + far.tok * a.v_stride + (r - a.hkv) * kHeadDim;
        from += 8 * p.c1;
      }
      copy16_if(ring_at + in, from, there);
      copy16_if(ring_at + in + kItem / 2, from + d2, there);
      in = in == kRing - kItem ? 0 : in + kItem;
      src += items.kStride;
      const int64_t was = far.tok;
      if (items.next(far)) {
        if (far.tok != was) next_place(far_place);
        settle_far();
        open();
      }
    }
    copies_commit();
  };
#pragma unroll 1
  for (int i = 0; i < kAhead; ++i) load();
  load_norm_weights(a.norm, s_w);
  load_frequencies(a.rope, s_freq);
  __syncthreads();

  RowCoef coef;
  int64_t tok = -1;  // whose angles are in shared memory
  bool fresh = true, skip = false, kept = false, writes = false;
  int64_t store_at = 0, stride = 0;  // the token's row of head 0, rows from a head to the next
  int32_t ring = 0, block = 0;
  __nv_bfloat16* dst = nullptr;
  uint32_t out = 0;
  while (at.tok < end) {
    const bool kv = at.is_k;
    const bool norm = (kv ? a.norm.wk : a.norm.wq) != nullptr;
    if (fresh) {
      if (at.tok != tok) {
        tok = at.tok;
        const Token t = token(at_place);
        if (t.none && a.status && lane == 0)
          atomicOr(a.status, t.bad && pos0[at_place.b] + at_place.t < 0 ? PS_DEV_BAD_POS
                                                                         : PS_DEV_POS_RANGE);
        // a token the store has no place for is skipped, its queries become zeros
        skip = t.none;
        kept = t.kept;
        if (kept) {
          const StoreArgs& st = a.store;
          ring = t.pos >= st.lp;
          const uint32_t slot = static_cast<uint32_t>(t.pos) - static_cast<uint32_t>(st.lp);
          store_at = ring ? slot % static_cast<uint32_t>(st.w) : t.pos;
          if (st.table)  // (looked at when the keys' turn comes)
            block = st.table[at_place.b * st.table_stride + (ring ? st.pre_blocks : 0) +
                             store_at / 64];
        }
        if (!kv || kept)
          rope_angles(a.rope, s_freq, t.bad ? 0 : t.pos, lane, s_cos[warp], s_sin[warp]);
      }
      if (kv && !kept) {  // on to the next token
        at = items.first(tok + items.step);
        next_place(at_place);
        continue;
      }
      if (kv) {
        const StoreArgs& st = a.store;
        writes = true;
        stride = st.table ? 64 : ring ? st.w : st.lp;
        if (st.table) {  // a bad entry only loses the row
          writes = block >= 0 && block < st.n_blocks;
          if (!writes && a.status && lane == 0) atomicOr(a.status, PS_DEV_POS_RANGE);
          store_at = (int64_t)block * a.hkv * 64 + store_at % 64;
          ring = 0;  // one pool holds both
        } else {
          store_at += at_place.b * a.hkv * stride;
        }
      }
      row_coef<INTER>(p, kv && norm, s_w + (kv ? kHeadDim : 0), s_cos[warp], s_sin[warp], coef);
      if (!kv) dst = a.q_out + (tok * a.hq + items.q0 * 4) * kHeadDim + o1;
    }
    load();
    copies_wait<kAhead>();
    const uint4 r1 = ring_of[out / sizeof(uint4)], r2 = ring_of[out / sizeof(uint4) + 32];
    out = out == kRing - kItem ? 0 : out + kItem;
    uint64_t u[4], v[4];
    unpack_pairs<INTER>(r1, r2, u, v);
    uint4 y1, y2;
    const bool live = row < at.rows && (!kv || writes);
    if (!kv) {
      norm_and_turn<INTER>(p, norm, false, coef, a.norm.eps, u, v);
      pack_pairs<INTER>(u, v, y1, y2);
      if (skip) y1 = y2 = make_uint4(0, 0, 0, 0);
      if (live) {
        *reinterpret_cast<uint4*>(dst) = y1;
        *reinterpret_cast<uint4*>(dst + d2) = y2;
      }
      dst += items.kStride;
    } else {
      norm_and_turn<INTER>(p, norm, true, coef, a.norm.eps, u, v);
      pack_pairs<INTER>(u, v, y1, y2);
      const int r = 2 * a.hkv - at.rows + row;
      const bool is_v = r >= a.hkv;
      if (is_v) y1 = r1, y2 = r2;  // values as they are
      const int64_t to = store_at + (is_v ? r - a.hkv : r) * stride;
      uint8_t* base = is_v ? a.store.v[ring] : a.store.k[ring];
      if (Q4) {
        quantise_row(p, y1, y2, live, lane & 7, base + to * kQ4RowBytes,
                     a.store.s[ring] + to * kQ4RecordBytes + (is_v ? 8 : 0));
      } else if (live) {
        __nv_bfloat16* to_row = reinterpret_cast<__nv_bfloat16*>(base) + to * kHeadDim + 8 * p.c1;
        *reinterpret_cast<uint4*>(to_row) = y1;
        *reinterpret_cast<uint4*>(to_row + d2) = y2;
      }
    }
    fresh = items.next(at);
    if (at.tok != tok) next_place(at_place);
  }
}

// x / y in 32 bits where x fits (the case in practice).
__device__ __forceinline__ int64_t quotient(int64_t x, int32_t y) {
  return x < (1ll << 32) ? static_cast<uint32_t>(x) / static_cast<uint32_t>(y) : x / y;
}

// Eight lanes a row: lane l takes the 8-dim block l of both groups (words 2 l, 2 l + 1).
__global__ void __launch_bounds__(kThreads) read_q4_kernel(const ReadQ4Args a) {
  pdl_wait();
  pdl_trigger();
  const int lane8 = threadIdx.x & 7;
  const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 3;  // (b, t, head)
  if (i >= a.batch * a.T * a.hkv) return;
  const int64_t tok = quotient(i, a.hkv), b = quotient(tok, a.T);
  const int head = static_cast<int>(i - tok * a.hkv);
  const int64_t p0 = a.pos0[b], pos = p0 + (tok - b * a.T);
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

template <int SPLIT, bool Q4, bool INTER>
static int launch_append(const AppendNormArgs& a, int64_t grid, cudaStream_t stream) {
  constexpr size_t ring = kWarps * (kAhead + 1) * 2 * 32 * sizeof(uint4);
  PS_TRY((allow_smem<append_norm_kernel<SPLIT, Q4, INTER>>(ring)));
  return check_cuda(launch_pdl(append_norm_kernel<SPLIT, Q4, INTER>,
                               dim3(static_cast<unsigned>(grid)), dim3(kThreads), ring, stream, a),
                    "append_norm_kernel launch");
}

template <int SPLIT>
static int launch_append_split(const AppendNormArgs& a, bool q4, int64_t grid,
                               cudaStream_t stream) {
  if (q4)
    return a.rope.interleaved ? launch_append<SPLIT, true, true>(a, grid, stream)
                              : launch_append<SPLIT, true, false>(a, grid, stream);
  return a.rope.interleaved ? launch_append<SPLIT, false, true>(a, grid, stream)
                            : launch_append<SPLIT, false, false>(a, grid, stream);
}

int launch_append_norm(const AppendNormArgs& a, bool q4, cudaStream_t stream) {
  const int64_t tokens = a.batch * a.T;
  if (tokens <= 0) return PS_OK;
  // eight warps share a token while every token has a block of its own in one wave
  const int64_t most = kBlocksPerSm * (int64_t)sm_count();
  if (tokens <= most) return launch_append_split<kWarps>(a, q4, tokens, stream);
  const int64_t blocks = (tokens + kWarps - 1) / kWarps;
  return launch_append_split<1>(a, q4, blocks < most ? blocks : most, stream);
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
