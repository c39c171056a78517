// Norm and rotation of queries and keys in one pass, and its backward, sm_100a.
//
//   forward:  y = R(p) (x rstd w),  rstd = 1 / sqrt(mean x^2 + eps)
//   backward: g = R(p)^T dy,  n = x rstd,  dw = sum g n,  dx = rstd (w g - n mean(w g n))
// Both stream every row once (forward one read and one write of each bf16 row, backward two
// reads and one write) and are bound by HBM.  A warp keeps a token's angles and weights in
// registers over all of its heads; the rows of the next items are in flight as asynchronous copies
// into a ring of shared memory, every lane its own 16-byte chunks, so that the depth of the
// prefetch costs no registers (two items ahead in registers: 132 us forward at 4 x 8192 tokens of
// 28 + 4 heads, 106 with the ring).  With few tokens eight warps share one.
//
// At 4 x 8192 tokens of 28 + 4 heads, back to back in a graph, the forward takes 86 us (6.2 TB/s,
// 96 % of a copy's rate), the backward 132 us (94 %); a call between others, which finds their
// lines in L2, 93 and 148.  Three blocks of 80 registers an SM: 97 and more.
#include <cuda_bf16.h>

#include "ps_norm_rope.cuh"

namespace ps {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Items in flight a warp: forward two (four: 97 us where these take 86), backward two, each twice
// the bytes.
constexpr int kBlocksPerSm = 2, kAhead = 2;
constexpr int kBwdBlocksPerSm = 2, kBwdAhead = 2;

// Warps stride over tokens; SPLIT of them share one (1 or 8) and take its items in turn.
template <int SPLIT, bool INTER>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) norm_rope_kernel(const NormRopeArgs a) {
  extern __shared__ __align__(16) uint4 s_all[];  // [kWarps][kAhead + 1][2][32]
  uint4 (*s_ring)[kAhead + 1][2][32] = reinterpret_cast<uint4 (*)[kAhead + 1][2][32]>(s_all);
  __shared__ __align__(16) float s_cos[kWarps][kHalfDim];
  __shared__ __align__(16) float s_sin[kWarps][kHalfDim];
  __shared__ __align__(16) float s_w[2 * kHeadDim];
  __shared__ double s_freq[kHalfDim];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const RopeLane p = rope_lane<INTER>(a.rope, lane & 7);
  const int64_t gw = (int64_t)blockIdx.x * kWarps + warp;
  const Items<SPLIT> items((int64_t)gridDim.x * kWarps / SPLIT, static_cast<int>(gw % SPLIT),
                           a.q ? a.hq : 0, a.k ? a.hkv : 0);
  const int row = lane >> 3;  // of an item's four heads
  const int o1 = row * kHeadDim + 8 * p.c1, d2 = 8 * (p.c2 - p.c1);
  pdl_wait();
  pdl_trigger();

  const int64_t end = items.any() ? a.n : 0;
  Segment at = items.first(gw / SPLIT), far = at;  // the item worked on, the next to load
  auto source = [&](const Segment& g) {
    return g.is_k ? a.k + g.tok * a.k_stride + items.k0 * 4 * kHeadDim + o1
                  : a.q + g.tok * a.q_stride + items.q0 * 4 * kHeadDim + o1;
  };
  const __nv_bfloat16* src = source(far);
  const uint32_t ring = smem_u32(&s_ring[warp][0][0][lane]);
  constexpr uint32_t kItem = 2 * 32 * sizeof(uint4), kRing = (kAhead + 1) * kItem;
  uint32_t in = 0;  // the next item's place in the ring
  auto load = [&]() {
    if (far.tok < end) {
      const bool there = row < far.rows;
      copy16_if(ring + in, src, there);
      copy16_if(ring + in + kItem / 2, src + d2, there);
      in = in == kRing - kItem ? 0 : in + kItem;
      src += items.kStride;
      if (items.next(far)) src = source(far);
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
  bool bad = false, fresh = true;  // fresh: the segment's first item
  __nv_bfloat16* dst = nullptr;
  int64_t next_pos = at.tok < end ? a.pos[at.tok] : 0;
  uint32_t out = 0;
  while (at.tok < end) {
    const bool norm = (at.is_k ? a.norm.wk : a.norm.wq) != nullptr;
    if (fresh) {
      if (at.tok != tok) {
        tok = at.tok;
        const int64_t pos = next_pos;
        if (tok + items.step < end) next_pos = a.pos[tok + items.step];
        bad = bad_rope_position(pos);
        if (bad && a.status && lane == 0) atomicOr(a.status, rope_position_flag(pos));
        rope_angles(a.rope, s_freq, bad ? 0 : pos, lane, s_cos[warp], s_sin[warp]);
      }
      row_coef<INTER>(p, at.is_k && norm, s_w + (at.is_k ? kHeadDim : 0), s_cos[warp],
                      s_sin[warp], coef);
      dst = at.is_k ? a.k_out + (tok * a.hkv + items.k0 * 4) * kHeadDim + o1
                    : a.q_out + (tok * a.hq + items.q0 * 4) * kHeadDim + o1;
    }
    load();
    copies_wait<kAhead>();
    uint64_t u[4], v[4];
    const uint4* r = &s_ring[warp][0][0][lane] + out / sizeof(uint4);
    unpack_pairs<INTER>(r[0], r[32], u, v);
    out = out == kRing - kItem ? 0 : out + kItem;
    norm_and_turn<INTER>(p, norm, at.is_k, coef, a.norm.eps, u, v);
    uint4 y1, y2;
    pack_pairs<INTER>(u, v, y1, y2);
    if (bad) y1 = y2 = make_uint4(0, 0, 0, 0);
    if (row < at.rows) {
      *reinterpret_cast<uint4*>(dst) = y1;
      *reinterpret_cast<uint4*>(dst + d2) = y2;
    }
    dst += items.kStride;
    fresh = items.next(at);
  }
}

// Backward.  A warp keeps its share of the query weight's gradient in registers, of the key
// weight's in shared memory (a token has fewer key heads).
template <int SPLIT, bool INTER>
__global__ void __launch_bounds__(kThreads, kBwdBlocksPerSm)
    norm_rope_bwd_kernel(const NormRopeBwdArgs a) {
  extern __shared__ __align__(16) uint4 s_ring[];  // [kWarps][kBwdAhead + 1][4][32]
  __shared__ __align__(16) float s_cos[kWarps][kHalfDim];
  __shared__ __align__(16) float s_sin[kWarps][kHalfDim];
  __shared__ __align__(16) float s_w[2 * kHeadDim];
  __shared__ double s_freq[kHalfDim];
  __shared__ uint64_t s_dwk[kWarps][8][32];  // a lane's sixteen sums, in pairs
  __shared__ float s_dw[kWarps][2 * kHeadDim];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const RopeLane p = rope_lane<INTER>(a.rope, lane & 7);
  const int64_t gw = (int64_t)blockIdx.x * kWarps + warp;
  const Items<SPLIT> items((int64_t)gridDim.x * kWarps / SPLIT, static_cast<int>(gw % SPLIT),
                           a.dq_out ? a.hq : 0, a.dk_out ? a.hkv : 0);
  const int row = lane >> 3;
  const int o1 = row * kHeadDim + 8 * p.c1, d2 = 8 * (p.c2 - p.c1);
  const bool norm_q = a.norm.wq != nullptr, norm_k = a.norm.wk != nullptr;
  pdl_wait();
  pdl_trigger();

  const int64_t end = items.any() ? a.n : 0;
  Segment at = items.first(gw / SPLIT), far = at;
  const __nv_bfloat16 *gsrc, *xsrc;  // the next item's output gradients and inputs
  auto open = [&](const Segment& g) {
    const int64_t first = (g.is_k ? items.k0 : items.q0) * 4 * kHeadDim + o1;
    gsrc = (g.is_k ? a.dk_out + g.tok * a.hkv * kHeadDim : a.dq_out + g.tok * a.hq * kHeadDim) +
           first;
    xsrc = (g.is_k ? a.k + g.tok * a.k_stride : a.q + g.tok * a.q_stride) + first;
  };
  open(far);
  const uint4* ring_of = s_ring + warp * (kBwdAhead + 1) * 4 * 32 + lane;
  const uint32_t ring = smem_u32(ring_of);
  constexpr uint32_t kItem = 4 * 32 * sizeof(uint4), kRing = (kBwdAhead + 1) * kItem;
  uint32_t in = 0;
  auto load = [&]() {
    if (far.tok < end) {
      const bool there = row < far.rows;
      copy16_if(ring + in, gsrc, there);
      copy16_if(ring + in + kItem / 4, gsrc + d2, there);
      if (far.is_k ? norm_k : norm_q) {
        copy16_if(ring + in + kItem / 2, xsrc, there);
        copy16_if(ring + in + kItem / 4 * 3, xsrc + d2, there);
      }
      in = in == kRing - kItem ? 0 : in + kItem;
      gsrc += items.kStride;
      xsrc += items.kStride;
      if (items.next(far)) open(far);
    }
    copies_commit();
  };
#pragma unroll 1
  for (int i = 0; i < kBwdAhead; ++i) load();
  load_norm_weights(a.norm, s_w);
  load_frequencies(a.rope, s_freq);
#pragma unroll
  for (int i = 0; i < 8; ++i) s_dwk[warp][i][lane] = 0;
  __syncthreads();

  uint64_t dwu[4], dwv[4];  // query weight's gradient, this lane's pairs
  uint64_t wu[4], wv[4], c[4], s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) dwu[i] = dwv[i] = 0;
  int64_t tok = -1;
  bool bad = false, fresh = true;
  __nv_bfloat16* dst = nullptr;
  int64_t next_pos = at.tok < end ? a.pos[at.tok] : 0;
  uint32_t out = 0;
  while (at.tok < end) {
    const bool is_k = at.is_k;
    const bool norm = is_k ? norm_k : norm_q;
    if (fresh) {
      if (at.tok != tok) {
        tok = at.tok;
        const int64_t pos = next_pos;
        if (tok + items.step < end) next_pos = a.pos[tok + items.step];
        bad = bad_rope_position(pos);
        if (bad && a.status && lane == 0) atomicOr(a.status, rope_position_flag(pos));
        rope_angles(a.rope, s_freq, bad ? 0 : pos, lane, s_cos[warp], s_sin[warp]);
        lane_angles(p, s_cos[warp], s_sin[warp], c, s);
      }
      lane_weights<INTER>(s_w + (is_k ? kHeadDim : 0), p, wu, wv);
      dst = is_k ? a.dk + tok * a.dk_stride + items.k0 * 4 * kHeadDim + o1
                 : a.dq + tok * a.dq_stride + items.q0 * 4 * kHeadDim + o1;
    }
    load();
    copies_wait<kBwdAhead>();
    const uint4* r = ring_of + out / sizeof(uint4);
    out = out == kRing - kItem ? 0 : out + kItem;
    const bool live = row < at.rows;
    uint4 y1 = make_uint4(0, 0, 0, 0), y2 = y1;
    if (!bad) {
      uint64_t gu[4], gv[4];
      unpack_pairs<INTER>(r[0], r[32], gu, gv);
#pragma unroll
      for (int i = 0; i < 4; ++i)  // (a branch for heads rotated whole, as forward: 3 % slower)
        if (i < 2 ? p.rot1 : p.rot2) {
          const uint64_t x = gu[i], y = gv[i];
          gu[i] = ffma2(y, s[i], fmul2(x, c[i]));
          gv[i] = ffma2(fmul2(x, s[i]), pack_f32x2(-1.f, -1.f), fmul2(y, c[i]));
        }
      if (norm) {
        uint64_t nu[4], nv[4];
        unpack_pairs<INTER>(r[64], r[96], nu, nv);
        float rstd = row_rstd(nu, nv, a.norm.eps);
        if (!live) rstd = 0.f;  // (eps may be 0)
        const uint64_t r2 = pack_f32x2(rstd, rstd);
        uint64_t dot = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t x = fmul2(nu[i], r2), y = fmul2(nv[i], r2);
          const uint64_t gx = gu[i], gy = gv[i];
          nu[i] = x;
          nv[i] = y;
          if (is_k) {
            s_dwk[warp][i][lane] = ffma2(gx, x, s_dwk[warp][i][lane]);
            s_dwk[warp][4 + i][lane] = ffma2(gy, y, s_dwk[warp][4 + i][lane]);
          } else {
            dwu[i] = ffma2(gx, x, dwu[i]);
            dwv[i] = ffma2(gy, y, dwv[i]);
          }
          const uint64_t hx = fmul2(gx, wu[i]), hy = fmul2(gy, wv[i]);
          dot = ffma2(hy, y, ffma2(hx, x, dot));
          gu[i] = hx;
          gv[i] = hy;
        }
        const float2 d = unpack_f32x2(dot);
        const float mean = row_sum(d.x + d.y) * (-1.f / kHeadDim);
        const uint64_t m2 = pack_f32x2(mean, mean);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          gu[i] = fmul2(r2, ffma2(nu[i], m2, gu[i]));
          gv[i] = fmul2(r2, ffma2(nv[i], m2, gv[i]));
        }
      }
      pack_pairs<INTER>(gu, gv, y1, y2);
    }
    if (live) {
      *reinterpret_cast<uint4*>(dst) = y1;
      *reinterpret_cast<uint4*>(dst + d2) = y2;
    }
    dst += items.kStride;
    fresh = items.next(at);
  }
  if (!a.partial) return;
  // the four rows of a warp, then the eight warps in order: one partial row a block
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 ku = unpack_f32x2(s_dwk[warp][i >> 1][lane]);
    const float2 kv = unpack_f32x2(s_dwk[warp][4 + (i >> 1)][lane]);
    const float2 qu = unpack_f32x2(dwu[i >> 1]), qv = unpack_f32x2(dwv[i >> 1]);
    float x[4] = {(i & 1) ? qu.y : qu.x, (i & 1) ? qv.y : qv.x, (i & 1) ? ku.y : ku.x,
                  (i & 1) ? kv.y : kv.x};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] += __shfl_xor_sync(0xffffffffu, x[j], 8);
      x[j] += __shfl_xor_sync(0xffffffffu, x[j], 16);
    }
    if (lane < 8) {
      const int du = INTER ? 8 * (i < 4 ? p.c1 : p.c2) + 2 * (i & 3) : 8 * p.c1 + i;
      const int dv = INTER ? du + 1 : 8 * p.c2 + i;
      s_dw[warp][du] = x[0];
      s_dw[warp][dv] = x[1];
      s_dw[warp][kHeadDim + du] = x[2];
      s_dw[warp][kHeadDim + dv] = x[3];
    }
  }
  __syncthreads();
  float sum = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) sum += s_dw[w][threadIdx.x];
  a.partial[(int64_t)blockIdx.x * (2 * kHeadDim) + threadIdx.x] = sum;
}

// dw[d] = the blocks' partials added up in block order: 32 columns a block, eight threads a
// column (every eighth partial), then those eight in order.  (32 threads a column: 0.5 us
// longer at 1021 tokens.)
__global__ void __launch_bounds__(256)
    norm_rope_dw_kernel(const float* __restrict__ partial, int32_t rows, float* dwq, float* dwk) {
  pdl_wait();
  pdl_trigger();
  __shared__ float s[8][32];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
  float v = 0.f;
#pragma unroll 8
  for (int r = part; r < rows; r += 8) v += partial[(int64_t)r * (2 * kHeadDim) + col];
  s[part][threadIdx.x & 31] = v;
  __syncthreads();
  if (part == 0) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += s[i][threadIdx.x];
    float* dst = col < kHeadDim ? dwq : dwk;
    if (dst) dst[col & (kHeadDim - 1)] = v;
  }
}

// Eight warps share a token while every token has a block of its own in one wave (16 + 2 heads, 296
// tokens: 3.9 us shared, 5.5 one warp each; 1021 tokens: 8.2 and 5.6).
bool split_tokens(int64_t n, int per_sm) { return n <= per_sm * (int64_t)sm_count(); }

// One wave of blocks, or as many as there are tokens for.
int64_t wave_grid(int64_t n, int per_sm) {
  const int64_t most = per_sm * (int64_t)sm_count();
  const int64_t blocks = split_tokens(n, per_sm) ? n : (n + kWarps - 1) / kWarps;
  return blocks < 1 ? 1 : blocks < most ? blocks : most;
}

}  // namespace

size_t norm_rope_bwd_workspace_bytes(int64_t n) {
  return size_t(wave_grid(n, kBwdBlocksPerSm)) * 2 * kHeadDim * sizeof(float);
}

template <int SPLIT, bool INTER>
static int launch_forward(const NormRopeArgs& a, cudaStream_t stream) {
  constexpr size_t ring = kWarps * (kAhead + 1) * 2 * 32 * sizeof(uint4);
  PS_TRY((allow_smem<norm_rope_kernel<SPLIT, INTER>>(ring)));
  return check_cuda(
      launch_pdl(norm_rope_kernel<SPLIT, INTER>,
                 dim3(static_cast<unsigned>(wave_grid(a.n, kBlocksPerSm))), dim3(kThreads), ring,
                 stream, a),
      "norm_rope_kernel launch");
}

int launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream) {
  if (split_tokens(a.n, kBlocksPerSm))
    return a.rope.interleaved ? launch_forward<kWarps, true>(a, stream)
                              : launch_forward<kWarps, false>(a, stream);
  return a.rope.interleaved ? launch_forward<1, true>(a, stream)
                            : launch_forward<1, false>(a, stream);
}

template <int SPLIT, bool INTER>
static int launch_backward(const NormRopeBwdArgs& a, int64_t grid, cudaStream_t stream) {
  constexpr size_t ring = kWarps * (kBwdAhead + 1) * 4 * 32 * sizeof(uint4);
  PS_TRY((allow_smem<norm_rope_bwd_kernel<SPLIT, INTER>>(ring)));
  return check_cuda(launch_pdl(norm_rope_bwd_kernel<SPLIT, INTER>,
                               dim3(static_cast<unsigned>(grid)), dim3(kThreads), ring, stream, a),
                    "norm_rope_bwd_kernel launch");
}

int launch_norm_rope_bwd(const NormRopeBwdArgs& a, float* dwq, float* dwk, cudaStream_t stream) {
  const int64_t grid = wave_grid(a.n, kBwdBlocksPerSm);  // (no tokens: one block leaves zeros)
  int rc;
  if (split_tokens(a.n, kBwdBlocksPerSm))
    rc = a.rope.interleaved ? launch_backward<kWarps, true>(a, grid, stream)
                            : launch_backward<kWarps, false>(a, grid, stream);
  else
    rc = a.rope.interleaved ? launch_backward<1, true>(a, grid, stream)
                            : launch_backward<1, false>(a, grid, stream);
  PS_TRY(rc);
  if (!dwq && !dwk) return PS_OK;
  return check_cuda(launch_pdl(norm_rope_dw_kernel, dim3(2 * kHeadDim / 32), dim3(256), 0, stream,
                               static_cast<const float*>(a.partial), static_cast<int32_t>(grid),
                               dwq, dwk),
                    "norm_rope_dw_kernel launch");
}

}  // namespace ps
