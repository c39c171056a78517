// Norm and rotation of queries and keys in one pass, and its backward, sm_100a.
//
//   forward:  y = R(p) (x rstd w),  rstd = 1 / sqrt(mean x^2 + eps)
//   backward: g = R(p)^T dy,  n = x rstd,  dw = sum g n,  dx = rstd (w g - n mean(w g n))
// Both stream every row once (forward one read and one write of each bf16 row, backward two
// reads and one write) and are bound by HBM; the arithmetic is a few fp32 operations an element
// and the token's angles, formed once per token in float64 and shared by all its heads.
#include <cuda_bf16.h>

#include "ps_norm_rope.cuh"

namespace ps {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// One item: four heads of one token's q or k.
struct Item {
  const __nv_bfloat16* src;
  __nv_bfloat16* dst;
  bool is_k, live;  // live: this lane's head exists
};

// One block handles TT tokens.
template <int TT>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRopeArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ __align__(16) float s_cos[TT][kHalfDim];
  __shared__ __align__(16) float s_sin[TT][kHalfDim];
  __shared__ __align__(16) float s_w[2 * kHeadDim];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t tok0 = (int64_t)blockIdx.x * TT;
  const int ntok = static_cast<int>(a.n - tok0 < TT ? a.n - tok0 : TT);
  const RopeLane p = rope_lane(a.rope, lane & 7);
  const int nq = a.q ? (a.hq + 3) / 4 : 0;
  const int nk = a.k ? (a.hkv + 3) / 4 : 0;
  const int per = nq + nk;

  for (int i = threadIdx.x; i < ntok * (a.rope.dim / 2); i += kThreads) {
    const int t = i / (a.rope.dim / 2), f = i % (a.rope.dim / 2);
    const int64_t pos = a.pos[tok0 + t];
    if (!bad_rope_position(pos)) rope_angle(a.rope, pos, f, s_cos[t], s_sin[t]);
  }
  load_norm_weights(a.norm, s_w);
  if (threadIdx.x < ntok && a.status) {
    const int64_t pos = a.pos[tok0 + threadIdx.x];
    if (bad_rope_position(pos)) atomicOr(a.status, rope_position_flag(pos));
  }
  __syncthreads();

  for (int it = warp; it < ntok * per; it += kWarps) {
    const int t = it / per, sub = it % per;
    const int64_t tok = tok0 + t;
    const bool is_k = sub >= nq;
    const int head = 4 * (is_k ? sub - nq : sub) + (lane >> 3);
    const int heads = is_k ? a.hkv : a.hq;
    const bool live = head < heads;
    const __nv_bfloat16* src =
        (is_k ? a.k + tok * a.k_stride : a.q + tok * a.q_stride) + head * kHeadDim;
    __nv_bfloat16* dst = (is_k ? a.k_out : a.q_out) + (tok * heads + head) * kHeadDim;
    uint4 v1 = make_uint4(0, 0, 0, 0), v2 = v1;
    if (live) {
      v1 = *reinterpret_cast<const uint4*>(src + 8 * p.c1);
      v2 = *reinterpret_cast<const uint4*>(src + 8 * p.c2);
    }
    float x[16];
    unpack8(v1, x);
    unpack8(v2, x + 8);
    norm_and_turn(a.rope, p, (is_k ? a.norm.wk : a.norm.wq) != nullptr,
                  s_w + (is_k ? kHeadDim : 0), a.norm.eps, s_cos[t], s_sin[t], x);
    if (bad_rope_position(a.pos[tok])) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = 0.f;
    }
    if (live) {
      *reinterpret_cast<uint4*>(dst + 8 * p.c1) = pack8(x);
      *reinterpret_cast<uint4*>(dst + 8 * p.c2) = pack8(x + 8);
    }
  }
}

// Backward; blocks stride over groups of kBwdTokens tokens and keep their share of the weights'
// gradients in registers: every lane holds sixteen dims of q's and of k's.
constexpr int kBwdTokens = 4;

__global__ void __launch_bounds__(kThreads, 2) norm_rope_bwd_kernel(const NormRopeBwdArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ __align__(16) float s_cos[kBwdTokens][kHalfDim];
  __shared__ __align__(16) float s_sin[kBwdTokens][kHalfDim];
  __shared__ __align__(16) float s_w[2 * kHeadDim];
  __shared__ float s_dw[kWarps][2 * kHeadDim];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const RopeLane p = rope_lane(a.rope, lane & 7);
  const int nq = a.dq_out ? (a.hq + 3) / 4 : 0;
  const int nk = a.dk_out ? (a.hkv + 3) / 4 : 0;
  const int per = nq + nk;
  float dwq[16], dwk[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) dwq[i] = dwk[i] = 0.f;
  load_norm_weights(a.norm, s_w);

  for (int64_t tok0 = (int64_t)blockIdx.x * kBwdTokens; tok0 < a.n;
       tok0 += (int64_t)gridDim.x * kBwdTokens) {
    const int ntok = static_cast<int>(a.n - tok0 < kBwdTokens ? a.n - tok0 : kBwdTokens);
    __syncthreads();
    for (int i = threadIdx.x; i < ntok * (a.rope.dim / 2); i += kThreads) {
      const int t = i / (a.rope.dim / 2), f = i % (a.rope.dim / 2);
      const int64_t pos = a.pos[tok0 + t];
      if (!bad_rope_position(pos)) rope_angle(a.rope, pos, f, s_cos[t], s_sin[t]);
    }
    if (threadIdx.x < ntok && a.status) {
      const int64_t pos = a.pos[tok0 + threadIdx.x];
      if (bad_rope_position(pos)) atomicOr(a.status, rope_position_flag(pos));
    }
    __syncthreads();
    for (int it = warp; it < ntok * per; it += kWarps) {
      const int t = it / per, sub = it % per;
      const int64_t tok = tok0 + t;
      const bool is_k = sub >= nq;
      const int head = 4 * (is_k ? sub - nq : sub) + (lane >> 3);
      const int heads = is_k ? a.hkv : a.hq;
      const bool bad = bad_rope_position(a.pos[tok]);
      const bool live = head < heads;
      const bool norm = (is_k ? a.norm.wk : a.norm.wq) != nullptr;
      const __nv_bfloat16* gsrc =
          (is_k ? a.dk_out : a.dq_out) + (tok * heads + head) * kHeadDim;
      const __nv_bfloat16* xsrc =
          (is_k ? a.k + tok * a.k_stride : a.q + tok * a.q_stride) + head * kHeadDim;
      __nv_bfloat16* dst =
          (is_k ? a.dk + tok * a.dk_stride : a.dq + tok * a.dq_stride) + head * kHeadDim;
      const uint4 z = make_uint4(0, 0, 0, 0);
      uint4 g1 = z, g2 = z, x1 = z, x2 = z;
      if (live && !bad) {
        g1 = *reinterpret_cast<const uint4*>(gsrc + 8 * p.c1);
        g2 = *reinterpret_cast<const uint4*>(gsrc + 8 * p.c2);
        if (norm) {
          x1 = *reinterpret_cast<const uint4*>(xsrc + 8 * p.c1);
          x2 = *reinterpret_cast<const uint4*>(xsrc + 8 * p.c2);
        }
      }
      float g[16];
      unpack8(g1, g);
      unpack8(g2, g + 8);
      if (!bad) rope_turn<-1>(a.rope, p, s_cos[t], s_sin[t], g);
      if (norm) {
        float x[16], w[16];
        unpack8(x1, x);
        unpack8(x2, x + 8);
        const float rstd = row_rstd(x, a.norm.eps);
        lane_weights(s_w + (is_k ? kHeadDim : 0), p, w);
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          x[i] *= rstd;  // n
          const float gn = (live && !bad) ? g[i] * x[i] : 0.f;
          if (is_k) dwk[i] += gn; else dwq[i] += gn;
          dot = fmaf(w[i], gn, dot);
        }
        const float mean = row_sum(dot) * (1.f / kHeadDim);
#pragma unroll
        for (int i = 0; i < 16; ++i) g[i] = rstd * (w[i] * g[i] - x[i] * mean);
      }
      if (live) {
        uint4 y1 = pack8(g), y2 = pack8(g + 8);
        if (bad) y1 = y2 = z;
        *reinterpret_cast<uint4*>(dst + 8 * p.c1) = y1;
        *reinterpret_cast<uint4*>(dst + 8 * p.c2) = y2;
      }
    }
  }
  if (!a.partial) return;
  // the four rows of a warp, then the eight warps in order: one partial row a block
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    dwq[i] += __shfl_xor_sync(0xffffffffu, dwq[i], 8);
    dwq[i] += __shfl_xor_sync(0xffffffffu, dwq[i], 16);
    dwk[i] += __shfl_xor_sync(0xffffffffu, dwk[i], 8);
    dwk[i] += __shfl_xor_sync(0xffffffffu, dwk[i], 16);
  }
  if (lane < 8) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int d = 8 * (i < 8 ? p.c1 : p.c2) + (i & 7);
      s_dw[warp][d] = dwq[i];
      s_dw[warp][kHeadDim + d] = dwk[i];
    }
  }
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += s_dw[w][threadIdx.x];
  a.partial[(int64_t)blockIdx.x * (2 * kHeadDim) + threadIdx.x] = s;
}

// dw[d] = the blocks' partials added up in block order: 32 columns a block, eight threads a
// column (every eighth partial), then those eight in order.
__global__ void __launch_bounds__(256)
    norm_rope_dw_kernel(const float* __restrict__ partial, int32_t rows, float* dwq, float* dwk) {
  pdl_wait();
  pdl_trigger();
  __shared__ float s[8][32];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
  float v = 0.f;
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

int64_t bwd_grid(int64_t n) {
  const int64_t groups = (n + kBwdTokens - 1) / kBwdTokens;
  const int64_t most = 2 * (int64_t)sm_count();
  return groups < most ? groups : most;
}

}  // namespace

size_t norm_rope_bwd_workspace_bytes(int64_t n) {
  return size_t(bwd_grid(n > 0 ? n : 1)) * 2 * kHeadDim * sizeof(float);
}

int launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream) {
  // four tokens a block share the set-up once there are blocks enough for every SM
  const bool wide = a.n > 8 * (int64_t)sm_count();
  const int64_t grid = wide ? (a.n + 3) / 4 : a.n;
  if (grid > 0x7fffffff) return fail(PS_ERR_UNSUPPORTED, "too many tokens");
  return check_cuda(launch_pdl(wide ? norm_rope_kernel<4> : norm_rope_kernel<1>,
                               dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, stream, a),
                    "norm_rope_kernel launch");
}

int launch_norm_rope_bwd(const NormRopeBwdArgs& a, float* dwq, float* dwk, cudaStream_t stream) {
  const int64_t grid = bwd_grid(a.n > 0 ? a.n : 1);  // no tokens: the weights' gradients are 0
  PS_TRY(check_cuda(launch_pdl(norm_rope_bwd_kernel, dim3(static_cast<unsigned>(grid)),
                               dim3(kThreads), 0, stream, a),
                    "norm_rope_bwd_kernel launch"));
  if (!dwq && !dwk) return PS_OK;
  return check_cuda(launch_pdl(norm_rope_dw_kernel, dim3(2 * kHeadDim / 32), dim3(256), 0, stream,
                               static_cast<const float*>(a.partial), static_cast<int32_t>(grid),
                               dwq, dwk),
                    "norm_rope_dw_kernel launch");
}

}  // namespace ps
