// Decode attention over the 4-bit store, sm_100a.
//
// The query of sequence b at position p attends its visible rows (prefix rows, then the window's
// ring slots), each standing for m_g + s_g u_d in its two groups g of 64 dims:
//   S_k = sum_g s_kg (sum_d q_d u_kd) + m_kg sum_{d in g} q_d
//   o_d = sum_k p_k (m_kg + s_kg u_kd) / sum_k p_k,  p = softmax(scale S)
// One block per (sequence, query head): four warps take every fourth visible row, four dims a
// lane (one warp reads a row's 64 bytes and its record), with an online softmax in fp32 per warp.
#include <cuda_bf16.h>
#include <math.h>

#include "ps_device.cuh"
#include "ps_internal.h"
#include "ps_ranges.cuh"
#include "ps_store.cuh"

namespace ps {
namespace {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct DecodeQ4Args {
  const __nv_bfloat16* q;
  const int64_t* pos;
  __nv_bfloat16* out;
  float* lse;
  int32_t* status;
  int32_t batch, hq, hkv;
  float scale_log2;
  StoreArgs store;
};

__device__ __forceinline__ int64_t visible_rows(const DecodeQ4Args& a, int64_t p) {
  if (p < 0 || p >= (1ll << 31) || (a.store.linear && p >= a.store.lp)) return 0;
  const int64_t n = p + 1, cap = (int64_t)a.store.lp + (a.store.linear ? 0 : a.store.w);
  return n < cap ? n : cap;
}

__global__ void __launch_bounds__(kWarps * 32) decode_q4_kernel(const DecodeQ4Args a) {
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / a.hq, head = blockIdx.x % a.hq, h = head / (a.hq / a.hkv);
  const int64_t p = a.pos[b];
  const int64_t n = visible_rows(a, p);
  if (n == 0 && threadIdx.x == 0 && a.status)
    atomicOr(a.status, p < 0 ? PS_DEV_BAD_POS : PS_DEV_POS_RANGE);
  // word `lane >> 1` holds eight dims; this lane takes four codes of it
  const int word = lane >> 1, g = word & 1, blk8 = word >> 1;
  const int e0 = 4 * (lane & 1);
  float q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    q[i] = __bfloat162float(
        a.q[((int64_t)b * a.hq + head) * kHeadDim + 64 * g + 8 * blk8 + e0 + i]);
  float M = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  const int64_t pre = n < a.store.lp ? n : a.store.lp;
  for (int64_t v = warp; v < n; v += kWarps) {
    // visible row v: prefix position v, or the window's (v - pre)-th oldest
    const int64_t at = v < pre ? v : p + 1 - (n - v);
    const StoreRow row = store_row(a.store, a.hkv, b, at);
    if (row.flag) {
      if (lane == 0 && a.status) atomicOr(a.status, row.flag);
      continue;
    }
    const int64_t r = row.unit + h * row.stride;
    const uint32_t kw = *reinterpret_cast<const uint32_t*>(a.store.k[row.ring] + r * 64 + 4 * word);
    const uint32_t vw = *reinterpret_cast<const uint32_t*>(a.store.v[row.ring] + r * 64 + 4 * word);
    const uint4 rec = *reinterpret_cast<const uint4*>(a.store.s[row.ring] + r * 16);
    const uint32_t kr = g ? rec.y : rec.x, vr = g ? rec.w : rec.z;
    const float ks = __uint_as_float(kr << 16), km = __uint_as_float(kr & 0xffff0000u);
    const float vs = __uint_as_float(vr << 16), vm = __uint_as_float(vr & 0xffff0000u);
    float s = 0.f, val[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = e0 + i, bit = 4 * (e >> 1) + 16 * (e & 1);
      s = fmaf(q[i], fmaf(ks, static_cast<float>((kw >> bit) & 15u), km), s);
      val[i] = fmaf(vs, static_cast<float>((vw >> bit) & 15u), vm);
    }
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= a.scale_log2;
    const float Mn = fmaxf(M, s);
    const float c = exp2f(M - Mn), e = exp2f(s - Mn);
    l = l * c + e;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = o[i] * c + e * val[i];
    M = Mn;
  }
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][32][4];
  if (lane == 0) s_m[warp] = M, s_l[warp] = l;
#pragma unroll
  for (int i = 0; i < 4; ++i) s_o[warp][lane][i] = o[i];
  __syncthreads();
  if (warp != 0) return;
  float Mx = -INFINITY, L = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int w = 0; w < kWarps; ++w) Mx = fmaxf(Mx, s_m[w]);
  for (int w = 0; w < kWarps; ++w) {
    const float f = s_m[w] == -INFINITY ? 0.f : exp2f(s_m[w] - Mx);
    L += f * s_l[w];
    for (int i = 0; i < 4; ++i) acc[i] += f * s_o[w][lane][i];
  }
  const int64_t row = (int64_t)b * a.hq + head;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    a.out[row * kHeadDim + 64 * g + 8 * blk8 + e0 + i] =
        __float2bfloat16_rn(L == 0.f ? 0.f : acc[i] / L);
  if (a.lse && lane == 0) a.lse[row] = L == 0.f ? -INFINITY : (Mx + log2f(L)) * kLn2;
}

}  // namespace

size_t decode_q4_workspace_bytes(int64_t, int32_t, int64_t) { return 0; }

int launch_decode_q4(const DecodeQ4Launch& l, cudaStream_t stream) {
  const int64_t grid = l.batch * l.hq;
  if (grid <= 0) return PS_OK;
  if (grid > 0x7fffffff) return fail(PS_ERR_UNSUPPORTED, "decode grid too large");
  DecodeQ4Args a;
  a.q = static_cast<const __nv_bfloat16*>(l.q);
  a.pos = l.pos;
  a.out = static_cast<__nv_bfloat16*>(l.out);
  a.lse = l.lse;
  a.status = l.status;
  a.batch = static_cast<int32_t>(l.batch);
  a.hq = l.hq;
  a.hkv = l.hkv;
  a.scale_log2 = l.scale * kLog2e;
  a.store = l.store;
  return check_cuda(launch_pdl(decode_q4_kernel, dim3(static_cast<unsigned>(grid)),
                               dim3(kWarps * 32), 0, stream, a),
                    "decode_q4_kernel launch");
}

}  // namespace ps
