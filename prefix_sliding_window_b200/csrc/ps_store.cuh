// Where a position's row lives in a prefix + ring store (contiguous or paged), for the kernels
// that take StoreArgs.
#pragma once

#include "ps_internal.h"
#include "ps_ranges.cuh"

namespace ps {

constexpr int kQ4RowBytes = 64;     // payload of a row: 128 4-bit codes
constexpr int kQ4RecordBytes = 16;  // K's and V's (s, m) of two groups

// Row `row` (of one KV head) in array `ring` (0: prefix, 1: ring) of sequence b; `flag` is the
// dev_status bit where there is none.
struct StoreRow {
  int32_t ring;
  int64_t unit;    // row index of the head-0 row, heads `stride` rows apart
  int64_t stride;
  int32_t flag;    // 0: the row exists
};

__device__ __forceinline__ StoreRow store_row(const StoreArgs& st, int32_t hkv, int64_t b,
                                              int64_t p) {
  StoreRow r{0, 0, 0, 0};
  if (p < 0 || p >= (1ll << 31)) {
    r.flag = p < 0 ? PS_DEV_BAD_POS : PS_DEV_POS_RANGE;
    return r;
  }
  r.ring = p >= st.lp;
  if (st.linear ? r.ring : (!r.ring && !st.k[0])) {  // past a linear store; below a ring-only one
    r.flag = PS_DEV_POS_RANGE;
    return r;
  }
  const int64_t row = r.ring ? mod_nonneg(p - st.lp, st.w) : p;
  if (st.table) {
    const int64_t i = (r.ring ? st.pre_blocks : 0) + row / 64;
    const int32_t blk = st.table[b * st.table_stride + i];
    if (blk < 0 || blk >= st.n_blocks) r.flag = PS_DEV_POS_RANGE;
    r.ring = 0;  // one pool holds both
    r.stride = 64;
    r.unit = (int64_t)blk * hkv * 64 + row % 64;
  } else {
    r.stride = r.ring ? st.w : st.lp;
    r.unit = b * hkv * r.stride + row;
  }
  return r;
}

}  // namespace ps
