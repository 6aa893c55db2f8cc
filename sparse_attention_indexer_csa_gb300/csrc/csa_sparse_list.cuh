// csa_sparse_list.cuh -- what the kernels of attention over listed blocks share:
// the keys that a row lists, and the maps of its queries.
#pragma once

#include "csa_attn_tiles.cuh"
#include "csa_sparse_internal.h"

namespace csa {

// ----------------------------------------------------------------- TMA maps (host)
// Heads of q (or dout): dims (D, Hq, Tq), box {64, heads, 1}.
inline bool make_heads_map(CUtensorMap* m, const SparseParams& p, const void* x, long long st, long long sh, int heads) {
  auto fn = attn_encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[3] = {(cuuint64_t)p.D, (cuuint64_t)p.Hq, (cuuint64_t)p.Tq};
  cuuint64_t strides[2] = {(cuuint64_t)sh * 2, (cuuint64_t)st * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)heads, 1}, estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(x), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// ----------------------------------------------------------------- lists
// The sequence of a query row: keys k0 .. k0+lk-1 (counted from 0 in a paged
// cache), the row's position, the sequence's number (-1: none, lk = 0).
struct ListRow {
  int seq, k0, lk, pos;
};

// Extents of sequence i, clamped to the tensors; what was clamped is recorded.
__device__ __forceinline__ SeqExt sparse_extent(const SparseParams& p, int i) {
  SeqExt s;
  const int a = p.cu_q[i], b = p.cu_q[i + 1];
  s.q0 = min(max(a, 0), p.Tq);
  s.q1 = min(max(b, s.q0), p.Tq);
  bool bad = a != s.q0 || b != s.q1;
  long long most;
  if (p.page > 0) {
    s.k0 = 0;
    most = static_cast<long long>(p.table_width) * p.page;
  } else {
    const int c = p.cu_k[i], d = p.cu_k[i + 1];
    s.k0 = min(max(c, 0), p.Tk);
    const int k1 = min(max(d, s.k0), p.Tk);
    bad |= c != s.k0 || d != k1;
    most = k1 - s.k0;
  }
  s.lk = static_cast<int>(min(most, 0x7FFFFFFFll));
  if (p.k_len != nullptr) {
    const int n = p.k_len[i], m = min(max(n, 0), s.lk);
    bad |= n != m;
    s.lk = m;
  }
  if (bad) record_error(kErrDevice);
  return s;
}

// The row's sequence, by a warp: the largest i with cu_q[i] <= t.  Sequences of
// equal lengths (one token each, when decoding) are met at the first look, others
// by 32 probes at a time.  Entries out of order give some sequence or none.
__device__ __forceinline__ ListRow find_list_row(const SparseParams& p, int t) {
  const int lane = static_cast<int>(lane_id());
  ListRow r{-1, 0, 0, -1};
  if (p.N <= 0) return r;
  int lo = static_cast<int>(static_cast<long long>(t) * p.N / p.Tq);
  if (t < p.cu_q[lo] || t >= p.cu_q[lo + 1]) {
    lo = 0;
    int hi = p.N;
    while (lo < hi) {
      const int span = hi - lo, stride = (span + 31) / 32;
      const int i = lo + min(span, (lane + 1) * stride);
      const unsigned out = __ballot_sync(0xffffffffu, p.cu_q[i] > t);
      if (out == 0u) {
        lo = hi;
      } else {
        const int n = __ffs(static_cast<int>(out)) - 1;
        hi = lo + min(span, (n + 1) * stride) - 1;
        lo = lo + min(span, n * stride);
      }
    }
    if (lo >= p.N) return r;
  }
  const SeqExt s = sparse_extent(p, lo);
  if (t < s.q0 || t >= s.q1) return r;
  r.seq = lo;
  r.k0 = s.k0;
  r.lk = s.lk;
  r.pos = p.causal ? t - s.q0 + s.lk - (s.q1 - s.q0) : s.lk - 1;
  return r;
}

// The slots of a row's list: first the window, newest key first, then top_k
// blocks.  A slot in three steps, so that the loads of the coming slots are in
// flight while the present ones are dealt with.  `bad` gathers what is out of range.
struct Slot {
  int j;     // key of the sequence; -1: none
  int page;  // its page (paged keys)
};
__device__ __forceinline__ int slot_block(const SparseParams& p, const int32_t* list, int s, int slots) {
  return s >= p.window && s < slots ? list[(s - p.window) >> p.block_shift] : -1;
}
__device__ __forceinline__ Slot slot_key(const SparseParams& p, const ListRow& r, int s, int slots, int b, bool& bad) {
  Slot x{-1, 0};
  if (s < p.window) {
    x.j = r.pos - s;  // negative: before the first key
  } else if (s < slots) {
    if (static_cast<unsigned>(b) <= static_cast<unsigned>((r.lk - 1) >> p.block_shift)) {
      const int j = (b << p.block_shift) + ((s - p.window) & ((1 << p.block_shift) - 1));
      if (j < r.lk && j <= r.pos - p.window) x.j = j;
    } else {
      bad |= b != -1;
    }
  }
  if (p.page > 0 && x.j >= 0) x.page = p.table[r.seq * p.table_st + x.j / p.page];
  return x;
}
// Rows of keys and values of slot x (key head 0); false: it has none.
__device__ __forceinline__ bool slot_rows(const SparseParams& p, const ListRow& r, const Slot& x, int& kr, int& vr,
                                          bool& bad) {
  if (x.j < 0) return false;
  if (p.page > 0) {
    if (static_cast<unsigned>(x.page) >= static_cast<unsigned>(p.pages)) {
      bad = true;
      return false;
    }
    const int off = x.j % p.page;
    kr = x.page * p.k.rp + off * p.k.rt;
    vr = x.page * p.v.rp + off * p.v.rt;
  } else {
    kr = (r.k0 + x.j) * p.k.rt;
    vr = (r.k0 + x.j) * p.v.rt;
  }
  return true;
}

}  // namespace csa
