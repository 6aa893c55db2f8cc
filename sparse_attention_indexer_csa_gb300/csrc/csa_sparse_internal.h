// csa_sparse_internal.h -- host-side interface between the C ABI of csa_sparse.h
// (csa_sparse_api.cu) and the translation units that launch the kernels.
#pragma once

#include <algorithm>

#include "csa_attn_internal.h"
#include "csa_sparse.h"

namespace csa {

// ----------------------------------------------------------------- attention over listed blocks
// Rows of keys or of values: row j of key head h starts at
// (page * rp +) j * rt + h * rh units, a unit being the strides' greatest common
// divisor, so that a row's number fits 32 bits in a long cache.
struct GatherRows {
  const void* base;
  uint32_t unit_bytes;
  int rp, rt, rh;  // units between pages, tokens, heads
};
struct SparseParams {
  int N, Tq, Tk, Hq, Hk, g, D;  // g = Hq / Hk
  int top_k, block_shift, window, causal;
  int page, pages, table_width;
  uint32_t page_mul, page_shift;  // division by page: multiply, shift
  float scale;
  const void* q;
  long long q_st, q_sh, idx_st, table_st;
  GatherRows k, v;
  const int32_t *idx, *cu_q, *cu_k, *k_len, *table;
  void* out;
  float* lse;
  // backward
  const void* dout;
  void *dq, *dk, *dv;
};
inline long long sparse_slots(const SparseParams& p) {
  return p.window + (static_cast<long long>(p.top_k) << p.block_shift);
}
cudaError_t launch_sparse_forward(const SparseParams& p, int dtype, void* workspace, cudaStream_t stream);
cudaError_t launch_sparse_backward(const SparseParams& p, int dtype, void* workspace, cudaStream_t stream);
size_t sparse_backward_workspace(const SparseParams& p, int dtype);
cudaError_t take_status_sparse_fwd(uint32_t* out, cudaStream_t stream);
cudaError_t take_status_sparse_bwd(uint32_t* out, cudaStream_t stream);

// Shares of a row's list: few rows are cut so that all SMs have work, in shares
// of at least two tiles of 128 slots.
inline int sparse_splits(int Tq, int Hk, long long slots) {
  const long long items = std::max(1ll, static_cast<long long>(Tq) * Hk), tiles = (slots + 127) / 128;
  if (2 * items > 152) return 1;
  return static_cast<int>(std::max(1ll, std::min({152 / items, tiles / 2, static_cast<long long>(kMaxSplit)})));
}

// ----------------------------------------------------------------- append to a paged cache
struct AppendParams {
  int N, pages, page, table_width;
  long long table_st;
  const void* v;
  long long v_st, v_sh;
  void *kc, *vc;
  long long kc_sp, kc_st, kc_sh, vc_sp, vc_st, vc_sh;
  const int32_t *cu_q, *k_len, *table;
};
cudaError_t launch_norm_rope_append(const NormRopeParams& p, const AppendParams& c, int dtype, bool inter,
                                    cudaStream_t stream);
cudaError_t take_status_append(uint32_t* out, cudaStream_t stream);

}  // namespace csa
