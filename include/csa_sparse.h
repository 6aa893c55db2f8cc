/*
 * csa_sparse.h -- C ABI of the operators that use the indexer's selection and
 * of the cache that they read: attention over listed blocks of keys (forward,
 * gradients, over a paged cache), and the norm and rotation of new tokens with
 * their append to that cache.
 *
 * They are exported by libcsa_index.so beside the entry points of csa_index.h
 * and csa_attn.h and follow their conventions: device pointers owned by the
 * caller, work enqueued on `stream` on the current device, no allocation and
 * no synchronisation, arguments checked on the host before anything is
 * launched (CSA_ERR_INVALID_ARG, CSA_ERR_UNSUPPORTED; no fallback),
 * CSA_ERR_CUDA for a failed launch, csa_index_device_status() for what a
 * kernel recorded.  Workspaces are the caller's; their contents need no
 * clearing, and calls that may be in flight together need separate ones.
 */
#ifndef CSA_SPARSE_H
#define CSA_SPARSE_H

#include "csa_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- attention over listed blocks
 * N sequences packed one behind the other, as for csa_attn_forward: sequence i
 * has the query rows cu_q[i] .. cu_q[i+1]-1 of q [Tq,Hq,D] and lk keys.
 * Query head h reads key head h / (Hq/Hk).  A sequence's keys 0 .. lk-1 are cut
 * into blocks of `block`; row t lists idx[t,0..top_k-1], block numbers within
 * its own sequence (a selection of csa_index_fused with its [B,S,top_k] read as
 * [B*S,top_k], or any other list in any order); -1 lists nothing.
 *   causal = 1: row r of lq stands at the position pos = r + lk - lq (the last
 *     query at the last key) and sees the last `window` keys j, pos - window < j
 *     <= pos, and the listed blocks' keys j <= pos - window.
 *   causal = 0: it sees all keys of the listed blocks (compressed entries whose
 *     visibility the selection has settled); window is 0.
 * So a key in the window counts once, listed or not.  The blocks of a list are
 * distinct; a block that is listed twice counts twice.
 *   s_j = scale * q.k_j,  out = sum_j softmax(s)_j v_j,  lse = log sum_j exp(s_j)
 * over the keys a row sees.  A row that sees none, and a row outside every
 * sequence, gives out = 0 and lse = -inf.  Keys that a row does not see are not
 * read for it and may hold anything, also NaN.
 *
 * Keys, packed (page = 0): k, v [Tk,Hk,D], sequence i has cu_k[i] ..
 *   cu_k[i+1]-1, with k_len given only the first k_len[i] of those.
 * Keys, paged (page > 0): k, v [pages,page,Hk,D] with Tk = pages * page; key j
 *   of sequence i is row j % page of page table[i * table_stride + j / page],
 *   table [N,table_width] int32; lk = k_len[i] (not NULL); cu_k is NULL.  Pages
 *   may be in any order and shared by sequences.
 *
 *   cu_q, cu_k [N+1], k_len [N], table and idx are int32 device memory.  Entries
 *   of cu_q, cu_k, k_len out of order or range are clamped; block numbers below
 *   -1 or past a row's sequence, and pages outside 0 .. pages-1, are skipped;
 *   each records CSA_ERR_DEVICE in the device status word and is never followed.
 *   Strides in elements between pages, tokens and heads (0 = contiguous); the
 *   innermost dimension is contiguous.  Bases are 16-byte aligned and strides of q, k
 *   and v multiples of 8 elements (a view of a projection's output, pages with
 *   keys and values side by side).  out, lse, the cotangent and the gradients are
 *   contiguous with 16-byte aligned bases.
 * Precision: as for csa_attn_forward: products of stored values are exact and
 * summed in fp32, as are the softmax's sums; exponentials are fp32.  The weights
 * that meet v (and dout), and ds that meets k and q, are rounded to dtype, half a
 * unit of the last place each.  In bf16 the share of a row in dk and dv of a key is
 * kept with 11 bits (fp16 at a power of two of its own) before the rows' shares
 * are added in fp32; in fp16 it is fp32.  In fp16, weights
 * count down to 2^-32 of the largest in out and 2^-39 in dv; ds' range is set by the
 * values that the row sees.  Groups of more than 64 heads have two shares.
 * Supported: D in {64, 128}, dtype CSA_BF16 or CSA_F16, Hq a multiple of Hk,
 * Hq / Hk <= 128, block a power of two up to 128, window + top_k * block up to
 * 2^20, scale up to 2^127, top_k >= 0 (0: idx is NULL), Tq, Tk, N >= 0; k and v span less than 2^31
 * times the greatest common divisor of their strides.                          */
typedef struct {
  int32_t N, Tq, Tk, Hq, Hk, D;
  int32_t top_k, block, window;
  int32_t page, table_width; /* page = 0: packed keys, no table */
  int32_t dtype, causal;
  float scale; /* > 0, up to 2^127 */
  int64_t idx_stride, table_stride; /* between rows of idx and table (0 = contiguous) */
  int64_t q_stride_t, q_stride_h;
  int64_t k_stride_p, k_stride_t, k_stride_h; /* _p: between pages */
  int64_t v_stride_p, v_stride_t, v_stride_h;
} csa_sparse_problem;

/* Writes out [Tq,Hq,D] (dtype) and lse [Tq,Hq] fp32, every element.  cu_k is
 * NULL for a paged problem, table for a packed one.  Needs `workspace`:
 * csa_sparse_attn_workspace_size(p, 0) bytes (may be 0), 16-byte aligned.      */
csa_status csa_sparse_attn_forward(const csa_sparse_problem* p, const void* q, const void* k, const void* v,
                                   const int32_t* idx, const int32_t* cu_q, const int32_t* cu_k,
                                   const int32_t* k_len, const int32_t* table, void* out, float* lse,
                                   void* workspace, size_t workspace_bytes, void* stream);

/* Gradients for the cotangent dout [Tq,Hq,D] of out, from the forward's out
 * and lse, or from those of several calls over different keys joined by their lse
 * (out = sum exp(lse_i - lse) out_i): then dq, dk and dv are this call's keys' part
 * of the gradients of the joined out.  dq [Tq,Hq,D], dk, dv [Tk,Hk,D] (dtype, every element; zero where
 * nothing reaches them).  Packed keys only (page > 0: CSA_ERR_UNSUPPORTED).  A
 * block that a row lists twice reaches dk and dv twice, as it does out.  The sums
 * are taken in a fixed order (the same bits on every call).  Needs `workspace`:
 * csa_sparse_attn_workspace_size(p, 1) bytes, 16-byte aligned: each row's share of
 * dk and dv for each key it lists, as many rows at a time as 4 GiB hold (one at
 * least; where not all, also fp32 sums of dk and dv), and the rows by key, up to
 * 1 GiB and 12 bytes for each block of keys.                                    */
csa_status csa_sparse_attn_backward(const csa_sparse_problem* p, const void* dout, const void* q, const void* k,
                                    const void* v, const void* out, const float* lse, const int32_t* idx,
                                    const int32_t* cu_q, const int32_t* cu_k, const int32_t* k_len, void* dq,
                                    void* dk, void* dv, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of device workspace: which = 0 for csa_sparse_attn_forward, 1 for
 * csa_sparse_attn_backward.  Depends only on the problem; 0 when it is invalid. */
size_t csa_sparse_attn_workspace_size(const csa_sparse_problem* p, int32_t which);

/* ---------------------------------------------------------------- append to a paged cache
 * csa_norm_rope of the new tokens' q [T,Hq,D] and k [T,Hk,D] (the problem `p`
 * with its types, strides and rotation; Hk >= 1), with k's result and the values
 * v [T,Hk,D] put into the cache: token t = cu_q[i] + r of sequence i, which has
 * lq new tokens and k_len[i] tokens with them, takes the place
 * j = k_len[i] - lq + r, row j % page of page table[i * table_stride + j / page]
 * of k_pages and v_pages [pages,page,Hk,D] (p's dtype).  q_out [T,Hq,D] is
 * contiguous.  positions [T] give the angles, as for csa_norm_rope.
 * A token whose place is negative or past the table, whose page is outside
 * 0 .. pages-1, or that belongs to no sequence, is not stored (its q_out is); the
 * first three record CSA_ERR_DEVICE.  No other row of the cache is written.  Of two
 * tokens with the same place (sequences that share a page) each value is either's.
 * Cache and inputs may not overlap.  Strides in elements, multiples of 16 bytes
 * (0 = contiguous); bases are 16-byte aligned.                                 */
typedef struct {
  int32_t N, pages, page, table_width;
  int64_t table_stride;
  int64_t v_stride_t, v_stride_h; /* of the new tokens' values */
  int64_t kc_stride_p, kc_stride_t, kc_stride_h; /* of k_pages, between pages, tokens, heads */
  int64_t vc_stride_p, vc_stride_t, vc_stride_h; /* of v_pages */
} csa_append_problem;

csa_status csa_norm_rope_append(const csa_norm_rope_problem* p, const csa_append_problem* c, const void* q,
                                const void* k, const void* v, const void* q_weight, const void* k_weight,
                                const int64_t* positions, const uint64_t* freqs, const int32_t* cu_q,
                                const int32_t* k_len, const int32_t* table, void* q_out, void* k_pages,
                                void* v_pages, void* stream);

/* Version of this header's part of the library (major * 100 + minor). */
int32_t csa_sparse_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* CSA_SPARSE_H */
