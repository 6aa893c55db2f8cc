/*
 * csa_attn.h -- C ABI of the operators around the CSA indexer: the norm and
 * rotation that make queries and keys, and causal attention over packed
 * sequences (forward, gradients, single tokens over a cache).
 *
 * They are exported by libcsa_index.so beside the entry points of
 * csa_index.h and follow its conventions: device pointers owned by the
 * caller, work enqueued on `stream` on the current device, no allocation and
 * no synchronisation, arguments checked on the host before anything is
 * launched (CSA_ERR_INVALID_ARG, CSA_ERR_UNSUPPORTED; no fallback),
 * CSA_ERR_CUDA for a failed launch, csa_index_device_status() for what a
 * kernel recorded.  Workspaces are the caller's; their contents need no
 * clearing, and calls that may be in flight together need separate ones.
 */
#ifndef CSA_ATTN_H
#define CSA_ATTN_H

#include "csa_index.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Third storage type, beside CSA_BF16 and CSA_F32 of csa_dtype. */
enum { CSA_F16 = 2 };

/* ---------------------------------------------------------------- norm + rotation
 * For every token t and head h of q (and of k), x = q[t,h,:], D values:
 *   n = x * rsqrt(mean(x^2) + eps) * w                     (w: q_weight or k_weight)
 *   the rot values from rot_offset on are turned in pairs by the angle
 *   a_i = positions[t] * theta^(-2i/rot), i = 0 .. rot/2-1:
 *     (u, v) -> (u cos a_i - v sin a_i, u sin a_i + v cos a_i)
 *   with (u, v) = (n[rot_offset+i], n[rot_offset+rot/2+i]), or, interleaved,
 *   (n[rot_offset+2i], n[rot_offset+2i+1]).  The other values stay n.
 * The angles come from `freqs`, rot/2 turns per position as 64-bit fixed-point
 * fractions (csa_rope_freqs): positions[t] * freqs[i] modulo 2^64 is the exact
 * fraction of a turn, at any position of either sign.
 *   T tokens (>= 0; 0 enqueues nothing), Hq >= 1 query heads, Hk >= 0 key
 *   heads (0: no keys; k, k_weight and their outputs are NULL), D head size,
 *   dtype of q, k, their outputs and gradients, w_dtype of the weights
 *   (each a csa_dtype or CSA_F16).
 *   Strides in elements between tokens and heads of q and k (views into a
 *   projection's output need no copy; 0 = contiguous [T,H,D]); the innermost
 *   dimension is contiguous.  Bases are 16-byte aligned and strides multiples
 *   of 16 bytes.  Outputs, cotangents and gradients are contiguous.
 * Supported: D a multiple of 8 in 8..256; rot_offset a multiple of 8; rot a
 * positive multiple of 8 (interleaved) or 16, rot_offset + rot <= D.       */
typedef struct {
  int32_t T, Hq, Hk, D;
  int32_t rot, rot_offset, interleaved;
  int32_t dtype, w_dtype;
  float eps; /* >= 0, finite */
  int64_t q_stride_t, q_stride_h;
  int64_t k_stride_t, k_stride_h;
} csa_norm_rope_problem;

/* Fills freqs[rot/2] (host memory) with theta^(-2i/rot) / (2 pi) turns as
 * 64-bit fractions, each rounded to the nearest: an angle is off by 1.8e-19
 * radians per position for it.  theta > 1 (up to 1e18), rot a positive even
 * number.                                                                    */
csa_status csa_rope_freqs(double theta, int32_t rot, uint64_t* freqs);

/* q [T,Hq,D], k [T,Hk,D], q_weight [D], k_weight [D], positions [T] int64,
 * freqs [rot/2] (device copy) -> q_out [T,Hq,D], k_out [T,Hk,D].  Sums and
 * products in fp32, rounded once to dtype.                                   */
csa_status csa_norm_rope(const csa_norm_rope_problem* p, const void* q, const void* k, const void* q_weight,
                         const void* k_weight, const int64_t* positions, const uint64_t* freqs, void* q_out,
                         void* k_out, void* stream);

/* Gradients for the cotangents dq_out [T,Hq,D], dk_out [T,Hk,D] (dtype):
 * dq, dk (dtype, every element) and dq_weight [D], dk_weight [D] (fp32).
 * The norm is recomputed from q and k.  The weights' sums over tokens and
 * heads are taken in a fixed order (the same bits on every call).
 * Needs `workspace`: csa_norm_rope_workspace_size(p) bytes, 16-byte aligned. */
csa_status csa_norm_rope_backward(const csa_norm_rope_problem* p, const void* dq_out, const void* dk_out,
                                  const void* q, const void* k, const void* q_weight, const void* k_weight,
                                  const int64_t* positions, const uint64_t* freqs, void* dq, void* dk,
                                  float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes,
                                  void* stream);
size_t csa_norm_rope_workspace_size(const csa_norm_rope_problem* p);

/* ---------------------------------------------------------------- attention
 * N sequences packed one behind the other: sequence i has the query rows
 * cu_q[i] .. cu_q[i+1]-1 of q [Tq,Hq,D] and the keys cu_k[i] .. cu_k[i+1]-1 of
 * k, v [Tk,Hk,D]; with k_len given only the first k_len[i] of those (a cache
 * [N,W,Hk,D] is Tk = N*W with cu_k[i] = i*W and k_len the sequences' lengths).
 * Query head h reads key head h / (Hq/Hk).  With lq query rows and lk keys,
 * row r of a sequence sees its keys j <= r + lk - lq (causal: the last query
 * stands at the last key) or all of them (causal = 0):
 *   s_j = scale * q.k_j,  out = sum_j softmax(s)_j v_j,  lse = log sum_j exp(s_j).
 * A row that sees no key, and a row outside every sequence, gives out = 0 and
 * lse = -inf.  Lengths of zero are allowed on either side.
 * What a sequence does not hold is never part of its results: rows of other
 * sequences and cache entries past k_len may hold anything, also NaN.  Keys of
 * the sequence itself that are hidden from a row (later ones) do not reach its
 * out and lse either, whatever they hold.  The gradients of a sequence that
 * holds infinite or NaN values are not specified; those of the others are
 * unaffected.
 *   cu_q, cu_k [N+1] int32 ascending in 0..Tq, 0..Tk; k_len [N] int32 or NULL.
 *   They are device memory; entries out of order or range are clamped, never
 *   followed, and record CSA_ERR_DEVICE in the device status word.
 *   Strides in elements between tokens and heads of q, k and v (0 =
 *   contiguous); the innermost dimension is contiguous.  Bases are 16-byte
 *   aligned and strides multiples of 8 elements.  out, lse, the cotangent and
 *   the gradients are contiguous, with 16-byte aligned bases.
 * Precision: products of stored values are exact and summed in fp32, as are the
 * softmax's sums; exponentials are fp32.  The weights p that meet v (and dout, for
 * dv), and ds = p (dout.v - dout.out) that meets k and q, are rounded to dtype,
 * the tensor cores' operand type: half a unit of the last place each, twice what an
 * fp32 computation rounded once has at worst.  dout.out is taken from the rounded
 * out, except for rows whose block sees 128 keys or fewer.  In fp16, p and ds are
 * formed at powers of two that keep them in range: p counts down to 2^-33 of the
 * largest in out and 2^-40 in dv, and cotangents of any size give finite gradients
 * where these fit fp16.
 * Supported: D in {64, 128}, dtype CSA_BF16 or CSA_F16, Hq a multiple of Hk,
 * Hq / Hk <= 128.  Tq, Tk, N >= 0 (nothing to write enqueues nothing).      */
typedef struct {
  int32_t N, Tq, Tk, Hq, Hk, D;
  int32_t dtype, causal;
  float scale; /* > 0, finite */
  int64_t q_stride_t, q_stride_h;
  int64_t k_stride_t, k_stride_h;
  int64_t v_stride_t, v_stride_h;
} csa_attn_problem;

/* Writes out [Tq,Hq,D] (dtype) and lse [Tq,Hq] fp32, every element.  Needs
 * `workspace`: csa_attn_workspace_size(p, 0) bytes (may be 0), 16-byte aligned. */
csa_status csa_attn_forward(const csa_attn_problem* p, const void* q, const void* k, const void* v,
                            const int32_t* cu_q, const int32_t* cu_k, const int32_t* k_len, void* out, float* lse,
                            void* workspace, size_t workspace_bytes, void* stream);

/* Gradients for the cotangent dout [Tq,Hq,D] of out, from the forward's out
 * and lse: dq [Tq,Hq,D], dk, dv [Tk,Hk,D] (dtype, every element; zero where
 * nothing reaches them).  The sums are taken in a fixed order (the same bits
 * on every call).  Needs `workspace`: csa_attn_workspace_size(p, 1) bytes.    */
csa_status csa_attn_backward(const csa_attn_problem* p, const void* dout, const void* q, const void* k,
                             const void* v, const void* out, const float* lse, const int32_t* cu_q,
                             const int32_t* cu_k, const int32_t* k_len, void* dq, void* dk, void* dv,
                             void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of device workspace: which = 0 for csa_attn_forward, 1 for
 * csa_attn_backward.  Depends only on the problem; 0 when it is invalid.      */
size_t csa_attn_workspace_size(const csa_attn_problem* p, int32_t which);

/* Version of this header's part of the library (major * 100 + minor). */
int32_t csa_attn_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* CSA_ATTN_H */
