// csa_attn_tiles.cuh -- what the attention kernels share: TMA maps of packed
// rows and keys, the walk over packed sequences, register splits, and small
// numeric helpers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "csa_attn_internal.h"

namespace csa {

constexpr uint32_t kChunkBytes = 128 * 128;  // 16 KB: 128 rows x 64 values of 2 bytes, 128-byte swizzled
constexpr unsigned long long kAttnWaitNs = 2000000000ull;

// ----------------------------------------------------------------- TMA maps (host)
inline PFN_cuTensorMapEncodeTiled_v12000 attn_encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag flag;
  std::call_once(flag, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// x [Tq,Hq,D] as dims (D, g, Tq, Hk): a box {64, g, tok, 1} lands as rows
// token * g + head of the heads that share a key head.
inline bool make_rows_map(CUtensorMap* m, const AttnParams& p, const void* x, long long st, long long sh, int tok) {
  auto fn = attn_encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[4] = {(cuuint64_t)p.D, (cuuint64_t)p.g, (cuuint64_t)p.Tq, (cuuint64_t)p.Hk};
  cuuint64_t strides[3] = {(cuuint64_t)sh * 2, (cuuint64_t)st * 2, (cuuint64_t)sh * p.g * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)p.g, (cuuint32_t)tok, 1}, estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(x), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// k or v [Tk,Hk,D] as dims (D, Tk, Hk), box {64, 128, 1}; keys past Tk read as
// zero.  Without any key the map describes one row of q that nothing loads.
inline bool make_keys_map(CUtensorMap* m, const AttnParams& p, const void* x, long long st, long long sh) {
  auto fn = attn_encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[3] = {(cuuint64_t)p.D, (cuuint64_t)(p.Tk > 0 ? p.Tk : 1), (cuuint64_t)p.Hk};
  cuuint64_t strides[2] = {(cuuint64_t)st * 2, (cuuint64_t)sh * 2};
  cuuint32_t box[3] = {64, 128, 1}, estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p.Tk > 0 ? x : p.q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ----------------------------------------------------------------- walk over packed sequences
// A run of consecutive query rows t0 .. t1-1 of one sequence (or of rows
// outside all sequences: lk = 0), at most `step` of them.
struct RowItem {
  int t0, t1;
  SeqExt s;
};

// The runs are what the multiples of `step` (nb of them below Tq) and the
// sequences' starts cu_q[0..N] cut 0..Tq into: run x of nb + N + 1 lies
// between the x-th and the next of those borders in ascending order (two
// borders that fall together leave an empty run).  The x-th is found by a
// search for how many multiples are among the first x+1 borders, 32 probes at
// a time.  A warp; every lane gets the result.  Entries out of order give some
// other runs inside 0..Tq.
template <bool KEYS>
__device__ __forceinline__ RowItem find_item(const AttnParams& a, int step, int nb, int x) {
  const int lane = static_cast<int>(lane_id());
  const int T = KEYS ? a.Tk : a.Tq;
  const int32_t* cu = KEYS ? a.cu_k : a.cu_q;
  auto start = [&](int i) { return min(max(cu[i], 0), T); };  // 0 <= i <= N
  const bool seqs = a.N > 0;
  const int nB = seqs ? a.N + 1 : 0;
  // the largest i whose i-th multiple is among the first k borders (a multiple
  // goes before a start of the same value)
  const int k = x + 1;
  int lo = max(0, k - nB), hi = min(k, nb);
  if (lo > hi) return RowItem{0, 0, SeqExt{0, 0, 0, 0}};
  while (lo < hi) {
    const int span = hi - lo, stride = (span + 31) / 32;
    const int i = lo + min(span, (lane + 1) * stride);  // lo < i <= hi, so 0 <= k - i < nB
    const bool in = static_cast<long long>(i - 1) * step <= start(k - i);
    const unsigned out = ~__ballot_sync(0xffffffffu, in);
    if (out == 0u) {  // also the last probe, hi
      lo = hi;
    } else {
      const int n = __ffs(static_cast<int>(out)) - 1;  // leading probes that hold
      hi = lo + min(span, (n + 1) * stride) - 1;
      lo = lo + min(span, n * stride);
    }
  }
  const int i = lo, j = k - lo;
  RowItem r;
  r.t0 = 0;
  if (i > 0) r.t0 = static_cast<int>(min(static_cast<long long>(T), static_cast<long long>(i - 1) * step));
  if (j > 0) r.t0 = max(r.t0, start(j - 1));
  r.t1 = i < nb ? static_cast<int>(min(static_cast<long long>(T), static_cast<long long>(i) * step)) : T;
  if (j < nB) r.t1 = min(r.t1, start(j));
  r.s = KEYS ? SeqExt{0, 0, r.t0, 0} : SeqExt{r.t0, r.t1, 0, 0};
  if (seqs && j > 0 && j <= a.N) r.s = seq_extent(a, j - 1);
  // entries out of order: a run never leaves its sequence
  r.t0 = max(r.t0, KEYS ? r.s.k0 : r.s.q0);
  if (!KEYS) r.t1 = min(r.t1, r.s.q1);
  if (r.t1 - r.t0 > step) r.t1 = r.t0 + step;
  return r;
}
__device__ __forceinline__ RowItem find_row_item(const AttnParams& a, int step, int nb, int x) {
  return find_item<false>(a, step, nb, x);
}
// The same over the keys: t0 .. t1-1 count from the tensor's first key.
__device__ __forceinline__ RowItem find_key_item(const AttnParams& a, int step, int nb, int x) {
  return find_item<true>(a, step, nb, x);
}

// ----------------------------------------------------------------- register splits
// 384 threads start with 168 registers each (64512): 256 of them grow to 200,
// 128 shrink to 104 (51200 + 13312 = 64512).
template <bool ON>
__device__ __forceinline__ void reg_grow() {
  if constexpr (ON) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
}
template <bool ON>
__device__ __forceinline__ void reg_shrink() {
  if constexpr (ON) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
}

// ----------------------------------------------------------------- small helpers
template <typename X>
__host__ __device__ constexpr bool is_bf16() {
  return false;
}
template <>
__host__ __device__ constexpr bool is_bf16<__nv_bfloat16>() {
  return true;
}
// Instruction descriptor of kind::f16 for the storage type X, fp32 results.
template <typename X>
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn) {
  const uint32_t t = is_bf16<X>() ? 1u : 0u;  // operand type: 0 f16, 1 bf16
  return (1u << 4) | (t << 7) | (t << 10) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  uint64_t A, B, D;
  asm("mov.b64 %0, {%1, %2};" : "=l"(A) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(B) : "f"(b.x), "f"(b.y));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(D) : "l"(A), "l"(B));
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(D));
  return r;
}
template <typename X>
__device__ __forceinline__ uint32_t pack_pair(float a, float b) {
  if constexpr (is_bf16<X>()) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}
template <typename X>
__device__ __forceinline__ float2 unpack_pair(uint32_t u) {
  if constexpr (is_bf16<X>())
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Largest of a row's 128 scores (NaN is passed over).
__device__ __forceinline__ float row_max(const float (&s)[4][32]) {
  float m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = fmaxf(s[i][0], s[i][1]);
#pragma unroll
    for (int u = 2; u < 32; u += 2) m[i] = max3(m[i], s[i][u], s[i][u + 1]);
  }
  return fmaxf(max3(m[0], m[1], m[2]), m[3]);
}

// Multiplies 16 TMEM columns of this thread's lane by r.
__device__ __forceinline__ void tmem_scale16(uint32_t t, float r) {
  float v[8];
  uint32_t u[16];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    tmem_ld8(t + 8 * h, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) u[8 * h + i] = __float_as_uint(v[i] * r);
  }
  tmem_st16(t, u);
}

// Clears the rows from `first` on of a 128-row tile (D/64 chunks), by
// `n` threads; the swizzle stays within a row's 128 bytes.
template <int D>
__device__ __forceinline__ void clear_tile_rows(uint8_t* tile, int first, int tid, int n) {
  for (int i = tid; i < 128 * (D / 64) * 8; i += n) {
    const int row = (i >> 3) & 127;
    if (row >= first)
      *reinterpret_cast<uint4*>(tile + (i >> 10) * kChunkBytes + row * 128 + (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
}

// Reads and clears the status word of the including translation unit.
inline cudaError_t take_status(uint32_t* out, cudaStream_t stream) {
  uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(out, g_status, sizeof(uint32_t), 0, cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e == cudaSuccess)
    e = cudaMemcpyToSymbolAsync(g_status, &zero, sizeof(uint32_t), 0, cudaMemcpyHostToDevice, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  return e;
}

}  // namespace csa
