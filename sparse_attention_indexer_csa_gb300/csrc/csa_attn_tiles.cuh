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
  int seq;  // its sequence (-1: none)
};

// The runs are what the multiples of `step` (nb of them below Tq) and the
// sequences' starts cu_q[0..N] cut 0..Tq into: run x of nb + N + 1 lies
// between the x-th and the next of those borders in ascending order (two
// borders that fall together leave an empty run).  The x-th is found by a
// search for how many multiples are among the first x+1 borders, 32 probes at
// a time by a warp, whose lanes all get the result (or by one thread).
// Entries out of order give some other runs inside 0..Tq.
template <bool KEYS, bool WARP = true>
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
  if (lo > hi) return RowItem{0, 0, SeqExt{0, 0, 0, 0}, -1};
  while (!WARP && lo < hi) {  // one thread: by halves
    const int i = (lo + hi + 1) >> 1;
    if (static_cast<long long>(i - 1) * step <= start(k - i))
      lo = i;
    else
      hi = i - 1;
  }
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
  r.seq = seqs && j > 0 && j <= a.N ? j - 1 : -1;
  if (r.seq >= 0) r.s = seq_extent(a, r.seq);
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

// TMA store of a 4-D box from shared memory, tracked by the bulk async-group of
// the issuing thread.
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* m, const void* src, int c0, int c1, int c2, int c3) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(m),
               "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}

// ----------------------------------------------------------------- next item
// Cluster launch control: asks for one block of the grid that has not started;
// the 16-byte answer at `slot` completes on `bar`.  One thread.
__device__ __forceinline__ void request_next(uint8_t* slot, uint64_t* bar) {
  mbar_arrive_expect_tx(bar, 16u);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
          smem_u32(slot)),
      "r"(smem_u32(bar))
      : "memory");
}
// The answer: false when none was left (no further request may follow), else
// `id` is the index of the block, which will not be launched.
__device__ __forceinline__ bool answer_next(const uint8_t* slot, uint32_t& id) {
  uint32_t ok, x = 0;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
      "ld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
      : "=r"(ok), "=r"(x)
      : "r"(smem_u32(slot))
      : "memory");
  id = x;
  fence_proxy_async_shared();  // the next answer is written by the async proxy
  return ok != 0u;
}

// ----------------------------------------------------------------- waits on the critical path
// As mbar_wait, by a whole warp whose control flow stays uniform (what follows
// keeps its operands in uniform registers), and polling without suspending the
// threads: suspended ones take longer to come back than the tensor pipe has
// work queued.  The limit is looked at every 1024 polls.
__device__ __forceinline__ bool mbar_look_warp(uint64_t* bar, uint32_t parity) {
  return __any_sync(0xffffffffu, mbar_test_wait(bar, parity)) != 0;
}
__device__ __forceinline__ bool mbar_spin_warp(uint64_t* bar, uint32_t parity, const WaitCtl& ctl) {
  uint64_t t0 = 0;
  for (uint32_t n = 0;; ++n) {
    if (mbar_look_warp(bar, parity)) return true;
    if ((n & 1023u) == 1023u) {
      const uint64_t t = globaltimer_ns();
      if (t0 == 0) t0 = t;
      const bool late = t - t0 > ctl.limit_ns;
      if (__any_sync(0xffffffffu, late || *ctl.abort_flag != 0u)) {
        *ctl.abort_flag = 1u;
        if (late) record_error(kErrTimeout);
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool elect_one() {
  uint32_t x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(x));
  return x != 0u;
}
// Lane 0's value, as one the compiler knows to be the same in all lanes.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// A meeting of warps at `bar` (initialised to their number), bounded as every
// wait is: named barriers would wait for a warp that gave up.  What the warps
// wrote to shared memory before is visible after; phase is kept by each warp.
__device__ __forceinline__ void meet(uint64_t* bar, uint32_t& phase, const WaitCtl& ctl) {
  __syncwarp();
  if (lane_id() == 0) mbar_arrive(bar);
  mbar_wait(bar, phase, ctl);
  phase ^= 1u;
}

// ----------------------------------------------------------------- register splits
// TILES = 2: 384 threads start with 168 registers each (64512): 256 of them grow
// to 216, 128 shrink to 72 (55296 + 9216 = 64512).  TILES = 1, two CTAs per SM:
// 256 threads start with 128 (32768): 128 grow to 184, 128 shrink to 72 (32768).
template <int TILES>
__device__ __forceinline__ void reg_grow() {
  if constexpr (TILES == 2)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
  else
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
}
__device__ __forceinline__ void reg_shrink() { asm volatile("setmaxnreg.dec.sync.aligned.u32 72;"); }

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

// The n lowest bits (n of any size, below 1: none; above 31: all).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
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

// Lanes 4 i + r (r = 0..3) hold four pieces each; afterwards lane 4 i + r holds
// piece r of the lanes 4 i .. 4 i + 3, in their order.
__device__ __forceinline__ void transpose4(uint4 (&q)[4], uint32_t lane) {
  auto swap = [&](uint4& x, uint4& y, uint32_t mask) {  // upper lane gives x, lower lane gives y
    const bool up = (lane & mask) != 0u;
    uint4 s = up ? x : y;
    s.x = __shfl_xor_sync(0xffffffffu, s.x, mask);
    s.y = __shfl_xor_sync(0xffffffffu, s.y, mask);
    s.z = __shfl_xor_sync(0xffffffffu, s.z, mask);
    s.w = __shfl_xor_sync(0xffffffffu, s.w, mask);
    if (up)
      x = s;
    else
      y = s;
  };
  swap(q[0], q[1], 1u);
  swap(q[2], q[3], 1u);
  swap(q[0], q[2], 2u);
  swap(q[1], q[3], 2u);
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
