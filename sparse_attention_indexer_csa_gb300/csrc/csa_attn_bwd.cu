// csa_attn_bwd.cu -- gradients of causal attention over packed sequences, one
// warp per query row and head (dq) or per key and key head (dk, dv).
//
//   delta = dout.out;  p_j = exp(s_j - lse);  ds_j = p_j (dout.v_j - delta)
//   dq = scale sum_j ds_j k_j;  dk_j = scale sum_rows ds_j q;  dv_j = sum_rows p_j dout
//
// A warp takes 32 keys (rows) at a time: lane j forms the dot products of
// key (row) j, then every lane adds the 32 weighted rows into its own D/32
// values.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "csa_attn_internal.h"
#include "csa_attn_tiles.cuh"

namespace csa {
namespace {

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <typename X>
__device__ __forceinline__ X from_f(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
  return __float2bfloat16(x);
}
template <>
__device__ __forceinline__ __half from_f<__half>(float x) {
  return __float2half(x);
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

constexpr int kWarps = 4;

template <typename X, int D>
__device__ __forceinline__ float dot(const X* a, const float* b) {
  float s = 0.f;
#pragma unroll 16
  for (int d = 0; d < D; ++d) s = fmaf(to_f(a[d]), b[d], s);
  return s;
}

template <typename X, int D>
__global__ void __launch_bounds__(kWarps * 32) attn_delta_kernel(const AttnParams p) {
  const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
  const long long item = static_cast<long long>(blockIdx.x) * kWarps + w;
  if (item >= static_cast<long long>(p.Tq) * p.Hq) return;
  float s = 0.f;
  for (int d = lane; d < D; d += 32)
    s = fmaf(to_f(static_cast<const X*>(p.dout)[item * D + d]), to_f(static_cast<const X*>(p.out)[item * D + d]), s);
  s = warp_sum(s);
  if (lane == 0) p.delta[item] = s;
}

template <typename X, int D>
__global__ void __launch_bounds__(kWarps * 32) attn_dq_kernel(const AttnParams p) {
  __shared__ float qs[kWarps][D], ds_[kWarps][D];
  if (blockIdx.x == 0) check_sequences(p);
  const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
  const long long item = static_cast<long long>(blockIdx.x) * kWarps + w;
  if (item >= static_cast<long long>(p.Tq) * p.Hq) return;
  const int t = static_cast<int>(item / p.Hq), h = static_cast<int>(item % p.Hq), hk = h / p.g;
  const X* q = static_cast<const X*>(p.q) + t * p.q_st + h * p.q_sh;
  for (int d = lane; d < D; d += 32) {
    qs[w][d] = to_f(q[d]);
    ds_[w][d] = to_f(static_cast<const X*>(p.dout)[item * D + d]);
  }
  __syncwarp();
  float acc[D / 32] = {};
  const int i = find_seq(p.cu_q, p.N, t);
  if (i >= 0) {
    const SeqExt e = seq_extent(p, i);
    const int see = keys_seen(p, e, t - e.q0);
    const float lse = p.lse[item], delta = p.delta[item];
    const X* k = static_cast<const X*>(p.k) + e.k0 * p.k_st + hk * p.k_sh;
    const X* v = static_cast<const X*>(p.v) + e.k0 * p.v_st + hk * p.v_sh;
    for (int j0 = 0; j0 < see; j0 += 32) {
      const int j = j0 + lane;
      float ds = 0.f;
      if (j < see)
        ds = expf(dot<X, D>(k + j * p.k_st, qs[w]) * p.scale - lse) * (dot<X, D>(v + j * p.v_st, ds_[w]) - delta);
      for (int u = 0; u < min(32, see - j0); ++u) {
        const float du = __shfl_sync(0xffffffffu, ds, u);
        for (int d = 0; d < D / 32; ++d) acc[d] = fmaf(du, to_f(k[(j0 + u) * p.k_st + d * 32 + lane]), acc[d]);
      }
    }
  }
  X* dq = static_cast<X*>(p.dq) + item * D;
  for (int d = 0; d < D / 32; ++d) dq[d * 32 + lane] = from_f<X>(acc[d] * p.scale);
}

template <typename X, int D>
__global__ void __launch_bounds__(kWarps * 32) attn_dkv_kernel(const AttnParams p) {
  __shared__ float ks[kWarps][D], vs[kWarps][D];
  if (blockIdx.x == 0) check_sequences(p);
  const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
  const long long item = static_cast<long long>(blockIdx.x) * kWarps + w;
  if (item >= static_cast<long long>(p.Tk) * p.Hk) return;
  const int t = static_cast<int>(item / p.Hk), hk = static_cast<int>(item % p.Hk);
  for (int d = lane; d < D; d += 32) {
    ks[w][d] = to_f((static_cast<const X*>(p.k) + t * p.k_st + hk * p.k_sh)[d]);
    vs[w][d] = to_f((static_cast<const X*>(p.v) + t * p.v_st + hk * p.v_sh)[d]);
  }
  __syncwarp();
  float ak[D / 32] = {}, av[D / 32] = {};
  const int i = find_seq(p.cu_k, p.N, t);
  if (i >= 0) {
    const SeqExt e = seq_extent(p, i);
    const int j = t - e.k0, lq = e.q1 - e.q0;
    const int r_lo = j >= e.lk ? lq : (p.causal ? max(0, j - (e.lk - lq)) : 0);
    const long long n = static_cast<long long>(max(0, lq - r_lo)) * p.g;
    for (long long u0 = 0; u0 < n; u0 += 32) {
      const long long u = u0 + lane;
      float pj = 0.f, ds = 0.f;
      const auto row = [&](long long x) { return e.q0 + r_lo + x / p.g; };
      const auto head = [&](long long x) { return hk * p.g + x % p.g; };
      if (u < n) {
        const long long qi = row(u) * p.Hq + head(u);
        pj = expf(dot<X, D>(static_cast<const X*>(p.q) + row(u) * p.q_st + head(u) * p.q_sh, ks[w]) * p.scale -
                  p.lse[qi]);
        ds = pj * (dot<X, D>(static_cast<const X*>(p.dout) + qi * D, vs[w]) - p.delta[qi]);
      }
      for (int x = 0; x < static_cast<int>(min(32ll, n - u0)); ++x) {
        const float px = __shfl_sync(0xffffffffu, pj, x), dx = __shfl_sync(0xffffffffu, ds, x);
        const X* q = static_cast<const X*>(p.q) + row(u0 + x) * p.q_st + head(u0 + x) * p.q_sh;
        const X* o = static_cast<const X*>(p.dout) + (row(u0 + x) * p.Hq + head(u0 + x)) * D;
        for (int d = 0; d < D / 32; ++d) {
          ak[d] = fmaf(dx, to_f(q[d * 32 + lane]), ak[d]);
          av[d] = fmaf(px, to_f(o[d * 32 + lane]), av[d]);
        }
      }
    }
  }
  for (int d = 0; d < D / 32; ++d) {
    (static_cast<X*>(p.dk) + item * D)[d * 32 + lane] = from_f<X>(ak[d] * p.scale);
    (static_cast<X*>(p.dv) + item * D)[d * 32 + lane] = from_f<X>(av[d]);
  }
}

unsigned blocks_of(long long items) { return static_cast<unsigned>((items + kWarps - 1) / kWarps); }

template <typename X, int D>
cudaError_t bwd(const AttnParams& p, cudaStream_t s) {
  if (p.Tq > 0) {
    const unsigned n = blocks_of(static_cast<long long>(p.Tq) * p.Hq);
    attn_delta_kernel<X, D><<<n, kWarps * 32, 0, s>>>(p);
    attn_dq_kernel<X, D><<<n, kWarps * 32, 0, s>>>(p);
  }
  if (p.Tk > 0) attn_dkv_kernel<X, D><<<blocks_of(static_cast<long long>(p.Tk) * p.Hk), kWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_backward(const AttnParams& p, int dtype, cudaStream_t s) {
  if (dtype == CSA_BF16) return p.D == 128 ? bwd<__nv_bfloat16, 128>(p, s) : bwd<__nv_bfloat16, 64>(p, s);
  return p.D == 128 ? bwd<__half, 128>(p, s) : bwd<__half, 64>(p, s);
}

cudaError_t take_status_attn_bwd(uint32_t* out, cudaStream_t stream) { return take_status(out, stream); }

}  // namespace csa
