// csa_norm_rope.cu -- norm of every query and key head and the position
// rotation in one pass, and its gradients.
//
//   n = x r w, r = rsqrt(mean(x^2) + eps);  y = R n, R turning each pair by
//   its angle.  With z = R^T dy (the opposite turn), xh = x r:
//   dw = sum over rows of z xh,  dx = r (z w - xh mean(z w xh)).
//
// Memory-bound: the forward reads and writes each value once, the backward
// reads x and dy and writes dx (nothing but x is kept from the forward: the
// norm of a head is a sum over values that are read anyway).  A row (one
// token, one head) is held by G lanes, eight values each, so every access is
// 16 bytes wide (two for fp32) and the mean is a shuffle within G lanes.  The
// partner of a value is in the same lane (interleaved pairs) or rot/16 lanes
// away (halves).  Rows are walked head-fastest, so a block's rows belong to a
// few tokens whose cosines and sines it computes once, into shared memory,
// while its first loads are in flight.
//
// Angles: position * freq modulo 2^64 is the fraction of a turn with 64 bits
// after the point, whatever the position; its upper 32 bits, as a signed
// number of half turns, go to sincospif (absolute error of the angle below
// 2e-7, against about 0.06 for a 32-bit product at position 1e6).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "csa_attn_internal.h"

namespace csa {
namespace {

constexpr int kThreads = 256;

// Eight consecutive values as fp32.
struct V8 {
  float v[8];
};
template <typename X>
struct Raw8 {
  uint4 a;
};
template <>
struct Raw8<float> {
  uint4 a, b;
};
template <typename X>
__device__ __forceinline__ Raw8<X> load8(const X* p) {
  Raw8<X> r;
  r.a = __ldcs(reinterpret_cast<const uint4*>(p));
  if constexpr (sizeof(X) == 4) r.b = __ldcs(reinterpret_cast<const uint4*>(p) + 1);
  return r;
}
__device__ __forceinline__ float2 unpack2(uint32_t u, __nv_bfloat16) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t u, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
template <typename X>
__device__ __forceinline__ V8 widen(const Raw8<X>& r) {
  V8 o;
  if constexpr (sizeof(X) == 4) {
    const uint32_t u[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] = __uint_as_float(u[i]);
  } else {
    const uint32_t u[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2(u[i], X{});
      o.v[2 * i] = f.x;
      o.v[2 * i + 1] = f.y;
    }
  }
  return o;
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename X>
__device__ __forceinline__ void store8(X* p, const V8& o) {
  if constexpr (sizeof(X) == 4) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(o.v[0], o.v[1], o.v[2], o.v[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(o.v[4], o.v[5], o.v[6], o.v[7]));
  } else {
    uint4 u;
    u.x = pack2(o.v[0], o.v[1], X{});
    u.y = pack2(o.v[2], o.v[3], X{});
    u.z = pack2(o.v[4], o.v[5], X{});
    u.w = pack2(o.v[6], o.v[7], X{});
    __stcs(reinterpret_cast<uint4*>(p), u);
  }
}
// Eight weights of the run-time type w_dtype (read once per block).
__device__ __forceinline__ V8 load_weight(const void* w, int w_dtype, int e, int D) {
  V8 o;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    o.v[i] = 0.f;
    if (e + i < D)
      o.v[i] = w_dtype == CSA_F32   ? static_cast<const float*>(w)[e + i]
               : w_dtype == CSA_F16 ? __half2float(static_cast<const __half*>(w)[e + i])
                                    : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[e + i]);
  }
  return o;
}

template <int G>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Cosines and sines of the tokens t0 .. t0+n-1 into cs[n][rot/2].
__device__ __forceinline__ void fill_angles(const NormRopeParams& p, int t0, int n, float2* cs) {
  const int half = p.rot / 2;
  for (int i = threadIdx.x; i < n * half; i += kThreads) {
    const int t = i / half, j = i - t * half;
    const uint64_t turns = static_cast<uint64_t>(p.pos[t0 + t]) * p.freqs[j];
    const float x = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 4.656612873077393e-10f;  // 2^-31
    float s, c;
    sincospif(x, &s, &c);
    cs[i] = make_float2(c, s);
  }
}

// Where this lane's eight values stand in the turned range.
struct Turn {
  bool in;     // the values are turned
  int pair0;   // index of the first pair
  float sign;  // halves: -1 in the first half, +1 in the second
  int src;     // halves: lane of the partner
};
template <int G, bool INTER>
__device__ __forceinline__ Turn make_turn(const NormRopeParams& p, int e) {
  Turn t;
  const int r = e - p.off;
  t.in = r >= 0 && r < p.rot;
  t.pair0 = 0;
  t.sign = 0.f;
  t.src = static_cast<int>(lane_id());
  if (!t.in) return t;
  if constexpr (INTER) {
    t.pair0 = r / 2;
  } else {
    const int half = p.rot / 2;
    const bool first = r < half;
    t.pair0 = first ? r : r - half;
    t.sign = first ? -1.f : 1.f;
    t.src += (first ? 1 : -1) * (half / 8);
  }
  return t;
}
// Turns v by the angles cs (dir = +1) or back (dir = -1).
template <bool INTER>
__device__ __forceinline__ void turn(V8& v, const Turn& t, const float2* cs, float dir) {
  if constexpr (INTER) {
    if (!t.in) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = cs[t.pair0 + i];
      const float s = a.y * dir, x = v.v[2 * i], y = v.v[2 * i + 1];
      v.v[2 * i] = x * a.x - y * s;
      v.v[2 * i + 1] = x * s + y * a.x;
    }
  } else {
    float other[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) other[i] = __shfl_sync(0xffffffffu, v.v[i], t.src);
    if (!t.in) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 a = cs[t.pair0 + i];
      v.v[i] = v.v[i] * a.x + other[i] * (a.y * (t.sign * dir));
    }
  }
}

// Row r of the walk: token, head, whether a query.
struct RowAt {
  int t, h;
};

template <typename X, int G, bool INTER, int U>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRopeParams p) {
  extern __shared__ float2 cs[];
  constexpr int PER = kThreads / G;  // rows per pass
  const int H = p.Hq + p.Hk, l = threadIdx.x % G, e = 8 * l;
  const bool lane_ok = e < p.D;
  const long long row0 = static_cast<long long>(blockIdx.x) * (PER * U);
  const int t0 = static_cast<int>(row0 / H);
  const long long last = min(p.rows, row0 + PER * U) - 1;
  const int ntok = static_cast<int>(last / H) - t0 + 1;
  RowAt at[U];
  Raw8<X> raw[U];
  {
    long long r = row0 + threadIdx.x / G;
    int t = static_cast<int>(r / H), h = static_cast<int>(r - static_cast<long long>(t) * H);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      at[u] = RowAt{t, h};
      raw[u] = Raw8<X>{};
      if (t < p.T && lane_ok) {
        const X* x = h < p.Hq ? static_cast<const X*>(p.q) + t * p.q_st + h * p.q_sh
                              : static_cast<const X*>(p.k) + t * p.k_st + (h - p.Hq) * p.k_sh;
        raw[u] = load8(x + e);
      }
      h += PER;
      while (h >= H) {
        h -= H;
        ++t;
      }
    }
  }
  const V8 wq = load_weight(p.qw, p.w_dtype, e, p.D);
  V8 wk = wq;
  if (p.Hk > 0) wk = load_weight(p.kw, p.w_dtype, e, p.D);
  fill_angles(p, t0, ntok, cs);
  const Turn tn = make_turn<G, INTER>(p, e);
  __syncthreads();
#pragma unroll
  for (int u = 0; u < U; ++u) {
    V8 x = widen(raw[u]);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x.v[i], x.v[i], ss);
    const float r = rsqrtf(group_sum<G>(ss) * p.inv_d + p.eps);
    const bool isq = at[u].h < p.Hq;
#pragma unroll
    for (int i = 0; i < 8; ++i) x.v[i] = x.v[i] * r * (isq ? wq.v[i] : wk.v[i]);
    const bool ok = at[u].t < p.T;
    turn<INTER>(x, tn, cs + (ok ? at[u].t - t0 : 0) * (p.rot / 2), 1.f);
    if (ok && lane_ok) {
      X* y = isq ? static_cast<X*>(p.yq) + (static_cast<long long>(at[u].t) * p.Hq + at[u].h) * p.D
                 : static_cast<X*>(p.yk) + (static_cast<long long>(at[u].t) * p.Hk + (at[u].h - p.Hq)) * p.D;
      store8(y + e, x);
    }
  }
}

// The backward walks its share of the rows with the weight gradients of its
// eight values (query and key weights) in registers; a block joins its
// groups' sums in shared memory and writes one partial row, and a second
// kernel adds the partial rows in order.
template <typename X, int G, bool INTER, int U>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(const NormRopeParams p) {
  extern __shared__ float2 cs[];
  constexpr int PER = kThreads / G;
  const int H = p.Hq + p.Hk, l = threadIdx.x % G, e = 8 * l;
  const bool lane_ok = e < p.D;
  const V8 wq = load_weight(p.qw, p.w_dtype, e, p.D);
  V8 wk = wq;
  if (p.Hk > 0) wk = load_weight(p.kw, p.w_dtype, e, p.D);
  const Turn tn = make_turn<G, INTER>(p, e);
  float aq[8] = {}, ak[8] = {};
  for (long long row0 = static_cast<long long>(blockIdx.x) * (PER * U); row0 < p.rows;
       row0 += static_cast<long long>(gridDim.x) * (PER * U)) {
    const int t0 = static_cast<int>(row0 / H);
    const long long last = min(p.rows, row0 + PER * U) - 1;
    const int ntok = static_cast<int>(last / H) - t0 + 1;
    RowAt at[U];
    Raw8<X> rx[U], rg[U];
    long long r = row0 + threadIdx.x / G;
    int t = static_cast<int>(r / H), h = static_cast<int>(r - static_cast<long long>(t) * H);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      at[u] = RowAt{t, h};
      rx[u] = Raw8<X>{};
      rg[u] = Raw8<X>{};
      if (t < p.T && lane_ok) {
        const bool isq = h < p.Hq;
        rx[u] = load8((isq ? static_cast<const X*>(p.q) + t * p.q_st + h * p.q_sh
                           : static_cast<const X*>(p.k) + t * p.k_st + (h - p.Hq) * p.k_sh) +
                      e);
        rg[u] = load8((isq ? static_cast<const X*>(p.gq) + (static_cast<long long>(t) * p.Hq + h) * p.D
                           : static_cast<const X*>(p.gk) + (static_cast<long long>(t) * p.Hk + (h - p.Hq)) * p.D) +
                      e);
      }
      h += PER;
      while (h >= H) {
        h -= H;
        ++t;
      }
    }
    __syncthreads();  // the former rows' angles are no longer read
    fill_angles(p, t0, ntok, cs);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      V8 x = widen(rx[u]);
      V8 z = widen(rg[u]);
      const bool ok = at[u].t < p.T, isq = at[u].h < p.Hq;
      turn<INTER>(z, tn, cs + (ok ? at[u].t - t0 : 0) * (p.rot / 2), -1.f);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x.v[i], x.v[i], ss);
      const float rr = rsqrtf(group_sum<G>(ss) * p.inv_d + p.eps);
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x.v[i] *= rr;  // xh
        const float zx = z.v[i] * x.v[i];
        if (ok) {
          if (isq)
            aq[i] += zx;
          else
            ak[i] += zx;
        }
        z.v[i] *= isq ? wq.v[i] : wk.v[i];
        dot = fmaf(z.v[i], x.v[i], dot);
      }
      dot = group_sum<G>(dot) * p.inv_d;
#pragma unroll
      for (int i = 0; i < 8; ++i) z.v[i] = rr * (z.v[i] - x.v[i] * dot);
      if (ok && lane_ok) {
        X* y = isq ? static_cast<X*>(p.yq) + (static_cast<long long>(at[u].t) * p.Hq + at[u].h) * p.D
                   : static_cast<X*>(p.yk) + (static_cast<long long>(at[u].t) * p.Hk + (at[u].h - p.Hq)) * p.D;
        store8(y + e, z);
      }
    }
  }
  __shared__ float red[kThreads * 8];  // [PER][8 G]
  for (int part = 0; part < 2; ++part) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) red[(threadIdx.x / G) * (8 * G) + e + i] = part ? ak[i] : aq[i];
    __syncthreads();
    for (int d = threadIdx.x; d < p.D; d += kThreads) {
      float s = 0.f;
      for (int r = 0; r < PER; ++r) s += red[r * (8 * G) + d];
      p.part[(static_cast<size_t>(blockIdx.x) * 2 + part) * p.D + d] = s;
    }
  }
}

// dqw, dkw = sums of the partial rows: 32 columns x 8 runs of rows per block.
__global__ void __launch_bounds__(256) norm_rope_dw_kernel(const float* part, int n, int D, float* dqw, float* dkw) {
  __shared__ float red[8][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), run = threadIdx.x >> 5;
  float s = 0.f;
  if (c < 2 * D)
    for (int i = run; i < n; i += 8) s += part[static_cast<size_t>(i) * 2 * D + c];
  red[run][threadIdx.x & 31] = s;
  __syncthreads();
  if (run == 0 && c < 2 * D) {
    for (int i = 1; i < 8; ++i) s += red[i][threadIdx.x & 31];
    if (c < D)
      dqw[c] = s;
    else if (dkw != nullptr)
      dkw[c - D] = s;
  }
}

// Shared memory of the angles of `rows` consecutive rows.
size_t angle_bytes(const NormRopeParams& p, int rows) {
  const int H = p.Hq + p.Hk;
  const long long tok = std::min<long long>(p.T, (rows - 1) / H + 2);
  return static_cast<size_t>(tok) * (p.rot / 2) * sizeof(float2);
}

template <typename X, int G, bool INTER>
cudaError_t run_forward(const NormRopeParams& p, cudaStream_t stream) {
  constexpr int PER = kThreads / G, U = 4;
  const long long blocks = (p.rows + PER * U - 1) / (PER * U);
  if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  norm_rope_kernel<X, G, INTER, U>
      <<<static_cast<unsigned>(blocks), kThreads, angle_bytes(p, PER * U), stream>>>(p);
  return cudaGetLastError();
}

template <typename X, int G, bool INTER>
cudaError_t run_backward(const NormRopeParams& p, cudaStream_t stream) {
  constexpr int PER = kThreads / G, U = 2;
  const long long chunks = (p.rows + PER * U - 1) / (PER * U);
  const int blocks = static_cast<int>(std::min<long long>(chunks, kNormRopeBlocks));
  norm_rope_bwd_kernel<X, G, INTER, U><<<blocks, kThreads, angle_bytes(p, PER * U), stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  norm_rope_dw_kernel<<<(2 * p.D + 31) / 32, 256, 0, stream>>>(p.part, blocks, p.D, p.dqw, p.dkw);
  return cudaGetLastError();
}

template <typename X, bool INTER>
cudaError_t by_size(const NormRopeParams& p, bool bwd, cudaStream_t s) {
  if (p.D <= 32) return bwd ? run_backward<X, 4, INTER>(p, s) : run_forward<X, 4, INTER>(p, s);
  if (p.D <= 64) return bwd ? run_backward<X, 8, INTER>(p, s) : run_forward<X, 8, INTER>(p, s);
  if (p.D <= 128) return bwd ? run_backward<X, 16, INTER>(p, s) : run_forward<X, 16, INTER>(p, s);
  return bwd ? run_backward<X, 32, INTER>(p, s) : run_forward<X, 32, INTER>(p, s);
}
template <typename X>
cudaError_t by_pairs(const NormRopeParams& p, bool inter, bool bwd, cudaStream_t s) {
  return inter ? by_size<X, true>(p, bwd, s) : by_size<X, false>(p, bwd, s);
}
cudaError_t dispatch(const NormRopeParams& p, int dtype, bool inter, bool bwd, cudaStream_t s) {
  if (dtype == CSA_F32) return by_pairs<float>(p, inter, bwd, s);
  if (dtype == CSA_F16) return by_pairs<__half>(p, inter, bwd, s);
  return by_pairs<__nv_bfloat16>(p, inter, bwd, s);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, int dtype, bool inter, cudaStream_t stream) {
  return dispatch(p, dtype, inter, false, stream);
}
cudaError_t launch_norm_rope_backward(const NormRopeParams& p, int dtype, bool inter, cudaStream_t stream) {
  return dispatch(p, dtype, inter, true, stream);
}

}  // namespace csa
