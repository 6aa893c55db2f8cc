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
// 16 bytes wide (8 for 16-bit halves) and the mean is a shuffle within G lanes.
// Both values of a pair are in the same lane.  Rows are walked head-fastest,
// so a block's rows belong to a few tokens whose cosines and sines it computes
// once, into shared memory.
//
// Measured (bf16, 64 + 8 heads of 128): forward, 16384 tokens, all values
// rotated, 126 us (4.8 TB/s, a plain copy gives 6.7); 32768 tokens, half
// rotated in neighbouring pairs, 216 us (5.6 TB/s), gradients 376 us (4.8
// TB/s).  64 tokens: 5 us, a launch.
//
// Angles: position * freq modulo 2^64 is the fraction of a turn with 64 bits
// after the point, whatever the position; its upper 32 bits, as a signed
// number of half turns, go to sincospif (absolute error of the angle below
// 2e-7, against about 0.06 for a 32-bit product at position 1e6).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "csa_attn_internal.h"
#include "csa_attn_tiles.cuh"

namespace csa {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsFwd = 4, kRowsBwd = 3;  // rows of a thread in a chunk
// Blocks per SM (the registers a thread has): fp32 rows take twice the
// registers while they are on their way, and spill at three.
template <typename X, bool BWD>
constexpr int kBlocks = BWD || sizeof(X) == 4 ? 2 : 3;

// Eight consecutive values as fp32, in pairs (packed arithmetic).
struct V8 {
  float2 p[4];
};
template <typename X>
struct Raw8 {
  uint4 a;
};
template <>
struct Raw8<float> {
  uint4 a, b;
};
// Four values from p and four from p + gap (8 bytes each, 16 for fp32); one
// access of 16 bytes where the eight are known to be consecutive.
template <typename X, bool INTER>
__device__ __forceinline__ Raw8<X> load8(const X* p, int gap) {
  Raw8<X> r;
  if constexpr (sizeof(X) == 4) {
    r.a = __ldcs(reinterpret_cast<const uint4*>(p));
    r.b = __ldcs(reinterpret_cast<const uint4*>(p + gap));
  } else if constexpr (INTER) {
    r.a = __ldcs(reinterpret_cast<const uint4*>(p));
  } else {
    const uint2 x = __ldcs(reinterpret_cast<const uint2*>(p)), y = __ldcs(reinterpret_cast<const uint2*>(p + gap));
    r.a = make_uint4(x.x, x.y, y.x, y.y);
  }
  return r;
}
template <typename X>
__device__ __forceinline__ V8 widen(const Raw8<X>& r) {
  V8 o;
  if constexpr (sizeof(X) == 4) {
    const uint32_t u[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) o.p[i] = make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
  } else {
    const uint32_t u[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) o.p[i] = unpack_pair<X>(u[i]);
  }
  return o;
}
template <typename X, bool INTER>
__device__ __forceinline__ void store8(X* p, int gap, const V8& o) {
  if constexpr (sizeof(X) == 4) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(o.p[0].x, o.p[0].y, o.p[1].x, o.p[1].y));
    __stcs(reinterpret_cast<float4*>(p + gap), make_float4(o.p[2].x, o.p[2].y, o.p[3].x, o.p[3].y));
  } else {
    const uint32_t a = pack_pair<X>(o.p[0].x, o.p[0].y), b = pack_pair<X>(o.p[1].x, o.p[1].y),
                   c = pack_pair<X>(o.p[2].x, o.p[2].y), d = pack_pair<X>(o.p[3].x, o.p[3].y);
    if constexpr (INTER) {
      __stcs(reinterpret_cast<uint4*>(p), make_uint4(a, b, c, d));
    } else {
      __stcs(reinterpret_cast<uint2*>(p), make_uint2(a, b));
      __stcs(reinterpret_cast<uint2*>(p + gap), make_uint2(c, d));
    }
  }
}
// Weight e of the run-time type w_dtype (0 past D).
__device__ __forceinline__ float weight_at(const void* w, int w_dtype, int e, int D) {
  if (e >= D) return 0.f;
  return w_dtype == CSA_F32   ? static_cast<const float*>(w)[e]
         : w_dtype == CSA_F16 ? __half2float(static_cast<const __half*>(w)[e])
                              : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[e]);
}
__device__ __forceinline__ V8 load_weight(const void* w, int w_dtype, int e, int gap, int D) {
  V8 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = e + (i >> 1) * gap + 2 * (i & 1);
    o.p[i] = make_float2(weight_at(w, w_dtype, at, D), weight_at(w, w_dtype, at + 1, D));
  }
  return o;
}

// The eight values of lane l of a row: e .. e+3 and e+gap .. e+gap+3.  Halves:
// the first rot/8 lanes hold four pairs each, (e, e+rot/2) and so on; the other
// lanes, and all lanes of interleaved rows, eight consecutive values.  e >= D: none.
struct Lane {
  int e, gap;
};
template <bool INTER>
__device__ __forceinline__ Lane make_lane(const NormRopeParams& p, int l) {
  if constexpr (INTER) return Lane{8 * l, 4};
  const int n = p.rot / 8;
  if (l < n) return Lane{p.off + 4 * l, p.rot / 2};
  const int e = 8 * (l - n);
  return Lane{e < p.off ? e : e + p.rot, 4};
}

template <int G>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Cosines and sines of the tokens t0 .. t0+n-1, rot/2 of each.  A lane takes
// four pairs of a token; pair p stands at (p % 4) * (rot/8) + p / 4, so that the
// lanes of a row read consecutive words (in the pairs' own order they meet in
// two to four banks).
__device__ __forceinline__ void fill_angles(const NormRopeParams& p, int t0, int n, float2* cs) {
  const int half = p.rot / 2, lanes = half / 4;
  for (int i = threadIdx.x; i < n * half; i += kThreads) {
    const int t = i / half, j = i - t * half;
    const uint64_t turns = static_cast<uint64_t>(p.pos[t0 + t]) * p.freqs[j];
    const float x = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 4.656612873077393e-10f;  // 2^-31
    float s, c;
    sincospif(x, &s, &c);
    cs[t * half + (j & 3) * lanes + (j >> 2)] = make_float2(c, s);
  }
}

// Turning as two products: value <- value * c + partner * s, both values of a
// pair being in the same lane, with s of the sign that its place asks for.  In
// the forward the weights are part of c and s (the partner's of s), formed once
// per token; rows of a token follow each other.  Values that are not turned
// have c = 1 (the weight) and s = 0.
template <bool INTER, bool BWD>
struct Turn {
  bool in;     // the values are turned
  int first;   // the lane's place among those of the pairs
  int lanes;   // lanes of the pairs
  int token;   // whose c and s are held
  float2 c[4], s[4];

  __device__ __forceinline__ Turn(const NormRopeParams& p, const Lane& ln) {
    const int r = ln.e - p.off;
    in = r >= 0 && r < (INTER ? p.rot : p.rot / 2);
    lanes = p.rot / 8;
    first = in ? r / (INTER ? 8 : 4) : 0;
    token = -1;
  }
  // The partners of v's values.
  __device__ __forceinline__ static V8 partners(const V8& v) {
    V8 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.p[i] = INTER ? make_float2(v.p[i].y, v.p[i].x) : v.p[i ^ 2];
    return o;
  }
  // c and s of token `tok` of those in `all`; w: this lane's weights (forward)
  __device__ __forceinline__ void hold(const float2* all, int tok, const V8& w) {
    if (tok == token) return;
    token = tok;
    const V8 wo = partners(w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = make_float2(1.f, 1.f);
      s[i] = make_float2(0.f, 0.f);
      if (in) {
        if constexpr (INTER) {
          const float2 a = all[(tok * 4 + i) * lanes + first];
          c[i] = make_float2(a.x, a.x);
          s[i] = BWD ? make_float2(a.y, -a.y) : make_float2(-a.y, a.y);
        } else {
          const int k = 2 * (i & 1);
          const float2 a = all[(tok * 4 + k) * lanes + first], b = all[(tok * 4 + k + 1) * lanes + first];
          c[i] = make_float2(a.x, b.x);
          s[i] = ((i < 2) != BWD) ? make_float2(-a.y, -b.y) : make_float2(a.y, b.y);
        }
      }
      if constexpr (!BWD) {
        c[i] = fmul2(c[i], w.p[i]);
        s[i] = fmul2(s[i], wo.p[i]);
      }
    }
  }
  __device__ __forceinline__ float2 turned(const V8& v, int i) const {
    const V8 o = partners(v);
    return ffma2(o.p[i], s[i], fmul2(v.p[i], c[i]));
  }
};

// The rows (token, head) of q or of k, as one block sees them: the blocks of
// a launch are dealt to q and k in proportion to their rows, so that weights,
// strides and head count are the same for all rows of a block.
template <typename X>
struct Part {
  const X* x;
  const X* g;  // cotangents (backward)
  X* y;
  const void* w;
  long long st, sh, rows;
  int H;
  bool is_q;
  int block, blocks;  // this block among those of its part
};
template <typename X>
__device__ __forceinline__ Part<X> make_part(const NormRopeParams& p) {
  Part<X> a;
  a.is_q = static_cast<int>(blockIdx.x) < p.q_blocks;
  a.x = static_cast<const X*>(a.is_q ? p.q : p.k);
  a.g = static_cast<const X*>(a.is_q ? p.gq : p.gk);
  a.y = static_cast<X*>(a.is_q ? p.yq : p.yk);
  a.w = a.is_q ? p.qw : p.kw;
  a.st = a.is_q ? p.q_st : p.k_st;
  a.sh = a.is_q ? p.q_sh : p.k_sh;
  a.H = a.is_q ? p.Hq : p.Hk;
  a.rows = static_cast<long long>(p.T) * a.H;
  a.block = static_cast<int>(blockIdx.x) - (a.is_q ? 0 : p.q_blocks);
  a.blocks = a.is_q ? p.q_blocks : static_cast<int>(gridDim.x) - p.q_blocks;
  return a;
}

// Position (token, head) of a row, moved on by a fixed number of rows without
// divisions; next() says whether the head count was passed.
struct Walk {
  int t, h, H, dt, dh;
  __device__ __forceinline__ Walk(long long row, int heads, int step) : H(heads) {
    t = static_cast<int>(row / heads);
    h = static_cast<int>(row - static_cast<long long>(t) * heads);
    dt = step / heads;
    dh = step - dt * heads;
  }
  __device__ __forceinline__ bool next() {
    t += dt;
    h += dh;
    const bool wrap = h >= H;
    if (wrap) {
      h -= H;
      ++t;
    }
    return wrap;
  }
};

// A block takes a run of chunks of PER * U consecutive rows; a thread's row u of
// the next chunk is requested as soon as row u of this one is taken from its
// registers, so loads are always in flight, and the next chunk's cosines and
// sines are formed while this one is worked on (one barrier a chunk).
template <typename X, int G, bool INTER, int U, bool BWD>
__global__ void __launch_bounds__(kThreads, kBlocks<X, BWD>) norm_rope_kernel(const NormRopeParams p) {
  extern __shared__ float2 cs_all[];
  constexpr int PER = kThreads / G, CHUNK = PER * U;
  const Part<X> a = make_part<X>(p);
  const Lane ln = make_lane<INTER>(p, threadIdx.x % G);
  const int e = ln.e, gap = ln.gap;
  const bool lane_ok = e < p.D;
  const long long chunks = (a.rows + CHUNK - 1) / CHUNK;
  const long long c0 = chunks * a.block / a.blocks, c1 = chunks * (a.block + 1) / a.blocks;
  float2 acc[4] = {};  // gradients of the weights
  if (c0 < c1) {
    const int half = p.rot / 2, cs_size = p.cs_tokens * half;
    const V8 w = load_weight(a.w, p.w_dtype, e, gap, p.D);
    Turn<INTER, BWD> tn(p, ln);
    // Pointers and 32-bit counts instead of row numbers: the integer work of a row is half of its instructions.
    const long long row0 = c0 * CHUNK + threadIdx.x / G, end = min(a.rows, c1 * CHUNK);
    Walk blk(c0 * CHUNK, a.H, CHUNK);  // first row of the chunk whose angles are formed
    Walk cur(row0, a.H, PER);          // the row worked on
    Walk ahead = cur;                  // the row requested
    int left = row0 < end ? static_cast<int>(min((end - row0 + PER - 1) / PER, 0x3fffffffll)) : 0, left_ahead = left;
    const X* xp = a.x + ahead.t * a.st + ahead.h * a.sh + e;
    const X* gp = BWD ? a.g + row0 * p.D + e : nullptr;
    X* yp = a.y + row0 * p.D + e;
    const long long step = ahead.dt * a.st + ahead.dh * a.sh, wrap = a.st - a.H * a.sh;
    const int lin = PER * p.D, nc = static_cast<int>(c1 - c0);
    Raw8<X> rx[U], rg[BWD ? U : 1];
    auto request = [&](int u) {
      rx[u] = Raw8<X>{};
      if constexpr (BWD) rg[u] = Raw8<X>{};
      if (left_ahead > 0 && lane_ok) {
        rx[u] = load8<X, INTER>(xp, gap);
        if constexpr (BWD) rg[u] = load8<X, INTER>(gp, gap);
      }
      --left_ahead;
      xp += step;
      if (ahead.next()) xp += wrap;
      if constexpr (BWD) gp += lin;
    };
    auto angles = [&](float2* cs) {
      // tokens blk.t .. of this chunk's rows
      const int n = blk.dt + (blk.h + blk.dh > 0 ? 1 : 0) + (blk.h + blk.dh > a.H ? 1 : 0);
      fill_angles(p, blk.t, min(n, p.T - blk.t), cs);
    };
#pragma unroll
    for (int u = 0; u < U; ++u) request(u);
    cur.t -= blk.t;  // counted from the chunk's first token
    int buf = 0;
    angles(cs_all);
    __syncthreads();
    for (int c = 0; c < nc; ++c) {
      const int t_first = blk.t;
      blk.next();
      const float2* cs = cs_all + buf * cs_size;
      if (c + 1 < nc) angles(cs_all + (buf ^ 1) * cs_size);
      tn.token = -1;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const Raw8<X> raw = BWD ? rg[BWD ? u : 0] : rx[u];  // what is turned: the cotangent, or the row
        V8 x = widen(rx[u]);
        const V8 v = BWD ? widen(raw) : x;
        request(u);
        const bool ok = left > 0;
        tn.hold(cs, ok ? cur.t : 0, w);
        float2 ss = fmul2(x.p[0], x.p[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) ss = ffma2(x.p[i], x.p[i], ss);
        float r = rsqrtf(group_sum<G>(ss.x + ss.y) * p.inv_d + p.eps);
        if (BWD && !ok) r = 0.f;  // no row: nothing may reach the weights' sums (eps may be 0)
        const float2 r2 = make_float2(r, r);
        V8 y;
        if constexpr (BWD) {
          float2 dot = make_float2(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 z = tn.turned(v, i), xh = fmul2(x.p[i], r2);
            const float2 zx = fmul2(z, xh);
            acc[i] = fadd2(acc[i], zx);
            dot = ffma2(zx, w.p[i], dot);
            y.p[i] = fmul2(z, w.p[i]);
            x.p[i] = xh;
          }
          const float m = -group_sum<G>(dot.x + dot.y) * p.inv_d;
#pragma unroll
          for (int i = 0; i < 4; ++i) y.p[i] = fmul2(r2, ffma2(x.p[i], make_float2(m, m), y.p[i]));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) y.p[i] = fmul2(r2, tn.turned(x, i));
        }
        if (ok && lane_ok) store8<X, INTER>(yp, gap, y);
        cur.next();
        --left;
        yp += lin;
      }
      cur.t -= blk.t - t_first;
      buf ^= 1;
      __syncthreads();
    }
  }
  if constexpr (BWD) {
    // the block's groups join their sums; one partial row per block, added in order by a second kernel
    __shared__ float red[kThreads * 8];  // [PER][8 G], by the lanes' own order of values
    float* mine = red + (threadIdx.x / G) * (8 * G);
    __syncthreads();
    if (lane_ok) {
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<float2*>(mine + e + (i >> 1) * gap + 2 * (i & 1)) = acc[i];
    }
    __syncthreads();
    for (int d = threadIdx.x; d < p.D; d += kThreads) {
      float s = 0.f;
      for (int r = 0; r < PER; ++r) s += red[r * (8 * G) + d];
      p.part[static_cast<size_t>(blockIdx.x) * p.D + d] = s;
    }
  }
}

// dqw, dkw = sums of the partial rows (q's blocks first): 32 columns of one of
// them and 32 runs of rows per block.
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float* part, int nq, int nk, int D, float* dqw,
                                                           float* dkw) {
  __shared__ float red[32][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), run = threadIdx.x >> 5;
  const bool q = blockIdx.y == 0;
  float s = 0.f;
  if (c < D)
    for (int i = run; i < (q ? nq : nk); i += 32) s += part[static_cast<size_t>(q ? i : nq + i) * D + c];
  red[run][threadIdx.x & 31] = s;
  __syncthreads();
  if (run == 0 && c < D) {
    for (int i = 1; i < 32; ++i) s += red[i][threadIdx.x & 31];
    (q ? dqw : dkw)[c] = s;
  }
}

template <typename X, int G, bool INTER, bool BWD>
cudaError_t run(NormRopeParams p, cudaStream_t stream) {
  constexpr int PER = kThreads / G, U = BWD ? kRowsBwd : kRowsFwd, CHUNK = PER * U;
  // blocks of q and k in proportion to their chunks, all on the GPU at once
  auto chunks = [&](int H) { return (static_cast<long long>(p.T) * H + CHUNK - 1) / CHUNK; };
  const long long cq = chunks(p.Hq), ck = chunks(p.Hk), most = 152 * kBlocks<X, BWD>;
  long long nq = cq, nk = ck;
  if (cq + ck > most) {
    nk = p.Hk > 0 ? std::max<long long>(1, std::min<long long>(ck, (most * ck + (cq + ck) / 2) / (cq + ck))) : 0;
    nq = std::min<long long>(cq, std::max<long long>(1, most - nk));
  }
  p.q_blocks = static_cast<int>(nq);
  // tokens that a chunk can meet, for both parts
  auto tokens = [&](int H) { return H > 0 ? std::min<long long>(p.T, (CHUNK - 1 + H - 1) / H + 1) : 0; };
  p.cs_tokens = static_cast<int>(std::max(tokens(p.Hq), tokens(p.Hk)));
  const size_t smem = static_cast<size_t>(2) * p.cs_tokens * (p.rot / 2) * sizeof(float2);
  cudaError_t e = cudaSuccess;
  if (smem > 40 * 1024 && (e = smem_limit_once<norm_rope_kernel<X, G, INTER, U, BWD>>(80 * 1024)) != cudaSuccess) return e;
  norm_rope_kernel<X, G, INTER, U, BWD><<<static_cast<unsigned>(nq + nk), kThreads, smem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || !BWD) return e;
  norm_rope_dw_kernel<<<dim3((p.D + 31) / 32, p.Hk > 0 ? 2 : 1), 1024, 0, stream>>>(
      p.part, static_cast<int>(nq), static_cast<int>(nk), p.D, p.dqw, p.dkw);
  return cudaGetLastError();
}

template <typename X, bool INTER>
cudaError_t by_size(const NormRopeParams& p, bool bwd, cudaStream_t s) {
  if (p.D <= 32) return bwd ? run<X, 4, INTER, true>(p, s) : run<X, 4, INTER, false>(p, s);
  if (p.D <= 64) return bwd ? run<X, 8, INTER, true>(p, s) : run<X, 8, INTER, false>(p, s);
  if (p.D <= 128) return bwd ? run<X, 16, INTER, true>(p, s) : run<X, 16, INTER, false>(p, s);
  return bwd ? run<X, 32, INTER, true>(p, s) : run<X, 32, INTER, false>(p, s);
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
