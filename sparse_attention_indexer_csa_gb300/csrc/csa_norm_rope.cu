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
// Both values of a pair are in the same lane.  A group of lanes takes rows in
// units of up to eight consecutive ones (head-fastest) and forms the cosines and
// sines of a token itself when it comes to it: four pairs a lane, once for the
// token's heads in the unit.  (In shared memory, once per block, they cost a
// barrier and its wait per chunk: 126 us against 98 for 16384 tokens.)  The units
// of all groups lie side by side in memory: one long run of rows for each group
// took 122 us, since as many places of the memory were open as there are groups.
//
// Measured (bf16, 64 + 8 heads of 128): forward, 16384 tokens, all values
// rotated, 98 us (6.15 TB/s, a plain copy gives 6.69); 32768 tokens, half
// rotated in neighbouring pairs, 189 us (6.4 TB/s), gradients 294 us (6.2
// TB/s).  64 tokens: 4.6 us, a launch.
// With the append of keys and values to a paged cache (APPEND): 16384 tokens, 120 us
// (5.6 TB/s; q 81 us and, in a launch of their own, k and v 34), 64 tokens, 5.7 us.
//
// Angles: position * freq modulo 2^64 is the fraction of a turn with 64 bits
// after the point, exactly what the table says whatever the position; its upper 32
// bits, as a signed number of half turns, go to sincospif (absolute error of the
// angle below 2e-7, against about 0.06 for a 32-bit product at position 1e6).  The
// table's own rounding adds 1.8e-19 per position: as much near position 1e12.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "csa_attn_internal.h"
#include "csa_attn_tiles.cuh"
#include "csa_sparse_internal.h"

namespace csa {
namespace {

constexpr int kThreads = 256;
// Rows of a thread on their way (gradients of 32768 tokens: 3, 313 us; 4, 294; fp32 has registers for two).
template <typename X, bool BWD>
constexpr int kRows = BWD && sizeof(X) == 4 ? 2 : 4;
// Consecutive rows of a group of lanes, at most (16384 tokens: 4, 104 us; 8, 98; 16, 124; 32, 120).
constexpr int kUnit = 8;
// Blocks per SM (the registers a thread has): fp32 rows take twice the
// registers while they are on their way, and spill at three.
// An append's rows of the cache take as many more.
template <typename X, bool BWD, bool APPEND = false>
constexpr int kBlocks = BWD || APPEND || sizeof(X) == 4 ? 2 : 3;

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
// Eight values as they were loaded.
template <typename X, bool INTER>
__device__ __forceinline__ void store_raw(X* p, int gap, const Raw8<X>& r) {
  if constexpr (sizeof(X) == 4) {
    __stcs(reinterpret_cast<uint4*>(p), r.a);
    __stcs(reinterpret_cast<uint4*>(p + gap), r.b);
  } else if constexpr (INTER) {
    __stcs(reinterpret_cast<uint4*>(p), r.a);
  } else {
    __stcs(reinterpret_cast<uint2*>(p), make_uint2(r.a.x, r.a.y));
    __stcs(reinterpret_cast<uint2*>(p + gap), make_uint2(r.a.z, r.a.w));
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

// Turning as two products: value <- value * c + partner * s, both values of a
// pair being in the same lane, with s of the sign that its place asks for.  In
// the forward the weights are part of c and s (the partner's of s).  Values
// that are not turned have c = 1 (the weight) and s = 0.
template <bool INTER, bool BWD>
struct Turn {
  const uint64_t* freqs;  // of the lane's four pairs; null: its values are not turned
  float2 c[4], s[4];

  __device__ __forceinline__ Turn(const NormRopeParams& p, const Lane& ln, const V8& w) {
    const int r = ln.e - p.off;
    freqs = r >= 0 && r < (INTER ? p.rot : p.rot / 2) ? p.freqs + (INTER ? r / 2 : r) : nullptr;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = BWD ? make_float2(1.f, 1.f) : w.p[i];
      s[i] = make_float2(0.f, 0.f);
    }
  }
  // The partners of v's values.
  __device__ __forceinline__ static V8 partners(const V8& v) {
    V8 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.p[i] = INTER ? make_float2(v.p[i].y, v.p[i].x) : v.p[i ^ 2];
    return o;
  }
  // c and s of a position; w: this lane's weights (forward)
  __device__ __forceinline__ void set(int64_t pos, const V8& w) {
    if (freqs == nullptr) return;
    float2 a[4];  // cosine and sine of each pair
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t turns = static_cast<uint64_t>(pos) * freqs[i];
      sincospif(static_cast<float>(static_cast<int32_t>(turns >> 32)) * 4.656612873077393e-10f, &a[i].y, &a[i].x);  // 2^-31
    }
    const V8 wo = partners(w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (INTER) {
        c[i] = make_float2(a[i].x, a[i].x);
        s[i] = BWD ? make_float2(a[i].y, -a[i].y) : make_float2(-a[i].y, a[i].y);
      } else {
        const int k = 2 * (i & 1);
        c[i] = make_float2(a[k].x, a[k + 1].x);
        s[i] = ((i < 2) != BWD) ? make_float2(-a[k].y, -a[k + 1].y) : make_float2(a[k].y, a[k + 1].y);
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
// What an append adds to the problem, and the blocks that work on k (those behind work on v).
struct AppendArgs {
  AppendParams c;
  int k_blocks;
};
struct NoAppend {};

// The cache row of a token.  Consecutive tokens are mostly of the sequence of
// the one before, whose extent is kept.
struct Places {
  int q0 = 0, q1 = 0;  // tokens of the sequence
  int off = 0;         // place of a token: t + off
  int seq = -1;
  // page * page size + row of token t; -1: it is not stored
  __device__ __forceinline__ long long find(const AppendParams& c, int T, int t) {
    if (t >= T || c.N <= 0) return -1;
    if (t < q0 || t >= q1) {
      // sequences of equal lengths (one token each, when decoding) are met at the first look
      int lo = static_cast<int>(static_cast<long long>(t) * c.N / T);
      int a = c.cu_q[lo], b = c.cu_q[lo + 1];
      if (t < a || t >= b) {
        int hi = c.N;  // the largest i with cu_q[i] <= t
        lo = 0;
        while (lo < hi) {
          const int i = (lo + hi + 1) >> 1;
          if (c.cu_q[i] <= t)
            lo = i;
          else
            hi = i - 1;
        }
        if (lo >= c.N) return -1;
        a = c.cu_q[lo];
        b = c.cu_q[lo + 1];
        if (t < a || t >= b) return -1;
      }
      q0 = max(a, 0);
      q1 = min(b, T);
      seq = lo;
      if (a != q0 || b != q1) record_error(kErrDevice);
      off = min(max(c.k_len[lo], 0), 0x7FFFFFFF - T) - q1;
    }
    const int j = t + off;
    const int n = j >= 0 ? j / c.page : 0;
    if (j < 0 || n >= c.table_width) {
      record_error(kErrDevice);
      return -1;
    }
    const int pg = c.table[seq * c.table_st + n];
    if (pg < 0 || pg >= c.pages) {
      record_error(kErrDevice);
      return -1;
    }
    return static_cast<long long>(pg) * c.page + (j - n * c.page);
  }
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

// A stretch of n() rows: one token's from head h on, in a unit of which k rows are left.
struct Stretch {
  int t, h, k;
  __device__ __forceinline__ int n(int H) const { return min(H - h, k); }
  // The one that follows; true where it opens the group's next unit.
  __device__ __forceinline__ bool advance(const RowDeal& d, int H) {
    const int m = n(H);
    if (k > m) {
      ++t;
      h = 0;
      k -= m;
      return false;
    }
    t += d.dt;
    h += m + d.dh;
    if (h >= H) {
      h -= H;
      ++t;
    }
    k = d.R;
    return true;
  }
};

// A row is requested U rows before it is worked on, as soon as its registers
// are free.  All groups walk as far (the shuffles need whole warps); what lies
// past a group's rows is neither read nor written.
//
// APPEND: k's rows go to the cache, and a third part of the blocks copies v's rows there.
template <typename X, int G, bool INTER, int U, bool BWD, bool APPEND = false>
__global__ void __launch_bounds__(kThreads, kBlocks<X, BWD, APPEND>)
    norm_rope_kernel(const NormRopeParams p, const std::conditional_t<APPEND, AppendArgs, NoAppend> more) {
  constexpr int PER = kThreads / G;
  Part<X> a = make_part<X>(p);
  bool is_v = false;
  if constexpr (APPEND) {
    is_v = !a.is_q && a.block >= more.k_blocks;
    if (is_v) {
      a.x = static_cast<const X*>(more.c.v);
      a.st = more.c.v_st;
      a.sh = more.c.v_sh;
      a.block -= more.k_blocks;
    }
  }
  const Lane ln = make_lane<INTER>(p, threadIdx.x % G);
  const int e = ln.e, gap = ln.gap;
  const bool lane_ok = e < p.D;
  const int group = a.block * PER + threadIdx.x / G;
  const RowDeal deal = a.is_q ? p.deal_q : p.deal_k;
  // rows of this group: only its last unit may be short
  const long long last = a.rows - (static_cast<long long>(deal.rounds - 1) * deal.groups + group) * deal.R;
  int left = (deal.rounds - 1) * deal.R + static_cast<int>(min(max(last, 0ll), static_cast<long long>(deal.R)));
  int left_ahead = left;
  const V8 w = load_weight(a.w, p.w_dtype, e, gap, p.D);
  Turn<INTER, BWD> tn(p, ln, w);
  const long long row0 = static_cast<long long>(group) * deal.R;
  const int t0 = a.rows < 0x7FFFFFFFll ? static_cast<int>(row0) / a.H : static_cast<int>(row0 / a.H);
  Stretch now{t0, static_cast<int>(row0 - static_cast<long long>(t0) * a.H), deal.R};  // of the row worked on
  Stretch ahead = now;                                                                // of the row requested
  const X* xp = a.x + ahead.t * a.st + ahead.h * a.sh + e;
  const X* gp = BWD ? a.g + row0 * p.D + e : nullptr;
  X* yp = APPEND && !a.is_q ? nullptr : a.y + row0 * p.D + e;
  float2 acc[4] = {};  // gradients of the weights
  Raw8<X> rx[U], rg[BWD ? U : 1];
  int n_ahead = ahead.n(a.H), n_now = n_ahead;
  auto request = [&](int u) {
    rx[u] = Raw8<X>{};
    if constexpr (BWD) rg[u] = Raw8<X>{};
    if (left_ahead > 0 && lane_ok) {
      rx[u] = load8<X, INTER>(xp, gap);
      if constexpr (BWD) rg[u] = load8<X, INTER>(gp, gap);
    }
    --left_ahead;
    xp += a.sh;
    if constexpr (BWD) gp += p.D;
    if (--n_ahead == 0) {
      const bool jump = ahead.advance(deal, a.H);
      n_ahead = ahead.n(a.H);
      xp = a.x + ahead.t * a.st + ahead.h * a.sh + e;
      if (BWD && jump) gp += static_cast<long long>(deal.skip) * p.D;
    }
  };
  // the position of the coming stretch is on its way while this one's heads are worked on
  auto position = [&](const Stretch& s) { return static_cast<unsigned>(s.t) < static_cast<unsigned>(p.T) ? p.pos[s.t] : 0; };
  auto coming = [&]() {
    Stretch s = now;
    s.advance(deal, a.H);
    return position(s);
  };
#pragma unroll
  for (int u = 0; u < U; ++u) request(u);
  int64_t pos = coming();
  Places places;
  long long y_step = p.D;  // between two rows of a stretch
  // the cache row of a stretch (its page is looked up with the coming position), and the pointer into it
  auto place = [&](const Stretch& s) -> long long {
    if constexpr (APPEND) {
      if (!a.is_q && static_cast<unsigned>(s.t) < static_cast<unsigned>(p.T)) return places.find(more.c, p.T, s.t);
    }
    return -1;
  };
  auto cache_row = [&](long long at, int h) -> X* {
    if constexpr (APPEND) {
      if (at < 0) return nullptr;
      const AppendParams& c = more.c;
      const long long page = at / c.page, row = at - page * c.page;
      return is_v ? static_cast<X*>(c.vc) + page * c.vc_sp + row * c.vc_st + h * c.vc_sh + e
                  : static_cast<X*>(c.kc) + page * c.kc_sp + row * c.kc_st + h * c.kc_sh + e;
    }
    return nullptr;
  };
  auto coming_place = [&]() {
    Stretch s = now;
    s.advance(deal, a.H);
    return place(s);
  };
  long long next_at = -1;
  if constexpr (APPEND) {
    if (!a.is_q) {
      y_step = is_v ? more.c.vc_sh : more.c.kc_sh;
      if (left > 0) yp = cache_row(place(now), now.h);
      if (left > n_now) next_at = coming_place();
    }
  }
  tn.set(position(now), w);
  const int most = deal.rounds * deal.R;  // all groups walk as far
  for (int i = 0; i < most; i += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Raw8<X> raw = BWD ? rg[BWD ? u : 0] : rx[u];  // what is turned: the cotangent, or the row
      V8 x = widen(rx[u]);
      const V8 v = BWD ? widen(raw) : x;
      request(u);
      const bool ok = left > 0;
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
      if constexpr (APPEND) {
        if (ok && lane_ok && yp != nullptr) {
          if (is_v)
            store_raw<X, INTER>(yp, gap, raw);
          else
            store8<X, INTER>(yp, gap, y);
        }
        if (yp != nullptr) yp += y_step;
      } else {
        if (ok && lane_ok) store8<X, INTER>(yp, gap, y);
        yp += p.D;
      }
      --left;
      if (--n_now == 0) {
        const bool jump = now.advance(deal, a.H);
        if (jump && !(APPEND && !a.is_q)) yp += static_cast<long long>(deal.skip) * p.D;
        n_now = now.n(a.H);
        if constexpr (APPEND) {
          if (!a.is_q) {
            yp = cache_row(next_at, now.h);
            next_at = left > n_now ? coming_place() : -1;
          }
        }
        tn.set(pos, w);
        pos = coming();
      }
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

// See RowDeal; rows > 0, groups > 0.
RowDeal deal_rows(long long rows, long long groups, int H) {
  RowDeal d;
  const long long rounds = (rows + groups * kUnit - 1) / (groups * kUnit);
  d.groups = static_cast<int>(groups);
  d.rounds = static_cast<int>(rounds);
  d.R = static_cast<int>((rows + groups * rounds - 1) / (groups * rounds));  // at most kUnit: only the last round is short
  d.skip = static_cast<int>((groups - 1) * d.R);
  d.dt = d.skip / H;
  d.dh = d.skip % H;
  return d;
}

template <typename X, int G, bool INTER, bool BWD>
cudaError_t run(NormRopeParams p, cudaStream_t stream) {
  constexpr int PER = kThreads / G, U = kRows<X, BWD>, CHUNK = PER * U;
  // Blocks of q and k in proportion to their chunks, all on the GPU at once.  A
  // small call has U rows for each group of lanes (64 tokens: 4.7 us; one row for each, 7.1).
  auto chunks = [&](int H) { return (static_cast<long long>(p.T) * H + CHUNK - 1) / CHUNK; };
  const long long cq = chunks(p.Hq), ck = chunks(p.Hk), most = 152 * kBlocks<X, BWD>;
  long long nq = cq, nk = ck;
  if (cq + ck > most) {
    nk = p.Hk > 0 ? std::max<long long>(1, std::min<long long>(ck, (most * ck + (cq + ck) / 2) / (cq + ck))) : 0;
    nq = std::min<long long>(cq, std::max<long long>(1, most - nk));
  }
  p.q_blocks = static_cast<int>(nq);
  p.deal_q = deal_rows(static_cast<long long>(p.T) * p.Hq, nq * PER, p.Hq);
  if (nk > 0) p.deal_k = deal_rows(static_cast<long long>(p.T) * p.Hk, nk * PER, p.Hk);
  norm_rope_kernel<X, G, INTER, U, BWD><<<static_cast<unsigned>(nq + nk), kThreads, 0, stream>>>(p, NoAppend{});
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !BWD) return e;
  norm_rope_dw_kernel<<<dim3((p.D + 31) / 32, p.Hk > 0 ? 2 : 1), 1024, 0, stream>>>(
      p.part, static_cast<int>(nq), static_cast<int>(nk), p.D, p.dqw, p.dkw);
  return cudaGetLastError();
}

// Blocks of q, of k and of v, in proportion to their rows, in one launch where all
// of them are on the GPU at once (64 tokens: 5.7 us).  More rows go in two: q as in
// norm_rope, with three blocks per SM, since the cache's rows take registers that
// leave room for two (16384 tokens, 64 + 8 heads: 140 us in one launch, 121 in two).
template <typename X, int G, bool INTER>
cudaError_t run_append(NormRopeParams p, const AppendParams& c, cudaStream_t stream) {
  constexpr int PER = kThreads / G, U = kRows<X, false>, CHUNK = PER * U;
  auto chunks = [&](int H) { return (static_cast<long long>(p.T) * H + CHUNK - 1) / CHUNK; };
  const long long most = 152 * kBlocks<X, false, true>;
  long long nq = chunks(p.Hq), nk = chunks(p.Hk);
  if (nq + 2 * nk > most) {
    NormRopeParams q = p;
    q.Hk = 0;
    const cudaError_t e = run<X, G, INTER, false>(q, stream);
    if (e != cudaSuccess) return e;
    nq = 0;
    nk = std::min(nk, most / 2);
  }
  p.q_blocks = static_cast<int>(nq);
  if (nq > 0) p.deal_q = deal_rows(static_cast<long long>(p.T) * p.Hq, nq * PER, p.Hq);
  p.deal_k = deal_rows(static_cast<long long>(p.T) * p.Hk, nk * PER, p.Hk);
  const AppendArgs more{c, static_cast<int>(nk)};
  norm_rope_kernel<X, G, INTER, U, false, true><<<static_cast<unsigned>(nq + 2 * nk), kThreads, 0, stream>>>(p, more);
  return cudaGetLastError();
}
template <typename X, bool INTER>
cudaError_t append_by_size(const NormRopeParams& p, const AppendParams& c, cudaStream_t s) {
  if (p.D <= 32) return run_append<X, 4, INTER>(p, c, s);
  if (p.D <= 64) return run_append<X, 8, INTER>(p, c, s);
  if (p.D <= 128) return run_append<X, 16, INTER>(p, c, s);
  return run_append<X, 32, INTER>(p, c, s);
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
cudaError_t launch_norm_rope_append(const NormRopeParams& p, const AppendParams& c, int dtype, bool inter,
                                    cudaStream_t s) {
  if (dtype == CSA_F32) return inter ? append_by_size<float, true>(p, c, s) : append_by_size<float, false>(p, c, s);
  if (dtype == CSA_F16) return inter ? append_by_size<__half, true>(p, c, s) : append_by_size<__half, false>(p, c, s);
  return inter ? append_by_size<__nv_bfloat16, true>(p, c, s) : append_by_size<__nv_bfloat16, false>(p, c, s);
}

cudaError_t take_status_append(uint32_t* out, cudaStream_t stream) { return take_status(out, stream); }

}  // namespace csa
