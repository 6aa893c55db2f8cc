// csa_attn_bwd.cu -- gradients of causal attention over packed sequences on
// the tensor cores.
//
//   delta = dout.out  (per row and head)
//   p_j = exp(s_j - lse),  ds_j = p_j (dout.v_j - delta)
//   dq = scale sum_j ds_j k_j,  dk_j = scale sum_rows ds_j q,  dv_j = sum_rows p_j dout
//
// Three kernels: delta (one pass over dout and out), dq, and dk with dv.  The
// scores are formed again from q, k and lse in both of the latter; P and dS
// never leave the SM.  That is seven products per tile where one kernel
// for everything needs five, but every output is summed by one CTA in a fixed
// order: no atomics (the same bits on every call), no fp32 dq in memory, and
// dk, dv of a key head sum over its g query heads in place.
//
//   attn_dkv_kernel  a CTA takes up to 128 keys of one sequence and key head
//     and walks the rows that see them in blocks of 128 (rows = token * g +
//     head, as in the forward):
//       S^T = K Q^T, dP^T = V dO^T           (operands in shared memory)
//       P^T, dS^T in the storage type over S^T, dP^T in TMEM
//       dV += P^T dO, dK += dS^T Q           (A in TMEM, B read MN-major)
//     TMEM: S^T, dP^T, dV, dK, 128 columns each.  The issue order dV(i),
//     S^T(i+1), dK(i), dP^T(i+1) leaves the elementwise warps the time of two
//     products for each of their two halves.
//   attn_dq_kernel   a CTA takes a block of 128 rows and walks the key tiles:
//       S = Q K^T, dP = dO V^T, dS over dP in TMEM, dQ += dS K
//     TMEM: S, two dP, dQ.
//
// Warps (12): 0-7 elementwise (TMEM lanes 32 (w % 4) .., column half w / 4) and
// output; 8 issuer of the products; 9 TMA producer; 10 row statistics of the
// coming block (dkv) and what must be cleared in a tile's end; 11 none.
//
// A tile's end that belongs to another sequence may hold NaN, which a zero
// factor does not cancel: rows (dkv) or keys (dq) past the end are cleared in
// shared memory before any product reads them: such a tile lands on a barrier
// of its own, and the warp that cleared its end completes the tile's in the ring.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "csa_attn_internal.h"
#include "csa_attn_tiles.cuh"

namespace csa {
namespace {

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8, kMmaWarp = 8, kTmaWarp = 9, kPrepWarp = 10;

struct BwdArgs {
  AttnParams a;
  int tq;  // tokens per block of 128 rows
  int nb;  // dq: ceil(Tq / tq); dkv: ceil(Tk / 128)
  float c;
  unsigned long long wait_ns;
};

// Two resident tiles (dq: Q, dO; dkv: K, V) and two rings of tiles: E, whose
// tile is used first and last in a step (dq: K for S and dQ; dkv: Q for S^T and
// dK), and F (dq: V for dP; dkv: dO for dP^T and dV), which is free earlier.
// With three E and two F tiles each copy has the time of three to six products
// to arrive (two stages of both together left it two: 6000 cycles a step where
// the products need 2048).
template <int D>
struct BwdCfg {
  static constexpr uint32_t kTile = kChunkBytes * (D / 64);
  static constexpr int kE = D == 128 ? 3 : 5, kF = D == 128 ? 2 : 4;
  static constexpr uint32_t kOffA = 0, kOffB = kTile, kOffE = 2 * kTile, kOffF = kOffE + kE * kTile;
  static constexpr uint32_t kOffStat = kOffF + kF * kTile;  // [2][2][128] fp32: -lse log2 e, delta
  static constexpr uint32_t kOffBar = kOffStat + 2 * 2 * 128 * 4;
  static constexpr int kBarRes = 0, kBarE = 1, kBarF = kBarE + kE, kBarFreeE = kBarF + kF, kBarFreeF = kBarFreeE + kE,
                       kBarLast = kBarFreeF + kF, kBarStat = kBarLast + 2, kBarStatFree = kBarStat + 2,
                       kBarS = kBarStatFree + 2, kBarP = kBarS + 1, kBarDp = kBarP + 1, kBarDs = kBarDp + 2,
                       kBarAcc = kBarDs + 2, kBarDone = kBarAcc + 1, kBars = kBarDone + 1;
  static constexpr uint32_t kOffMisc = kOffBar + 8 * kBars, kSmem = kOffMisc + 64;
};
static_assert(BwdCfg<128>::kSmem <= 227 * 1024, "shared memory");

template <int D>
struct Cta {
  uint8_t* base;
  uint64_t* bars;
  WaitCtl ctl;
  uint32_t tmem;
};

// Common set-up: barriers, TMEM.  `work` is uniform over the CTA.
template <int D>
__device__ __forceinline__ void init_barriers(uint64_t* bars) {
  using C = BwdCfg<D>;
  for (int i = 0; i < C::kBars; ++i) {
    int n = 1;
    if (i == C::kBarStatFree || i == C::kBarStatFree + 1 || i == C::kBarP || i == C::kBarDs || i == C::kBarDs + 1)
      n = kEpiWarps;
    mbar_init(bars + i, n);
  }
  fence_mbar_init();
}

// S or dP of one tile: D[128,128] = A . B^T, both K-major over D.
template <typename X, int D>
__device__ __forceinline__ void product_abt(uint32_t d, uint64_t ad, uint64_t bd) {
  constexpr uint32_t kId = idesc_f16<X>(128, 128, false);
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    const uint64_t o = static_cast<uint64_t>(((ks >> 2) * kChunkBytes + (ks & 3) * 32) >> 4);
    umma_bf16(d, ad + o, bd + o, kId, ks != 0 ? 1u : 0u);
  }
}
// Acc[128,D] (+)= A . B with A in TMEM (two halves of 64 in columns 0.. and
// 64.. of `x`) and B [128,D] read MN-major.
template <typename X, int D>
__device__ __forceinline__ void product_acc(uint32_t acc, uint32_t x, uint64_t bd, bool first) {
  constexpr uint32_t kId = idesc_f16<X>(128, D, true);
#pragma unroll
  for (int ks = 0; ks < 8; ++ks)
    umma_bf16_tmem_a(acc, x + 64u * (ks >> 2) + 8u * (ks & 3), bd + static_cast<uint64_t>(128 * ks), kId,
                     (!first || ks != 0) ? 1u : 0u);
}

// Position in a ring of n tiles.
struct Ring {
  int n, at;
  uint32_t phase;
  __device__ explicit Ring(int size) : n(size), at(0), phase(0u) {}
  __device__ void next() {
    if (++at == n) {
      at = 0;
      phase ^= 1u;
    }
  }
};

// Waits until the copies of the first `used` tiles of a ring have landed.
__device__ __forceinline__ void drain_ring(uint64_t* full, int n, int used, const WaitCtl& ctl) {
  if (*ctl.abort_flag != 0u) return;
  volatile uint32_t dummy = 0;
  const WaitCtl dctl{&dummy, ctl.limit_ns};
  for (int i = 0; i < n && i < used; ++i)
    mbar_wait(full + (used - 1 - i) % n, (static_cast<uint32_t>(used - 1 - i) / n) & 1u, dctl);
}

// Copies tile i of a ring (rows: a block of query rows; else 128 keys).  The
// last tile lands on `last` instead when its end has to be cleared.
template <int D>
__device__ __forceinline__ void load_ring(uint8_t* base, uint32_t off, uint64_t* full, uint64_t* free, uint64_t* last,
                                          const Ring& r, const CUtensorMap* map, bool rows, int at, int hk,
                                          uint32_t bytes, uint64_t pol, const WaitCtl& ctl) {
  constexpr uint32_t kTile = kChunkBytes * (D / 64);
  if (!mbar_wait(free + r.at, r.phase ^ 1u, ctl)) return;
  uint64_t* bar = last != nullptr ? last : full + r.at;
  uint8_t* dst = base + off + r.at * kTile;
  mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
  for (int ch = 0; ch < D / 64; ++ch) {
    if (rows)
      tma_load_4d_hint(dst + ch * kChunkBytes, map, bar, ch * 64, 0, at, hk, pol);
    else
      tma_load_3d_hint(dst + ch * kChunkBytes, map, bar, ch * 64, at, hk, pol);
  }
}

// One accumulator lane (D fp32 values times f) to D values of X at dst.
template <typename X, int D>
__device__ __forceinline__ void store_lane(uint32_t t, float f, X* dst, bool some, bool write) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    float o[32];
    __syncwarp();
    if (some) {
      tmem_ld32_start(t + 32 * i, o);
      tmem_wait32(o);
    }
    if (!write) continue;
#pragma unroll
    for (int u = 0; u < 32; ++u) o[u] = some ? o[u] * f : 0.f;
    uint4* d4 = reinterpret_cast<uint4*>(dst + 32 * i);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      d4[u] = make_uint4(pack_pair<X>(o[8 * u], o[8 * u + 1]), pack_pair<X>(o[8 * u + 2], o[8 * u + 3]),
                         pack_pair<X>(o[8 * u + 4], o[8 * u + 5]), pack_pair<X>(o[8 * u + 6], o[8 * u + 7]));
  }
}

// ----------------------------------------------------------------- delta
// delta = dout.out: D/8 lanes per row and head, 16 bytes of each tensor a lane.
template <typename X, int D>
__global__ void __launch_bounds__(256) attn_delta_kernel(const AttnParams p) {
  constexpr int G = D / 8;
  const long long r = static_cast<long long>(blockIdx.x) * (256 / G) + threadIdx.x / G;
  const long long rows = static_cast<long long>(p.Tq) * p.Hq;
  const int l = threadIdx.x % G;
  float s = 0.f;
  if (r < rows) {
    const uint4 x = reinterpret_cast<const uint4*>(static_cast<const X*>(p.dout) + r * D)[l];
    const uint4 y = reinterpret_cast<const uint4*>(static_cast<const X*>(p.out) + r * D)[l];
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = unpack_pair<X>(xs[i]), b = unpack_pair<X>(ys[i]);
      s = fmaf(a.x, b.x, s);
      s = fmaf(a.y, b.y, s);
    }
  }
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (r < rows && l == 0) p.delta[r] = s;
}

// ----------------------------------------------------------------- dk, dv
template <typename X, int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_dkv_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_do,
                    const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                    const BwdArgs f) {
  using C = BwdCfg<D>;
  extern __shared__ __align__(1024) uint8_t base[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + C::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + C::kOffMisc);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(base + C::kOffMisc + 4);
  RowItem* item = reinterpret_cast<RowItem*>(base + C::kOffMisc + 16);
  const AttnParams& a = f.a;
  const int warp = threadIdx.x / 32;
  const uint32_t lane = lane_id();
  const int hk = static_cast<int>(blockIdx.x % a.Hk);

  if (warp == kMmaWarp) {
    const RowItem it = find_key_item(a, 128, f.nb, static_cast<int>(blockIdx.x / a.Hk));
    if (lane == 0) *item = it;
    if (blockIdx.x == 0)
      for (int i = static_cast<int>(lane); i < a.N; i += 32) seq_extent(a, i);
  }
  if (threadIdx.x == 0) {
    init_barriers<D>(bars);
    if ((smem_u32(base) & 1023u) != 0u) record_error(kErrDevice);  // the swizzled tiles would be misread
    *abort_flag = 0u;
  }
  __syncthreads();
  const RowItem it = *item;  // keys it.t0 .. it.t1-1 of the tensor
  if (it.t0 >= it.t1) return;

  // keys of the sequence among them, and the rows (tokens of the sequence) that see the first
  const int j0 = it.t0 - it.s.k0, lq = it.s.q1 - it.s.q0;
  const int n_key = max(0, min(it.t1 - it.t0, it.s.lk - j0));
  const int r_lo = n_key > 0 ? (a.causal ? min(lq, max(0, j0 - (it.s.lk - lq))) : 0) : lq;
  const int n_blk = (lq - r_lo + f.tq - 1) / f.tq;
  const bool work = n_blk > 0;
  const int rows_blk = f.tq * a.g;  // rows of a full block (128 when g divides it)

  if (work && rows_blk < 128)  // rows that no copy writes: zero factors must meet finite values
    for (int s = 0; s < C::kE + C::kF; ++s)
      clear_tile_rows<D>(base + C::kOffE + s * C::kTile, rows_blk, static_cast<int>(threadIdx.x), kThreads);
  fence_proxy_async_shared();
  if (work && warp == kMmaWarp) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const Cta<D> ct{base, bars, WaitCtl{abort_flag, f.wait_ns}, work ? *tmem_slot : 0u};
  const uint32_t t_s = ct.tmem, t_dp = ct.tmem + 128, t_dv = ct.tmem + 256, t_dk = ct.tmem + 384;
  const WaitCtl& ctl = ct.ctl;
  // the last block may hold fewer tokens than tq
  const int tail = lq - r_lo - (n_blk - 1) * f.tq;

  if (warp == kTmaWarp) {
    if (work && lane == 0) {
      const uint64_t first = l2_policy_evict_first(), last = l2_policy_evict_last();
      mbar_arrive_expect_tx(bars + C::kBarRes, 2 * C::kTile);
      for (int ch = 0; ch < D / 64; ++ch) {
        tma_load_3d_hint(base + C::kOffA + ch * kChunkBytes, &tmap_k, bars + C::kBarRes, ch * 64, it.t0, hk, first);
        tma_load_3d_hint(base + C::kOffB + ch * kChunkBytes, &tmap_v, bars + C::kBarRes, ch * 64, it.t0, hk, first);
      }
      Ring e(C::kE), o(C::kF);
      const uint32_t bytes = static_cast<uint32_t>(rows_blk) * 128u * (D / 64);
      for (int i = 0; i < n_blk; ++i) {
        const bool cut = i == n_blk - 1 && tail < f.tq;
        const int t = it.s.q0 + r_lo + i * f.tq;
        load_ring<D>(base, C::kOffE, bars + C::kBarE, bars + C::kBarFreeE, cut ? bars + C::kBarLast : nullptr, e, &tmap_q,
                     true, t, hk, bytes, last, ctl);
        load_ring<D>(base, C::kOffF, bars + C::kBarF, bars + C::kBarFreeF, cut ? bars + C::kBarLast + 1 : nullptr, o,
                     &tmap_do, true, t, hk, bytes, last, ctl);
        e.next();
        o.next();
      }
      drain_ring(bars + C::kBarE, C::kE, n_blk, ctl);
      drain_ring(bars + C::kBarF, C::kF, n_blk, ctl);
      mbar_wait(bars + C::kBarRes, 0u, ctl);
    }
  } else if (warp == kMmaWarp) {
    // the warp runs as one, with uniform operands; an elected thread issues the products
    if (work) {
      const uint32_t tm = static_cast<uint32_t>(uniform(static_cast<int>(ct.tmem)));
      const uint32_t m_s = tm, m_dp = tm + 128, m_dv = tm + 256, m_dk = tm + 384;
      const int n = uniform(n_blk);
      const uint64_t kd = smem_desc_kmajor(smem_u32(base + C::kOffA), 128);
      const uint64_t vd = smem_desc_kmajor(smem_u32(base + C::kOffB), 128);
      const uint64_t qd = smem_desc_kmajor(smem_u32(base + C::kOffE), 128);
      const uint64_t od = smem_desc_kmajor(smem_u32(base + C::kOffF), 128);
      const uint64_t qm = smem_desc_mn_sw128(smem_u32(base + C::kOffE), kChunkBytes, 1024u);
      const uint64_t om = smem_desc_mn_sw128(smem_u32(base + C::kOffF), kChunkBytes, 1024u);
      constexpr uint64_t kT = C::kTile >> 4;
      bool alive = true;
      auto wait = [&](int bar, uint32_t parity) { alive = alive && mbar_spin_warp(bars + bar, parity, ctl); };
      Ring e(C::kE), o(C::kF);  // e: the coming block's Q; o: this block's dO
      auto scores = [&](const Ring& r) {
        wait(C::kBarE + r.at, r.phase);
        tc_fence_after();
        if (elect_one()) {
          if (alive) product_abt<X, D>(m_s, kd, qd + static_cast<uint64_t>(r.at) * kT);
          umma_commit(bars + C::kBarS);
        }
        __syncwarp();
      };
      auto dprob = [&](const Ring& r) {
        wait(C::kBarF + r.at, r.phase);
        tc_fence_after();
        if (elect_one()) {
          if (alive) product_abt<X, D>(m_dp, vd, od + static_cast<uint64_t>(r.at) * kT);
          umma_commit(bars + C::kBarDp);
        }
        __syncwarp();
      };
      wait(C::kBarRes, 0u);
      scores(e);
      dprob(o);
      for (int i = 0; i < n; ++i) {
        const int q_at = e.at, o_at = o.at;
        e.next();
        o.next();
        wait(C::kBarP, static_cast<uint32_t>(i) & 1u);
        tc_fence_after();
        if (elect_one()) {
          if (alive) product_acc<X, D>(m_dv, m_s, om + static_cast<uint64_t>(o_at) * kT, i == 0);
          umma_commit(bars + C::kBarFreeF + o_at);
        }
        __syncwarp();
        if (i + 1 < n) scores(e);
        wait(C::kBarDs, static_cast<uint32_t>(i) & 1u);
        tc_fence_after();
        if (elect_one()) {
          if (alive) product_acc<X, D>(m_dk, m_dp, qm + static_cast<uint64_t>(q_at) * kT, i == 0);
          umma_commit(bars + C::kBarFreeE + q_at);
        }
        __syncwarp();
        if (i + 1 < n) dprob(o);
      }
      if (elect_one()) {
        umma_commit(bars + C::kBarAcc);
        umma_commit(bars + C::kBarDone);
      }
      __syncwarp();
      volatile uint32_t dummy = 0;
      const WaitCtl dctl{&dummy, ctl.limit_ns};
      mbar_wait(bars + C::kBarDone, 0u, dctl);
    }
  } else if (warp == kPrepWarp) {
    if (work) {
      for (int i = 0; i < n_blk; ++i) {
        const int b = i & 1, t0 = it.s.q0 + r_lo + i * f.tq;
        const int rows = (i == n_blk - 1 ? tail : f.tq) * a.g;
        float* st = reinterpret_cast<float*>(base + C::kOffStat) + b * 256;
        // all eight loads in flight before the buffer is waited for: one latency per block, off its path
        float l[4], de[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int r = u * 32 + static_cast<int>(lane), tok = r / a.g;
          const long long at = static_cast<long long>(t0 + tok) * a.Hq + hk * a.g + (r - tok * a.g);
          l[u] = -INFINITY;
          de[u] = 0.f;
          if (r < rows) {
            l[u] = __ldg(a.lse + at);
            de[u] = __ldg(a.delta + at);
          }
        }
        if (mbar_wait(bars + C::kBarStatFree + b, ((i >> 1) & 1u) ^ 1u, ctl)) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int r = u * 32 + static_cast<int>(lane);
            const bool none = l[u] == -INFINITY;
            st[r] = none ? -INFINITY : -l[u] * 1.4426950408889634f;
            st[128 + r] = none ? 0.f : de[u];
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + C::kBarStat + b);
        if (i == n_blk - 1 && tail < f.tq) {
          for (int x = 0; x < 2; ++x) {  // Q, dO
            const int at = i % (x ? C::kF : C::kE);
            if (mbar_wait(bars + C::kBarLast + x, 0u, ctl))
              clear_tile_rows<D>(base + (x ? C::kOffF : C::kOffE) + at * C::kTile, rows, static_cast<int>(lane), 32);
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars + (x ? C::kBarF : C::kBarE) + at);
          }
        }
      }
    }
  } else if (warp < kEpiWarps) {
    const int hf = warp >> 2, key = (warp & 3) * 32 + static_cast<int>(lane);
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = t_s + lane_off + 64 * hf, tp = t_dp + lane_off + 64 * hf;
    const float2 c2 = make_float2(f.c, f.c);
    // the first token (relative to r_lo) that sees this key, as a row; and the first that sees all keys
    const int first_row = a.causal ? (j0 + key - (it.s.lk - lq) - r_lo) * a.g : 0;
    const int all_rows = a.causal ? (j0 + n_key - 1 - (it.s.lk - lq) - r_lo) * a.g : 0;
    bool ok = true;
    for (int i = 0; i < n_blk; ++i) {
      const int b = i & 1;
      const float4* st4 = reinterpret_cast<const float4*>(base + C::kOffStat + b * 1024) + 16 * hf;
      ok = ok && mbar_wait(bars + C::kBarStat + b, (i >> 1) & 1u, ctl);
      ok = ok && mbar_wait(bars + C::kBarS, static_cast<uint32_t>(i) & 1u, ctl);
      tc_fence_after();
      float p[2][32];
      if (ok) {
        tmem_ld32_start(ts, p[0]);
        tmem_ld32_start(ts + 32, p[1]);
        tmem_wait32(p[0]);
        tmem_wait32(p[1]);
        if (i * rows_blk < all_rows) {
          const int skip = first_row - i * rows_blk - 64 * hf;  // columns before the first row that sees this key
#pragma unroll
          for (int u = 0; u < 64; ++u)
            if (u < skip) p[u >> 5][u & 31] = -INFINITY;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[16];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const float4 nl = st4[8 * h + u];
            float* x = p[h] + 4 * u;
            const float2 e0 = ffma2(make_float2(x[0], x[1]), c2, make_float2(nl.x, nl.y));
            const float2 e1 = ffma2(make_float2(x[2], x[3]), c2, make_float2(nl.z, nl.w));
            x[0] = exp2_approx(e0.x);
            x[1] = exp2_approx(e0.y);
            x[2] = exp2_approx(e1.x);
            x[3] = exp2_approx(e1.y);
            pk[2 * u] = pack_pair<X>(x[0], x[1]);
            pk[2 * u + 1] = pack_pair<X>(x[2], x[3]);
          }
          tmem_st16(ts + 16 * h, pk);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + C::kBarP);
      ok = ok && mbar_wait(bars + C::kBarDp, static_cast<uint32_t>(i) & 1u, ctl);
      tc_fence_after();
      if (ok) {
        float d[2][32];
        tmem_ld32_start(tp, d[0]);
        tmem_ld32_start(tp + 32, d[1]);
        tmem_wait32(d[0]);
        tmem_wait32(d[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[16];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const float4 de = st4[32 + 8 * h + u];
            const float* x = p[h] + 4 * u;
            const float* y = d[h] + 4 * u;
            const float2 a0 = fmul2(make_float2(x[0], x[1]), fadd2(make_float2(y[0], y[1]), make_float2(-de.x, -de.y)));
            const float2 a1 = fmul2(make_float2(x[2], x[3]), fadd2(make_float2(y[2], y[3]), make_float2(-de.z, -de.w)));
            pk[2 * u] = pack_pair<X>(a0.x, a0.y);
            pk[2 * u + 1] = pack_pair<X>(a1.x, a1.y);
          }
          tmem_st16(tp + 16 * h, pk);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bars + C::kBarDs);
        mbar_arrive(bars + C::kBarStatFree + b);
      }
    }
    // output: the first four warps dv, the others dk
    if (work) {
      ok = ok && mbar_wait(bars + C::kBarAcc, 0u, ctl);
      tc_fence_after();
    }
    const bool write = key < it.t1 - it.t0;
    const long long at = (static_cast<long long>(it.t0 + key) * a.Hk + hk) * D;
    // keys the sequence does not hold (past k_len, or outside every sequence) get zeros
    const float fac = hf == 0 ? 1.f : a.scale;
    store_lane<X, D>((hf == 0 ? t_dv : t_dk) + lane_off, fac, static_cast<X*>(hf == 0 ? a.dv : a.dk) + at, work && ok,
                     write && key < n_key);
    if (write && key >= n_key) {
      uint4* d4 = reinterpret_cast<uint4*>(static_cast<X*>(hf == 0 ? a.dv : a.dk) + at);
      for (int u = 0; u < D / 8; ++u) d4[u] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (work && warp == kMmaWarp) tmem_dealloc(ct.tmem, 512);
}

// ----------------------------------------------------------------- dq
template <typename X, int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_dq_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_do,
                   const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                   const BwdArgs f) {
  using C = BwdCfg<D>;
  extern __shared__ __align__(1024) uint8_t base[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + C::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + C::kOffMisc);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(base + C::kOffMisc + 4);
  RowItem* item = reinterpret_cast<RowItem*>(base + C::kOffMisc + 16);
  const AttnParams& a = f.a;
  const int warp = threadIdx.x / 32;
  const uint32_t lane = lane_id();
  const int hk = static_cast<int>(blockIdx.x % a.Hk);

  if (warp == kMmaWarp) {
    const RowItem it = find_row_item(a, f.tq, f.nb, f.nb + a.N - static_cast<int>(blockIdx.x / a.Hk));
    if (lane == 0) *item = it;
    if (blockIdx.x == 0)
      for (int i = static_cast<int>(lane); i < a.N; i += 32) seq_extent(a, i);
  }
  if (threadIdx.x == 0) {
    init_barriers<D>(bars);
    if ((smem_u32(base) & 1023u) != 0u) record_error(kErrDevice);  // the swizzled tiles would be misread
    *abort_flag = 0u;
  }
  __syncthreads();
  const RowItem it = *item;
  if (it.t0 >= it.t1) return;
  const int n_tok = min(f.tq, it.t1 - it.t0);
  const int top = (keys_seen(a, it.s, it.t0 + n_tok - 1 - it.s.q0) + 127) >> 7;  // key tiles
  const bool work = top > 0;
  if (work && warp == kMmaWarp) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const Cta<D> ct{base, bars, WaitCtl{abort_flag, f.wait_ns}, work ? *tmem_slot : 0u};
  const uint32_t t_s = ct.tmem, t_dp = ct.tmem + 128, t_dq = ct.tmem + 384;  // two dP buffers
  const WaitCtl& ctl = ct.ctl;
  const bool fix = top * 128 > it.s.lk;  // the last tile reaches past the sequence's keys

  if (warp == kTmaWarp) {
    if (work && lane == 0) {
      const uint64_t first = l2_policy_evict_first(), last = l2_policy_evict_last();
      mbar_arrive_expect_tx(bars + C::kBarRes, static_cast<uint32_t>(f.tq * a.g) * 256u * (D / 64));
      for (int ch = 0; ch < D / 64; ++ch) {
        tma_load_4d_hint(base + C::kOffA + ch * kChunkBytes, &tmap_q, bars + C::kBarRes, ch * 64, 0, it.t0, hk, first);
        tma_load_4d_hint(base + C::kOffB + ch * kChunkBytes, &tmap_do, bars + C::kBarRes, ch * 64, 0, it.t0, hk, first);
      }
      Ring k(C::kE), v(C::kF);
      for (int j = 0; j < top; ++j) {
        const bool cut = j == top - 1 && fix;
        load_ring<D>(base, C::kOffE, bars + C::kBarE, bars + C::kBarFreeE, cut ? bars + C::kBarLast : nullptr, k, &tmap_k,
                     false, it.s.k0 + j * 128, hk, C::kTile, last, ctl);
        load_ring<D>(base, C::kOffF, bars + C::kBarF, bars + C::kBarFreeF, cut ? bars + C::kBarLast + 1 : nullptr, v,
                     &tmap_v, false, it.s.k0 + j * 128, hk, C::kTile, last, ctl);
        k.next();
        v.next();
      }
      drain_ring(bars + C::kBarE, C::kE, top, ctl);
      drain_ring(bars + C::kBarF, C::kF, top, ctl);
      mbar_wait(bars + C::kBarRes, 0u, ctl);
    }
  } else if (warp == kMmaWarp) {
    // the warp runs as one, with uniform operands; an elected thread issues the products
    if (work) {
      const uint32_t tm = static_cast<uint32_t>(uniform(static_cast<int>(ct.tmem)));
      const int n = uniform(top);
      const uint64_t qd = smem_desc_kmajor(smem_u32(base + C::kOffA), 128);
      const uint64_t od = smem_desc_kmajor(smem_u32(base + C::kOffB), 128);
      const uint64_t kd = smem_desc_kmajor(smem_u32(base + C::kOffE), 128);
      const uint64_t vd = smem_desc_kmajor(smem_u32(base + C::kOffF), 128);
      const uint64_t km = smem_desc_mn_sw128(smem_u32(base + C::kOffE), kChunkBytes, 1024u);
      constexpr uint64_t kT = C::kTile >> 4;
      bool alive = true;
      auto wait = [&](int bar, uint32_t parity) { alive = alive && mbar_spin_warp(bars + bar, parity, ctl); };
      Ring k(C::kE), v(C::kF);
      int free_at = 0;
      auto scores = [&](int j) {  // S(j) and dP(j); dS(j-2), whose buffer this is, went into dQ before
        wait(C::kBarE + k.at, k.phase);
        tc_fence_after();
        if (elect_one()) {
          if (alive) product_abt<X, D>(tm, qd, kd + static_cast<uint64_t>(k.at) * kT);
          umma_commit(bars + C::kBarS);
        }
        __syncwarp();
        wait(C::kBarF + v.at, v.phase);
        tc_fence_after();
        if (elect_one()) {
          if (alive) product_abt<X, D>(tm + 128 + 128 * (j & 1), od, vd + static_cast<uint64_t>(v.at) * kT);
          umma_commit(bars + C::kBarDp + (j & 1));
          umma_commit(bars + C::kBarFreeF + v.at);
        }
        __syncwarp();
        k.next();
        v.next();
      };
      wait(C::kBarRes, 0u);
      scores(0);
      for (int j = 0; j < n; ++j) {
        if (j + 1 < n) {
          wait(C::kBarP, static_cast<uint32_t>(j) & 1u);  // S(j) is in registers
          scores(j + 1);
        }
        wait(C::kBarDs + (j & 1), static_cast<uint32_t>(j >> 1) & 1u);
        tc_fence_after();
        if (elect_one()) {
          if (alive)
            product_acc<X, D>(tm + 384, tm + 128 + 128 * (j & 1), km + static_cast<uint64_t>(free_at) * kT, j == 0);
          umma_commit(bars + C::kBarFreeE + free_at);
        }
        __syncwarp();
        if (++free_at == C::kE) free_at = 0;
      }
      if (elect_one()) {
        umma_commit(bars + C::kBarAcc);
        umma_commit(bars + C::kBarDone);
      }
      __syncwarp();
      volatile uint32_t dummy = 0;
      const WaitCtl dctl{&dummy, ctl.limit_ns};
      mbar_wait(bars + C::kBarDone, 0u, dctl);
    }
  } else if (warp == kPrepWarp) {
    if (work && fix) {
      const int j = top - 1;
      for (int x = 0; x < 2; ++x) {  // K, V
        const int at = j % (x ? C::kF : C::kE);
        if (mbar_wait(bars + C::kBarLast + x, 0u, ctl))
          clear_tile_rows<D>(base + (x ? C::kOffF : C::kOffE) + at * C::kTile, it.s.lk - j * 128,
                             static_cast<int>(lane), 32);
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + (x ? C::kBarF : C::kBarE) + at);
      }
    }
  } else if (warp < kEpiWarps) {
    const int hf = warp >> 2, row = (warp & 3) * 32 + static_cast<int>(lane);
    const int tok = row / a.g, head = row - tok * a.g;
    const bool row_ok = tok < n_tok;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = t_s + lane_off + 64 * hf;
    const long long at = static_cast<long long>(it.t0 + tok) * a.Hq + hk * a.g + head;
    float nl = -INFINITY, de = 0.f;
    if (row_ok) {
      const float l = a.lse[at];
      if (l != -INFINITY) {
        nl = -l * 1.4426950408889634f;
        de = a.delta[at];
      }
    }
    const int see = row_ok ? keys_seen(a, it.s, it.t0 + tok - it.s.q0) : 0;
    const int see_all = keys_seen(a, it.s, it.t0 - it.s.q0);
    const float2 c2 = make_float2(f.c, f.c), nl2 = make_float2(nl, nl), nd2 = make_float2(-de, -de);
    bool ok = true;
    for (int j = 0; j < top; ++j) {
      ok = ok && mbar_wait(bars + C::kBarS, static_cast<uint32_t>(j) & 1u, ctl);
      tc_fence_after();
      float p[2][32];
      if (ok) {
        tmem_ld32_start(ts, p[0]);
        tmem_ld32_start(ts + 32, p[1]);
        tmem_wait32(p[0]);
        tmem_wait32(p[1]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + C::kBarP);
      if (ok) {
        if ((j + 1) * 128 > see_all) {
          const int lim = see - j * 128 - 64 * hf;
#pragma unroll
          for (int u = 0; u < 64; ++u)
            if (u >= lim) p[u >> 5][u & 31] = -INFINITY;
        }
#pragma unroll
        for (int u = 0; u < 32; ++u) {
          float* x = p[u >> 4] + 2 * (u & 15);
          const float2 e = ffma2(make_float2(x[0], x[1]), c2, nl2);
          x[0] = exp2_approx(e.x);
          x[1] = exp2_approx(e.y);
        }
      }
      ok = ok && mbar_wait(bars + C::kBarDp + (j & 1), static_cast<uint32_t>(j >> 1) & 1u, ctl);
      tc_fence_after();
      if (ok) {
        const uint32_t tp = t_dp + 128 * (j & 1) + lane_off + 64 * hf;
        float d[2][32];
        tmem_ld32_start(tp, d[0]);
        tmem_ld32_start(tp + 32, d[1]);
        tmem_wait32(d[0]);
        tmem_wait32(d[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[16];
#pragma unroll
          for (int u = 0; u < 16; ++u) {
            const float2 y = fadd2(make_float2(d[h][2 * u], d[h][2 * u + 1]), nd2);
            const float2 z = fmul2(make_float2(p[h][2 * u], p[h][2 * u + 1]), y);
            pk[u] = pack_pair<X>(z.x, z.y);
          }
          tmem_st16(tp + 16 * h, pk);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + C::kBarDs + (j & 1));
    }
    if (work) {
      ok = ok && mbar_wait(bars + C::kBarAcc, 0u, ctl);
      tc_fence_after();
    }
    // output: each half of the warps takes half of the columns; rows that see nothing get zeros
    const bool none = nl == -INFINITY;
    X* dst = static_cast<X*>(a.dq) + at * D + (D / 2) * hf;
    store_lane<X, D / 2>(t_dq + lane_off + (D / 2) * hf, none ? 0.f : a.scale, dst, work && ok, row_ok && !none);
    if (row_ok && none) {
      uint4* d4 = reinterpret_cast<uint4*>(dst);
      for (int u = 0; u < D / 16; ++u) d4[u] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (work && warp == kMmaWarp) tmem_dealloc(ct.tmem, 512);
}

// ----------------------------------------------------------------- launches
template <typename X, int D>
cudaError_t run(const AttnParams& p, cudaStream_t stream) {
  using C = BwdCfg<D>;
  BwdArgs f;
  f.a = p;
  f.tq = 128 / p.g;
  f.c = p.scale * 1.4426950408889634f;
  f.wait_ns = kAttnWaitNs;
  static_assert(C::kOffA % 1024 == 0 && C::kTile % 1024 == 0, "swizzled tiles start on 1024 bytes");
  cudaError_t e;
  if ((e = smem_limit_once<attn_dq_kernel<X, D>>(C::kSmem)) != cudaSuccess) return e;
  if ((e = smem_limit_once<attn_dkv_kernel<X, D>>(C::kSmem)) != cudaSuccess) return e;
  CUtensorMap tq, to, tk, tv;
  if (p.Tq > 0) {
    if (!make_rows_map(&tq, p, p.q, p.q_st, p.q_sh, f.tq) ||
        !make_rows_map(&to, p, p.dout, static_cast<long long>(p.Hq) * D, D, f.tq))
      return cudaErrorInvalidValue;
    if (!make_keys_map(&tk, p, p.k, p.k_st, p.k_sh) || !make_keys_map(&tv, p, p.v, p.v_st, p.v_sh))
      return cudaErrorInvalidValue;
    const long long rows = static_cast<long long>(p.Tq) * p.Hq;
    constexpr int PER = 256 / (D / 8);
    attn_delta_kernel<X, D><<<static_cast<unsigned>((rows + PER - 1) / PER), 256, 0, stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (p.Tk > 0) {
    // without any query row nothing is seen: the maps describe rows that nothing loads
    if (p.Tq == 0) {
      const size_t n = static_cast<size_t>(p.Tk) * p.Hk * D * sizeof(X);
      if ((e = cudaMemsetAsync(p.dk, 0, n, stream)) != cudaSuccess) return e;
      return cudaMemsetAsync(p.dv, 0, n, stream);
    }
    f.nb = static_cast<int>((static_cast<long long>(p.Tk) + 127) / 128);
    const long long grid = (static_cast<long long>(f.nb) + p.N + 1) * p.Hk;
    if (grid > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    attn_dkv_kernel<X, D><<<static_cast<unsigned>(grid), kThreads, C::kSmem, stream>>>(tq, to, tk, tv, f);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  f.nb = static_cast<int>((static_cast<long long>(p.Tq) + f.tq - 1) / f.tq);
  const long long grid = (static_cast<long long>(f.nb) + p.N + 1) * p.Hk;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  attn_dq_kernel<X, D><<<static_cast<unsigned>(grid), kThreads, C::kSmem, stream>>>(tq, to, tk, tv, f);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_backward(const AttnParams& p, int dtype, cudaStream_t s) {
  if (dtype == CSA_BF16) return p.D == 128 ? run<__nv_bfloat16, 128>(p, s) : run<__nv_bfloat16, 64>(p, s);
  return p.D == 128 ? run<__half, 128>(p, s) : run<__half, 64>(p, s);
}

cudaError_t take_status_attn_bwd(uint32_t* out, cudaStream_t stream) { return take_status(out, stream); }

}  // namespace csa
