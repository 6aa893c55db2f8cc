// csa_attn_bwd.cu -- gradients of causal attention over packed sequences on
// the tensor cores.
//
//   delta = dout.out  (per row and head)
//   p_j = exp(s_j - lse),  ds_j = p_j (dout.v_j - delta)
//   dq = scale sum_j ds_j k_j,  dk_j = scale sum_rows ds_j q,  dv_j = sum_rows p_j dout
//
// Three kernels: delta (one pass over dout and out; fp16: and v), dq, and dk with dv.  The
// scores are formed again from q, k and lse in both of the latter; P and dS
// never leave the SM.  That is seven products per tile where one kernel
// for everything needs five, but every output is summed by one CTA in a fixed
// order: no atomics (the same bits on every call), no fp32 dq in memory, and
// dk, dv of a key head sum over its g query heads in place.
//
//   attn_dkv_kernel  an item is up to 128 keys of one sequence and key head; a
//     CTA walks the rows that see them in blocks of 128 (rows = token * g +
//     head, as in the forward):
//       S^T = K Q^T, dP^T = V dO^T           (operands in shared memory)
//       P^T, dS^T in the storage type over S^T, dP^T in TMEM
//       dV += P^T dO, dK += dS^T Q           (A in TMEM, B read MN-major)
//     TMEM: S^T, dP^T, dV, dK, 128 columns each.  The issue order dV(i),
//     S^T(i+1), dK(i), dP^T(i+1) leaves the elementwise warps the time of two
//     products for each of their two halves.
//   attn_dq_kernel   an item is a block of 128 rows; a CTA walks the key tiles:
//       S = Q K^T, dP = dO V^T               (Q, dO in TMEM, K, V in shared memory)
//       dS over dP in TMEM, dQ += dS K
//     TMEM: S, dP, dQ, 128 columns each, Q and dO, 64 each.  Issue order
//     S(j+1), dQ(j), dP(j+1).
//
// Warps (12): 0-7 elementwise (TMEM lanes 32 (w % 4) .., column half w / 4) and
// output; 8 issuer of the products; 9 TMA producer; 10 row statistics of the
// coming block (dkv) and what must be cleared in a tile's end; 11 items (as in
// the forward: the next one is taken from the grid while this one runs).
//
// A tile's end that belongs to another sequence may hold NaN, which a zero
// factor does not cancel: rows (dkv) or keys (dq) past the end are cleared in
// shared memory before any product reads them: such a tile lands on a barrier
// of its own, and the warp that cleared its end completes the tile's in the ring.
//
// fp16 holds neither dS of a scaled loss's cotangent (p (dP - delta) passes 65504
// where the gradients do not) nor that of a small one.  |dP - delta| is at most
// 2 |dout_r| max_j |v_j|: dS is formed times a power of two that brings this bound
// to 2^15, and dq and dk are taken back in fp32.  dq has a power for each row, dk,
// which sums over rows, one for each sequence and key head: nothing of another
// sequence has a part in it.  P^T, at most 1, is formed 2^15 times its size for dv
// (weights down to 2^-40 count, 2^-25 as they come).  attn_range_kernel takes the norms and delta in one
// pass (56 us for delta's 42 at the size below); bf16 has the range and none of this.
//
// Measured (bf16, 64 + 8 heads of 128, 8192 tokens in 5 documents): 0.83 to 0.85
// ms, 1025 TFLOP/s of the five products that count, 1435 of the seven executed (a
// library product: 1885).  dkv 0.410 ms, tensor pipe active 79 %: the products;
// dq 0.370 ms, 62 %: dP has one buffer, so that the next dP waits until dS of this
// tile has been formed and read; delta 0.042 ms, 6.4 TB/s.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "csa_attn_internal.h"
#include "csa_attn_tiles.cuh"

namespace csa {
namespace {

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8, kMmaWarp = 8, kTmaWarp = 9, kPrepWarp = 10, kItemWarp = 11;

struct BwdArgs {
  AttnParams a;
  int tq;  // tokens per block of 128 rows
  int nb;  // dq: ceil(Tq / tq); dkv: ceil(Tk / 128)
  float c;
  unsigned long long wait_ns;
  const int32_t* order;  // dkv: runs of keys by falling work, or null
  int n_split;           // dkv: shares of the rows of a run of keys
  float *part_dk, *part_dv;  // n_split > 1: their sums, [n_split][Tk * Hk][D]
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
                       kBarLast = kBarFreeF + kF, kBarStat = kBarLast + kE + kF, kBarStatFree = kBarStat + 2,
                       kBarS = kBarStatFree + 2, kBarP = kBarS + 1, kBarDp = kBarP + 1, kBarDs = kBarDp + 1,
                       kBarAcc = kBarDs + 1, kBarResFree = kBarAcc + 1, kBarCopied = kBarResFree + 1,
                       kBarItem = kBarCopied + 1, kBarItemFree = kBarItem + 2, kBarNext = kBarItemFree + 2,
                       kBarSoon = kBarNext + 1, kBarMeet = kBarSoon + 1, kBarDone = kBarMeet + 4, kBars = kBarDone + 1;
  static constexpr uint32_t kOffMisc = (kOffBar + 8 * kBars + 15) / 16 * 16, kOffItem = kOffMisc + 32;
  static constexpr uint32_t kSmem = kOffItem + 2 * 64;
};
static_assert(BwdCfg<128>::kSmem <= 227 * 1024, "shared memory");

// One item: a run of rows (dq) or keys (dkv) of one sequence (or outside all
// of them), and one key head.
struct BwdItem {
  SeqExt s;
  int t0, t1;  // rows or keys; t0 >= t1: no more items
  int hk;
  int n;       // steps: key tiles (dq) or blocks of rows (dkv)
  int lo;      // dkv: first block of this share
  int z;       // dkv: share
  int own;     // tokens (dq) or keys of the sequence (dkv) among t0 .. t1-1
  int r_lo;    // dkv: first row that sees a key of the run
  float fit;   // fp16: dq: the largest |v|^2 of the sequence; dkv: the power of two of dP - delta
};
static_assert(sizeof(BwdItem) <= 64, "a slot");

template <int D>
__device__ __forceinline__ void init_barriers(uint64_t* bars) {
  using C = BwdCfg<D>;
  for (int i = 0; i < C::kBars; ++i) {
    int n = 1;
    if (i == C::kBarStatFree || i == C::kBarStatFree + 1 || i == C::kBarP || i == C::kBarDs || i == C::kBarCopied)
      n = kEpiWarps;
    if (i >= C::kBarMeet && i < C::kBarMeet + 4) n = 2;
    if (i == C::kBarItemFree || i == C::kBarItemFree + 1) n = kEpiWarps + 3;  // + issuer, producer, preparer
    mbar_init(bars + i, n);
  }
  fence_mbar_init();
}

// What every role of a CTA uses: barriers, slots of items, the wait limit.
template <int D>
struct Cta {
  using C = BwdCfg<D>;
  uint8_t* base;
  uint64_t* bars;
  WaitCtl ctl;
  uint32_t n_item;  // items this role has taken

  // The role's next item, its until give() by one thread of each of its warps; null after the last one.
  __device__ const volatile BwdItem* next() {
    const uint32_t sl = n_item & 1u;
    if (!mbar_wait(bars + C::kBarItem + sl, (n_item >> 1) & 1u, ctl)) return nullptr;
    const volatile BwdItem* it = reinterpret_cast<const volatile BwdItem*>(base + C::kOffItem + 64 * sl);
    return it->t0 < it->t1 ? it : nullptr;
  }
  // A whole warp.
  __device__ void give() {
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(bars + C::kBarItemFree + (n_item & 1u));
    ++n_item;
  }
};

// The warp that prepares items, one ahead of the other roles; `make(id)` is
// the item of block `id`.
template <int D, typename F>
__device__ __forceinline__ void run_items(const Cta<D>& ct, F make) {
  using C = BwdCfg<D>;
  const uint32_t lane = lane_id();
  uint8_t* answer = ct.base + C::kOffMisc;
  uint32_t id = blockIdx.x, n = 0, asked = 0;
  bool more = true;
  while (more) {
    const BwdItem it = make(id);
    if (it.t0 < it.t1) {  // two borders may fall together: nothing between them
      const uint32_t sl = n & 1u;
      if (lane == 0) *reinterpret_cast<BwdItem*>(ct.base + C::kOffItem + 64 * sl) = it;
      __syncwarp();
      if (lane == 0) mbar_arrive(ct.bars + C::kBarItem + sl);
      ++n;
      // Another one is asked for when the copies of this one have all been started, two or three tiles before its
      // end: an item that a CTA holds ahead is one that no idle CTA can take.
      more = mbar_wait(ct.bars + C::kBarSoon, (n - 1u) & 1u, ct.ctl) &&
             mbar_wait(ct.bars + C::kBarItemFree + (n & 1u), ((n >> 1) & 1u) ^ 1u, ct.ctl);
    }
    if (!more) break;
    if (lane == 0) request_next(answer, ct.bars + C::kBarNext);
    volatile uint32_t dummy = 0;  // the answer is waited for even when a role gave up: it writes shared memory
    const WaitCtl dctl{&dummy, ct.ctl.limit_ns};
    const bool got = mbar_wait(ct.bars + C::kBarNext, asked & 1u, dctl);
    ++asked;
    more = got && answer_next(answer, id);
  }
  if (*ct.ctl.abort_flag == 0u) {
    const uint32_t sl = n & 1u;
    mbar_wait(ct.bars + C::kBarItemFree + sl, ((n >> 1) & 1u) ^ 1u, ct.ctl);
    if (lane == 0) reinterpret_cast<BwdItem*>(ct.base + C::kOffItem + 64 * sl)->t1 = INT32_MIN;
    __syncwarp();
    if (lane == 0) mbar_arrive(ct.bars + C::kBarItem + sl);
  }
}

// S^T or dP^T of one tile: D[128,128] = A . B^T, both K-major over D.
template <typename X, int D>
__device__ __forceinline__ void product_abt(uint32_t d, uint64_t ad, uint64_t bd) {
  constexpr uint32_t kId = idesc_f16<X>(128, 128, false);
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    const uint64_t o = static_cast<uint64_t>(((ks >> 2) * kChunkBytes + (ks & 3) * 32) >> 4);
    umma_bf16(d, ad + o, bd + o, kId, ks != 0 ? 1u : 0u);
  }
}
// The same with A (bf16 or fp16 pairs, D/2 columns) in TMEM.
template <typename X, int D>
__device__ __forceinline__ void product_tbt(uint32_t d, uint32_t a, uint64_t bd) {
  constexpr uint32_t kId = idesc_f16<X>(128, 128, false);
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    const uint64_t o = static_cast<uint64_t>(((ks >> 2) * kChunkBytes + (ks & 3) * 32) >> 4);
    umma_bf16_tmem_a(d, a + 8u * ks, bd + o, kId, ks != 0 ? 1u : 0u);
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

// fp16: 2 |dout| |v| < 2^E for the squares of the two norms.
__device__ __forceinline__ int ds_exponent(float dout2, float v2) {
  const int e = static_cast<int>((__float_as_uint(2.f * sqrtf(dout2 * v2)) >> 23) & 255u) - 126;
  return min(max(e, -60), 60);
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// The power of two of P^T (dkv).
template <typename X>
constexpr int kProbExp = is_bf16<X>() ? 0 : 15;

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

// Waits until no copy of the producer is in flight: the rings' (stages of E, then of F) and the n_res resident pairs.
template <int D>
__device__ __forceinline__ void drain_copies(uint64_t* bars, const Copies& copies, uint32_t n_res, const WaitCtl& ctl) {
  using C = BwdCfg<D>;
  volatile uint32_t dummy = 0;  // also when a role gave up
  const WaitCtl dctl{&dummy, ctl.limit_ns};
  copies.drain([&](int st, bool mend, uint32_t parity) { mbar_wait(bars + (mend ? C::kBarLast : C::kBarE) + st, parity, dctl); });
  if (n_res > 0) mbar_wait(bars + C::kBarRes, (n_res - 1u) & 1u, dctl);
}

// Copies tile i of a ring (rows: a block of query rows; else 128 keys).  A tile
// whose end has to be cleared lands on the stage's barrier in `last` instead
// (null: none to clear).  Several such tiles may be on their way at once.
template <int D>
__device__ __forceinline__ void load_ring(uint8_t* base, uint32_t off, uint64_t* full, uint64_t* free, uint64_t* last,
                                          const Ring& r, Copies& copies, int stage0, const CUtensorMap* map, bool rows,
                                          int at, int hk, uint32_t bytes, uint64_t pol, const WaitCtl& ctl) {
  constexpr uint32_t kTile = kChunkBytes * (D / 64);
  if (!mbar_wait(free + r.at, r.phase ^ 1u, ctl)) return;
  uint64_t* bar = (last != nullptr ? last : full) + r.at;
  uint8_t* dst = base + off + r.at * kTile;
  copies.start(stage0 + r.at, last != nullptr, r.phase);
  mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
  for (int ch = 0; ch < D / 64; ++ch) {
    if (rows)
      tma_load_4d_hint(dst + ch * kChunkBytes, map, bar, ch * 64, 0, at, hk, pol);
    else
      tma_load_3d_hint(dst + ch * kChunkBytes, map, bar, ch * 64, at, hk, pol);
  }
}

// Accumulator columns t .. t + N-1 of this thread's lane, times f, to N values
// of X at row `at` of dst (element offset; -1: no row).  Lanes 4 i .. 4 i + 3
// exchange 16-byte pieces so that four lanes store 64 bytes of one row.
template <typename X, int N>
__device__ __forceinline__ void store_lanes(uint32_t t, float f, X* dst, long long at, bool some) {
  const uint32_t lane = lane_id();
  long long at4[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) at4[u] = __shfl_sync(0xffffffffu, at, (lane & ~3u) + u);
  // (not unrolled: this runs once per item, and its time is that of fetching its instructions)
#pragma unroll 1
  for (int i = 0; i < N / 32; ++i) {
    float o[32];
    __syncwarp();
    if (some) {
      tmem_ld32_start(t + 32 * i, o);
      tmem_wait32(o);
    }
#pragma unroll
    for (int u = 0; u < 32; ++u) o[u] = some && f != 0.f ? o[u] * f : 0.f;
    if constexpr (sizeof(X) == 4) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // 16 values: four pieces
        uint4 q[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          q[u] = make_uint4(__float_as_uint(o[16 * h + 4 * u]), __float_as_uint(o[16 * h + 4 * u + 1]),
                            __float_as_uint(o[16 * h + 4 * u + 2]), __float_as_uint(o[16 * h + 4 * u + 3]));
        transpose4(q, lane);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (at4[u] >= 0) reinterpret_cast<uint4*>(dst + at4[u] + 32 * i + 16 * h)[lane & 3] = q[u];
      }
    } else {
      uint4 q[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        q[u] = make_uint4(pack_pair<X>(o[8 * u], o[8 * u + 1]), pack_pair<X>(o[8 * u + 2], o[8 * u + 3]),
                          pack_pair<X>(o[8 * u + 4], o[8 * u + 5]), pack_pair<X>(o[8 * u + 6], o[8 * u + 7]));
      transpose4(q, lane);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (at4[u] >= 0) reinterpret_cast<uint4*>(dst + at4[u] + 32 * i)[lane & 3] = q[u];
    }
  }
}

// ----------------------------------------------------------------- delta
// Work of run x of keys: the blocks of rows that see it.
__device__ __forceinline__ int key_run_blocks(const AttnParams& a, const RowItem& r, int tq) {
  if (r.t0 >= r.t1) return 0;
  const int j0 = r.t0 - r.s.k0, lq = r.s.q1 - r.s.q0;
  const int own = max(0, min(r.t1 - r.t0, r.s.lk - j0));
  const int r_lo = own > 0 ? (a.causal ? min(lq, max(0, j0 - (r.s.lk - lq))) : 0) : lq;
  return (lq - r_lo + tq - 1) / tq;
}

constexpr int kClasses = 1024;
// order[] = the n runs of keys in classes of falling work (a counting sort by
// one block; within a class in no fixed order, which no result depends on).
// The longest run of a packed batch can take as long as a fair share of all
// the work, so it has to begin first.
__device__ void order_runs(const AttnParams& p, int32_t* order, int n, int nb, int tq) {
  __shared__ int count[kClasses];
  const int most = (p.Tq + tq - 1) / tq;
  auto cls = [&](int x) {
    const int w = key_run_blocks(p, find_item<true, false>(p, 128, nb, x), tq);
    return kClasses - 1 - static_cast<int>(static_cast<long long>(w) * (kClasses - 1) / max(most, 1));
  };
  for (int i = threadIdx.x; i < kClasses; i += blockDim.x) count[i] = 0;
  __syncthreads();
  for (int x = threadIdx.x; x < n; x += blockDim.x) atomicAdd(count + cls(x), 1);
  __syncthreads();
  if (threadIdx.x < 32) {  // exclusive sums: 32 classes a lane
    int s = 0;
    for (int i = 0; i < kClasses / 32; ++i) s += count[threadIdx.x * (kClasses / 32) + i];
    int before = s;
    for (int o = 1; o < 32; o *= 2) {
      const int y = __shfl_up_sync(0xffffffffu, before, o);
      if (static_cast<int>(threadIdx.x) >= o) before += y;
    }
    before -= s;
    for (int i = 0; i < kClasses / 32; ++i) {
      int& c = count[threadIdx.x * (kClasses / 32) + i];
      const int m = c;
      c = before;
      before += m;
    }
  }
  __syncthreads();
  for (int x = threadIdx.x; x < n; x += blockDim.x) order[atomicAdd(count + cls(x), 1)] = x;
}

// delta = dout.out: D/8 lanes per row and head, 16 bytes of each tensor a lane.
// Block 0 orders the runs of keys meanwhile, when asked to.
template <typename X, int D>
__global__ void __launch_bounds__(256, 8) attn_delta_kernel(const AttnParams p, int32_t* order, int n_runs, int nb, int tq) {
  constexpr int G = D / 8;
  if (order != nullptr && blockIdx.x == 0) {
    order_runs(p, order, n_runs, nb, tq);
    return;
  }
  const long long block = order != nullptr ? blockIdx.x - 1u : blockIdx.x;
  const long long r = block * (256 / G) + threadIdx.x / G;
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

// The same for fp16, with what dS can reach: the squares of the norms of dout's
// rows, and the largest of dout and of v for each sequence and key head.  A block
// takes a run of rows (or of keys, past `row_blocks`) of one sequence and key head
// and raises its maximum once: looked at for each row, the few words of a batch of
// long sequences took four times as long as the values.
template <typename X, int D>
__global__ void __launch_bounds__(256, 4)
    attn_range_kernel(const AttnParams p, int32_t* order, int n_runs, int nb_k, int nb_q, int tq, unsigned row_blocks) {
  constexpr int G = D / 8, PER = 256 / G, U = 4;
  __shared__ uint32_t most;
  if (order != nullptr && blockIdx.x == 0) {
    order_runs(p, order, n_runs, nb_k, tq);
    return;
  }
  unsigned block = order != nullptr ? blockIdx.x - 1u : blockIdx.x;
  const bool values = block >= row_blocks;
  if (values) block -= row_blocks;
  const int x = static_cast<int>(block / static_cast<unsigned>(p.Hk)), hk = static_cast<int>(block % static_cast<unsigned>(p.Hk));
  const RowItem it = values ? find_key_item(p, 128, nb_k, x) : find_row_item(p, tq, nb_q, x);
  if (it.seq < 0 || it.t0 >= it.t1) return;  // the same for the whole block
  if (threadIdx.x == 0) most = 0u;
  __syncthreads();
  const int l = threadIdx.x % G;
  // keys past k_len are not the sequence's
  const int rows = values ? max(0, min(it.t1 - it.t0, it.s.lk - (it.t0 - it.s.k0))) : (it.t1 - it.t0) * p.g;
  float top = 0.f;
  for (int r0 = threadIdx.x / G; r0 < 128; r0 += U * PER) {
    uint4 a[U], b[U];
    long long at[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * PER, tok = values ? r : r / p.g;
      a[u] = b[u] = make_uint4(0u, 0u, 0u, 0u);
      at[u] = static_cast<long long>(it.t0 + tok) * p.Hq + hk * p.g + (r - tok * p.g);
      if (r >= rows) continue;
      if (values) {
        a[u] = reinterpret_cast<const uint4*>(static_cast<const X*>(p.v) + (it.t0 + tok) * p.v_st + hk * p.v_sh)[l];
      } else {
        a[u] = reinterpret_cast<const uint4*>(static_cast<const X*>(p.dout) + at[u] * D)[l];
        b[u] = reinterpret_cast<const uint4*>(static_cast<const X*>(p.out) + at[u] * D)[l];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t xs[4] = {a[u].x, a[u].y, a[u].z, a[u].w}, ys[4] = {b[u].x, b[u].y, b[u].z, b[u].w};
      float s = 0.f, n2 = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = unpack_pair<X>(xs[i]), w = unpack_pair<X>(ys[i]);
        s = fmaf(v.x, w.x, s);
        s = fmaf(v.y, w.y, s);
        n2 = fmaf(v.x, v.x, fmaf(v.y, v.y, n2));
      }
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        n2 += __shfl_xor_sync(0xffffffffu, n2, o);
      }
      if (l == 0 && !values && r0 + u * PER < rows) {
        p.delta[at[u]] = s;
        p.norm2[at[u]] = n2;
      }
      top = fmaxf(top, n2);
    }
  }
  // not negative: ordered as their bits
  if (l == 0) atomicMax(&most, __float_as_uint(top));
  __syncthreads();
  if (threadIdx.x == 0) atomicMax(p.range + (static_cast<long long>(it.seq) * p.Hk + hk) * 2 + values, most);
}

// dk, dv = the sums of the shares, in order: D/4 threads per key and key head.
template <typename X, int D>
__global__ void __launch_bounds__(256) attn_join_dkv_kernel(const AttnParams a, const float* part_dk, const float* part_dv,
                                                            int n_split) {
  constexpr int PER = 256 / (D / 4);
  const long long rows = static_cast<long long>(a.Tk) * a.Hk;
  const long long r = static_cast<long long>(blockIdx.x) * PER + threadIdx.x / (D / 4);
  const int l = threadIdx.x % (D / 4);
  if (r >= rows) return;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const float* part = x ? part_dv : part_dk;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int z = 0; z < n_split; ++z) {
      const float4 v = reinterpret_cast<const float4*>(part + (z * rows + r) * D)[l];
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    uint2 u;
    u.x = pack_pair<X>(s.x, s.y);
    u.y = pack_pair<X>(s.z, s.w);
    reinterpret_cast<uint2*>(static_cast<X*>(x ? a.dv : a.dk) + r * D)[l] = u;
  }
}

// ----------------------------------------------------------------- dk, dv
#define CSA_BWD_SETUP                                                                                          \
  using C = BwdCfg<D>;                                                                                         \
  extern __shared__ __align__(1024) uint8_t base[];                                                            \
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + C::kOffBar);                                             \
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + C::kOffMisc + 16);                                  \
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(base + C::kOffMisc + 20);               \
  const AttnParams& a = f.a;                                                                                   \
  const int warp = threadIdx.x / 32;                                                                           \
  const uint32_t lane = lane_id();                                                                             \
  if (threadIdx.x == 0) {                                                                                      \
    init_barriers<D>(bars);                                                                                    \
    if ((smem_u32(base) & 1023u) != 0u) record_error(kErrDevice); /* the swizzled tiles would be misread */    \
    *abort_flag = 0u;                                                                                          \
  }                                                                                                            \
  if (warp == kTmaWarp && lane == 0) {                                                                         \
    prefetch_tmap(&tmap_q);                                                                                    \
    prefetch_tmap(&tmap_do);                                                                                   \
    prefetch_tmap(&tmap_k);                                                                                    \
    prefetch_tmap(&tmap_v);                                                                                    \
  }                                                                                                            \
  if (warp == kMmaWarp) {                                                                                      \
    tmem_alloc(tmem_slot, 512);                                                                                \
    tmem_relinquish();                                                                                         \
  }

// SPLIT: the items are shares of a run's rows, and their sums go to the workspace.
template <typename X, int D, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    attn_dkv_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_do,
                    const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                    const BwdArgs f) {
  CSA_BWD_SETUP
  const int rows_blk = f.tq * a.g;  // rows of a full block (128 when g divides it)
  if (rows_blk < 128)               // rows that no copy writes: zero factors must meet finite values
    for (int s = 0; s < C::kE + C::kF; ++s)
      clear_tile_rows<D>(base + C::kOffE + s * C::kTile, rows_blk, static_cast<int>(threadIdx.x), kThreads);
  fence_proxy_async_shared();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot, t_s = tmem, t_dp = tmem + 128, t_dv = tmem + 256, t_dk = tmem + 384;
  const WaitCtl ctl{abort_flag, f.wait_ns};
  Cta<D> ct{base, bars, ctl, 0u};

  if (warp == kItemWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (blockIdx.x == 0)
      for (int i = static_cast<int>(lane); i < a.N; i += 32) seq_extent(a, i);
    run_items<D>(ct, [&](uint32_t id) {
      BwdItem it;
      const uint32_t rest = id / static_cast<uint32_t>(a.Hk);
      it.hk = static_cast<int>(id - rest * static_cast<uint32_t>(a.Hk));
      const uint32_t x = rest / static_cast<uint32_t>(f.n_split);
      it.z = static_cast<int>(rest - x * static_cast<uint32_t>(f.n_split));
      const RowItem r = find_key_item(a, 128, f.nb, f.order != nullptr ? f.order[x] : static_cast<int>(x));
      it.s = r.s;
      it.t0 = r.t0;
      it.t1 = r.t1;
      const int j0 = r.t0 - r.s.k0, lq = r.s.q1 - r.s.q0;
      it.own = max(0, min(r.t1 - r.t0, r.s.lk - j0));
      it.r_lo = it.own > 0 ? (a.causal ? min(lq, max(0, j0 - (r.s.lk - lq))) : 0) : lq;
      // blocks lo .. lo + n - 1 of all that see the run
      const int all = key_run_blocks(a, r, f.tq), share = (all + f.n_split - 1) / f.n_split;
      it.lo = min(all, it.z * share);
      it.n = min(all, it.lo + share) - it.lo;
      it.fit = 1.f;
      if (!is_bf16<X>() && r.seq >= 0) {
        const uint32_t* m = a.range + (static_cast<long long>(r.seq) * a.Hk + it.hk) * 2;
        it.fit = power_of_two(15 - kProbExp<X> - ds_exponent(__uint_as_float(m[0]), __uint_as_float(m[1])));
      }
      return it;
    });
  } else if (warp == kTmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    const uint64_t first = l2_policy_evict_first(), last = l2_policy_evict_last();
    Ring e(C::kE), o(C::kF);
    const uint32_t bytes = static_cast<uint32_t>(rows_blk) * 128u * (D / 64);
    uint32_t n_res = 0;
    Copies copies;
    while (const volatile BwdItem* it = ct.next()) {
      const int n = it->n, hk = it->hk, t0 = it->t0, q0 = it->s.q0 + it->r_lo + it->lo * f.tq, rows = it->s.q1 - q0;
      ct.give();
      if (lane == 0 && n > 0) {
        const bool cut = rows < n * f.tq;  // the last block is not full
        if (mbar_wait(bars + C::kBarResFree, (n_res & 1u) ^ 1u, ctl)) {
          ++n_res;
          mbar_arrive_expect_tx(bars + C::kBarRes, 2 * C::kTile);
          for (int ch = 0; ch < D / 64; ++ch) {
            tma_load_3d_hint(base + C::kOffA + ch * kChunkBytes, &tmap_k, bars + C::kBarRes, ch * 64, t0, hk, first);
            tma_load_3d_hint(base + C::kOffB + ch * kChunkBytes, &tmap_v, bars + C::kBarRes, ch * 64, t0, hk, first);
          }
        }
        for (int i = 0; i < n; ++i) {
          const bool c = cut && i == n - 1;
          load_ring<D>(base, C::kOffE, bars + C::kBarE, bars + C::kBarFreeE, c ? bars + C::kBarLast : nullptr, e, copies, 0,
                       &tmap_q, true, q0 + i * f.tq, hk, bytes, last, ctl);
          load_ring<D>(base, C::kOffF, bars + C::kBarF, bars + C::kBarFreeF, c ? bars + C::kBarLast + C::kE : nullptr, o,
                       copies, C::kE, &tmap_do, true, q0 + i * f.tq, hk, bytes, last, ctl);
          e.next();
          o.next();
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + C::kBarSoon);
    }
    if (lane == 0) drain_copies<D>(bars, copies, n_res, ctl);
  } else if (warp == kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    // the warp runs as one, with uniform operands; an elected thread issues the products
    const uint32_t tm = static_cast<uint32_t>(uniform(static_cast<int>(tmem)));
    const uint32_t m_s = tm, m_dp = tm + 128, m_dv = tm + 256, m_dk = tm + 384;
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
    uint32_t step = 0, res = 0;  // parities of P and dS, of the resident tiles
    auto scores = [&](const Ring& r) {
      wait(C::kBarE + r.at, r.phase);
      tc_fence_after();
      if (elect_one()) {
        if (alive) product_abt<X, D>(m_s, kd, qd + static_cast<uint64_t>(r.at) * kT);
        umma_commit(bars + C::kBarS);
      }
      __syncwarp();
    };
    auto dprob = [&](const Ring& r, bool last) {
      wait(C::kBarF + r.at, r.phase);
      tc_fence_after();
      if (elect_one()) {
        if (alive) product_abt<X, D>(m_dp, vd, od + static_cast<uint64_t>(r.at) * kT);
        umma_commit(bars + C::kBarDp);
        if (last) umma_commit(bars + C::kBarResFree);  // the last product with K and V
      }
      __syncwarp();
    };
    while (const volatile BwdItem* it = ct.next()) {
      const int n = uniform(it->n);
      ct.give();
      if (n == 0) continue;
      wait(C::kBarRes, res);
      res ^= 1u;
      scores(e);
      dprob(o, n == 1);
      for (int i = 0; i < n; ++i, step ^= 1u) {
        const int q_at = e.at, o_at = o.at;
        e.next();
        o.next();
        wait(C::kBarP, step);
        tc_fence_after();
        if (elect_one()) {
          if (alive) product_acc<X, D>(m_dv, m_s, om + static_cast<uint64_t>(o_at) * kT, i == 0);
          umma_commit(bars + C::kBarFreeF + o_at);
        }
        __syncwarp();
        if (i + 1 < n) scores(e);
        wait(C::kBarDs, step);
        tc_fence_after();
        if (elect_one()) {
          if (alive) product_acc<X, D>(m_dk, m_dp, qm + static_cast<uint64_t>(q_at) * kT, i == 0);
          umma_commit(bars + C::kBarFreeE + q_at);
          if (i + 1 == n) umma_commit(bars + C::kBarAcc);
        }
        __syncwarp();
        if (i + 1 < n) dprob(o, i + 2 == n);
      }
    }
    if (elect_one()) umma_commit(bars + C::kBarDone);
    __syncwarp();
    volatile uint32_t dummy = 0;
    const WaitCtl dctl{&dummy, ctl.limit_ns};
    mbar_wait(bars + C::kBarDone, 0u, dctl);
  } else if (warp == kPrepWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    uint32_t blk = 0, last_par = 0;  // blocks so far; parities of the stages' barriers of cut blocks
    Ring e(C::kE), o(C::kF);
    while (const volatile BwdItem* it = ct.next()) {
      const int n = it->n, hk = it->hk, q0 = it->s.q0 + it->r_lo + it->lo * f.tq, all = it->s.q1 - q0;
      const float fit = is_bf16<X>() ? 1.f : it->fit;
      for (int i = 0; i < n; ++i, ++blk) {
        const uint32_t b = blk & 1u;
        const int t0 = q0 + i * f.tq, rows = min(f.tq, all - i * f.tq) * a.g;
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
        if (mbar_wait(bars + C::kBarStatFree + b, ((blk >> 1) & 1u) ^ 1u, ctl)) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int r = u * 32 + static_cast<int>(lane);
            const bool none = l[u] == -INFINITY;
            st[r] = none ? -INFINITY : -l[u] * 1.4426950408889634f + static_cast<float>(kProbExp<X>);
            st[128 + r] = none ? 0.f : is_bf16<X>() ? de[u] : de[u] * fit;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + C::kBarStat + b);
        if (i == n - 1 && all < n * f.tq) {
          for (int x = 0; x < 2; ++x) {  // Q, dO
            const int at = x ? o.at : e.at, bit = x ? C::kE + at : at;
            if (mbar_wait(bars + C::kBarLast + bit, (last_par >> bit) & 1u, ctl))
              clear_tile_rows<D>(base + (x ? C::kOffF : C::kOffE) + at * C::kTile, rows, static_cast<int>(lane), 32);
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars + (x ? C::kBarF : C::kBarE) + at);
            last_par ^= 1u << bit;
          }
        }
        e.next();
        o.next();
      }
      ct.give();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const int hf = warp >> 2, key = (warp & 3) * 32 + static_cast<int>(lane);
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = t_s + lane_off + 64 * hf, tp = t_dp + lane_off + 64 * hf;
    const float2 c2 = make_float2(f.c, f.c);
    uint32_t blk = 0, acc = 0;
    bool ok = true;
    while (const volatile BwdItem* it = ct.next()) {
      const int n = it->n;
      int first_row, all_rows;  // the first row (from the share's first on) that sees this key; that sees all keys
      {
        // in tokens, and clamped there: a key far before the first row is seen from it on, and the distance times the
        // heads need not fit 32 bits
        const int d = max(it->t0 - it->s.k0 - (it->s.lk - (it->s.q1 - it->s.q0)), -128) - it->r_lo - it->lo * f.tq;
        first_row = a.causal ? max(0, d + key) * a.g : 0;
        all_rows = a.causal ? max(0, d + it->own - 1) * a.g : 0;
      }
      const float fit = is_bf16<X>() ? 1.f : it->fit;
      // dP - delta, for fp16 times the item's power of two (delta comes with it)
      auto less_delta = [&](float2 dp, float2 de) {
        return is_bf16<X>() ? fadd2(dp, make_float2(-de.x, -de.y))
                            : ffma2(dp, make_float2(fit, fit), make_float2(-de.x, -de.y));
      };
      for (int i = 0; i < n; ++i, ++blk) {
        const uint32_t b = blk & 1u;
        // (loads in program order: hoisted ones would take the registers of the scores)
        const uint32_t st4 = smem_u32(base + C::kOffStat) + b * 1024u + 256u * hf;
        ok = ok && mbar_wait(bars + C::kBarStat + b, (blk >> 1) & 1u, ctl);
        ok = ok && mbar_wait(bars + C::kBarS, blk & 1u, ctl);
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
            for (int h = 0; h < 2; ++h) {
              const uint32_t drop = low_bits(skip - 32 * h);
#pragma unroll
              for (int u = 0; u < 32; ++u)
                if ((drop & (1u << u)) != 0u) p[h][u] = -INFINITY;
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t pk[16];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const float4 nl = lds_f4(st4 + 16u * (8 * h + u));
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
        ok = ok && mbar_wait(bars + C::kBarDp, blk & 1u, ctl);
        tc_fence_after();
        if (ok) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float d[32];  // dS goes over columns that were read: 16 h .. of 32 (h + 1)
            tmem_ld32_start(tp + 32 * h, d);
            tmem_wait32(d);
            uint32_t pk[16];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const float4 de = lds_f4(st4 + 512u + 16u * (8 * h + u));
              const float* x = p[h] + 4 * u;
              const float* y = d + 4 * u;
              const float2 a0 = fmul2(make_float2(x[0], x[1]), less_delta(make_float2(y[0], y[1]), make_float2(de.x, de.y)));
              const float2 a1 = fmul2(make_float2(x[2], x[3]), less_delta(make_float2(y[2], y[3]), make_float2(de.z, de.w)));
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
      // output: the first four warps dv, the others dk; keys the sequence does not hold (past k_len, or outside
      // every sequence) get zeros
      if (n > 0) {
        ok = ok && mbar_wait(bars + C::kBarAcc, acc, ctl);
        acc ^= 1u;
        tc_fence_after();
      }
      const int t0 = it->t0;
      const long long at = key < it->t1 - t0 ? (static_cast<long long>(t0 + key) * a.Hk + it->hk) * D : -1;
      const float fac = key < it->own ? (hf == 0 ? 1.f : is_bf16<X>() ? a.scale : a.scale / fit) * (1.f / (1 << kProbExp<X>)) : 0.f;
      const uint32_t src = (hf == 0 ? t_dv : t_dk) + lane_off;
      if constexpr (SPLIT)
        store_lanes<float, D>(src, fac, (hf == 0 ? f.part_dv : f.part_dk) + it->z * (static_cast<long long>(a.Tk) * a.Hk * D),
                              at, n > 0 && ok);
      else
        store_lanes<X, D>(src, fac, static_cast<X*>(hf == 0 ? a.dv : a.dk), at, n > 0 && ok);
      tc_fence_before();
      ct.give();
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// ----------------------------------------------------------------- dq
template <typename X, int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_dq_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_do,
                   const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                   const BwdArgs f) {
  CSA_BWD_SETUP
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t t_s = tmem, t_dp = tmem + 128, t_dq = tmem + 256, t_q = tmem + 384, t_do = tmem + 448;
  const WaitCtl ctl{abort_flag, f.wait_ns};
  Cta<D> ct{base, bars, ctl, 0u};

  if (warp == kItemWarp) {
    reg_shrink();
    if (blockIdx.x == 0)
      for (int i = static_cast<int>(lane); i < a.N; i += 32) seq_extent(a, i);
    run_items<D>(ct, [&](uint32_t id) {
      BwdItem it;
      const uint32_t x = id / static_cast<uint32_t>(a.Hk);
      it.hk = static_cast<int>(id - x * static_cast<uint32_t>(a.Hk));
      const RowItem r = find_row_item(a, f.tq, f.nb, f.nb + a.N - static_cast<int>(x));
      it.s = r.s;
      it.t0 = r.t0;
      it.t1 = r.t1;
      it.own = min(f.tq, r.t1 - r.t0);
      it.n = it.own > 0 ? (keys_seen(a, r.s, r.t0 + it.own - 1 - r.s.q0) + 127) >> 7 : 0;
      it.r_lo = it.lo = it.z = 0;
      it.fit = 0.f;
      if (!is_bf16<X>() && r.seq >= 0) it.fit = __uint_as_float(a.range[(static_cast<long long>(r.seq) * a.Hk + it.hk) * 2 + 1]);
      return it;
    });
  } else if (warp == kTmaWarp) {
    reg_shrink();
    const uint64_t first = l2_policy_evict_first(), last = l2_policy_evict_last();
    Ring k(C::kE), v(C::kF);
    uint32_t n_res = 0;
    Copies copies;
    while (const volatile BwdItem* it = ct.next()) {
      const int n = it->n, hk = it->hk, t0 = it->t0, k0 = it->s.k0, lk = it->s.lk;
      ct.give();
      if (lane == 0 && n > 0) {
        if (mbar_wait(bars + C::kBarResFree, (n_res & 1u) ^ 1u, ctl)) {
          ++n_res;
          mbar_arrive_expect_tx(bars + C::kBarRes, static_cast<uint32_t>(f.tq * a.g) * 256u * (D / 64));
          for (int ch = 0; ch < D / 64; ++ch) {
            tma_load_4d_hint(base + C::kOffA + ch * kChunkBytes, &tmap_q, bars + C::kBarRes, ch * 64, 0, t0, hk, first);
            tma_load_4d_hint(base + C::kOffB + ch * kChunkBytes, &tmap_do, bars + C::kBarRes, ch * 64, 0, t0, hk, first);
          }
        }
        for (int j = 0; j < n; ++j) {
          const bool c = j == n - 1 && n * 128 > lk;  // the tile reaches past the sequence's keys
          load_ring<D>(base, C::kOffE, bars + C::kBarE, bars + C::kBarFreeE, c ? bars + C::kBarLast : nullptr, k, copies, 0,
                       &tmap_k, false, k0 + j * 128, hk, C::kTile, last, ctl);
          load_ring<D>(base, C::kOffF, bars + C::kBarF, bars + C::kBarFreeF, c ? bars + C::kBarLast + C::kE : nullptr, v,
                       copies, C::kE, &tmap_v, false, k0 + j * 128, hk, C::kTile, last, ctl);
          k.next();
          v.next();
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + C::kBarSoon);
    }
    if (lane == 0) drain_copies<D>(bars, copies, n_res, ctl);
  } else if (warp == kMmaWarp) {
    reg_shrink();
    const uint32_t tm = static_cast<uint32_t>(uniform(static_cast<int>(tmem)));
    const uint64_t kd = smem_desc_kmajor(smem_u32(base + C::kOffE), 128);
    const uint64_t vd = smem_desc_kmajor(smem_u32(base + C::kOffF), 128);
    const uint64_t km = smem_desc_mn_sw128(smem_u32(base + C::kOffE), kChunkBytes, 1024u);
    constexpr uint64_t kT = C::kTile >> 4;
    bool alive = true;
    auto wait = [&](int bar, uint32_t parity) { alive = alive && mbar_spin_warp(bars + bar, parity, ctl); };
    Ring k(C::kE), v(C::kF);
    uint32_t step = 0, cop = 0;
    auto scores = [&] {  // S = Q . K^T, Q in TMEM
      wait(C::kBarE + k.at, k.phase);
      tc_fence_after();
      if (elect_one()) {
        if (alive) product_tbt<X, D>(tm, tm + 384, kd + static_cast<uint64_t>(k.at) * kT);
        umma_commit(bars + C::kBarS);
      }
      __syncwarp();
    };
    auto dprob = [&] {  // dP = dO . V^T, dO in TMEM
      wait(C::kBarF + v.at, v.phase);
      tc_fence_after();
      if (elect_one()) {
        if (alive) product_tbt<X, D>(tm + 128, tm + 448, vd + static_cast<uint64_t>(v.at) * kT);
        umma_commit(bars + C::kBarDp);
        umma_commit(bars + C::kBarFreeF + v.at);
      }
      __syncwarp();
      v.next();
    };
    while (const volatile BwdItem* it = ct.next()) {
      const int n = uniform(it->n);
      ct.give();
      if (n == 0) continue;
      wait(C::kBarCopied, cop);
      cop ^= 1u;
      scores();
      dprob();
      for (int j = 0; j < n; ++j, step ^= 1u) {
        const int at = k.at;
        k.next();
        if (j + 1 < n) {
          wait(C::kBarP, step);  // S(j) is in registers
          scores();
        }
        wait(C::kBarDs, step);
        tc_fence_after();
        if (elect_one()) {
          if (alive) product_acc<X, D>(tm + 256, tm + 128, km + static_cast<uint64_t>(at) * kT, j == 0);
          umma_commit(bars + C::kBarFreeE + at);
          if (j + 1 == n) umma_commit(bars + C::kBarAcc);
        }
        __syncwarp();
        if (j + 1 < n) dprob();
      }
    }
    if (elect_one()) umma_commit(bars + C::kBarDone);
    __syncwarp();
    volatile uint32_t dummy = 0;
    const WaitCtl dctl{&dummy, ctl.limit_ns};
    mbar_wait(bars + C::kBarDone, 0u, dctl);
  } else if (warp == kPrepWarp) {
    reg_shrink();
    uint32_t last_par = 0;
    int used = 0;
    while (const volatile BwdItem* it = ct.next()) {
      const int n = it->n, left = it->s.lk - (n - 1) * 128;  // keys of the sequence in the last tile
      ct.give();
      used += n;
      if (n == 0 || left >= 128) continue;
      for (int x = 0; x < 2; ++x) {  // K, V
        const int at = (used - 1) % (x ? C::kF : C::kE), bit = x ? C::kE + at : at;
        if (mbar_wait(bars + C::kBarLast + bit, (last_par >> bit) & 1u, ctl))
          clear_tile_rows<D>(base + (x ? C::kOffF : C::kOffE) + at * C::kTile, left, static_cast<int>(lane), 32);
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + (x ? C::kBarF : C::kBarE) + at);
        last_par ^= 1u << bit;
      }
    }
  } else {
    reg_grow<2>();
    const int hf = warp >> 2, row = (warp & 3) * 32 + static_cast<int>(lane);
    const int tok = row / a.g, head = row - tok * a.g;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = t_s + lane_off + 64 * hf, tp = t_dp + lane_off + 64 * hf;
    const float2 c2 = make_float2(f.c, f.c);
    uint32_t step = 0, item = 0, met = 0;
    bool ok = true;
    while (const volatile BwdItem* it = ct.next()) {
      const int n = it->n;
      const bool row_ok = tok < it->own;
      const long long at = row_ok ? static_cast<long long>(it->t0 + tok) * a.Hq + it->hk * a.g + head : -1;
      float nl = -INFINITY, de = 0.f;
      int see = 0, see_all = 0, fit = 0;  // fit: exponent of the row's power of two
      if (n > 0) {
        if (row_ok) {
          const float l = a.lse[at], d = a.delta[at];
          if constexpr (!is_bf16<X>()) fit = 15 - ds_exponent(a.norm2[at], it->fit);
          if (l != -INFINITY) {
            nl = -l * 1.4426950408889634f;
            de = d;
          }
        }
        const SeqExt e{it->s.q0, it->s.q1, it->s.k0, it->s.lk};
        see_all = keys_seen(a, e, it->t0 - e.q0);
        if (row_ok) see = keys_seen(a, e, it->t0 + tok - e.q0);
        // Q and dO go to TMEM as A operands, one half of the warps each: their products then read shared memory
        // for K and V alone (both from there left the products waiting for it)
        ok = ok && mbar_wait(bars + C::kBarRes, item & 1u, ctl);
        const uint8_t* src = base + (hf == 0 ? C::kOffA : C::kOffB) + row * 128;
        const uint32_t dst = (hf == 0 ? t_q : t_do) + lane_off;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {  // 32 values: four 16-byte pieces of a swizzled row
          uint32_t w[16];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int piece = (4 * c + u) & 7;
            const uint4 q = *reinterpret_cast<const uint4*>(src + (c >> 1) * kChunkBytes + ((piece ^ (row & 7)) * 16));
            w[4 * u] = q.x;
            w[4 * u + 1] = q.y;
            w[4 * u + 2] = q.z;
            w[4 * u + 3] = q.w;
          }
          tmem_st16(dst + 16 * c, w);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + C::kBarCopied);
        ++item;
      }
      const float nf = is_bf16<X>() ? nl : nl + static_cast<float>(fit);
      const float2 nl2 = make_float2(nf, nf);
      float2 nd2 = make_float2(-de, -de);
      if (n == 1) {
        // All the keys these rows see are in one tile: delta = sum p dP, without the rounding of out that dout.out
        // has (and that shows where a row averages few values).  The dk, dv kernel uses it too.  The tile's scores
        // and dP are read once more below (in the loop itself this took registers from every tile).
        ok = ok && mbar_wait(bars + C::kBarS, step, ctl);
        ok = ok && mbar_wait(bars + C::kBarDp, step, ctl);
        tc_fence_after();
        float sum = 0.f;
        if (ok) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x[32], d[32];
            tmem_ld32_start(ts + 32 * h, x);
            tmem_ld32_start(tp + 32 * h, d);
            tmem_wait32(x);
            tmem_wait32(d);
#pragma unroll
            for (int u = 0; u < 32; ++u)
              if (64 * hf + 32 * h + u < see) sum = fmaf(exp2_approx(fmaf(x[u], f.c, nl)), d[u], sum);
          }
        }
        float* xch = reinterpret_cast<float*>(base + C::kOffStat) + row;
        xch[128 * hf] = sum;
        meet(bars + C::kBarMeet + (warp & 3), met, ctl);
        const float delta = xch[0] + xch[128];
        meet(bars + C::kBarMeet + (warp & 3), met, ctl);
        if (nl != -INFINITY) {
          nd2 = make_float2(-delta, -delta);
          if (hf == 0) a.delta[at] = delta;
        }
      }
      for (int j = 0; j < n; ++j, step ^= 1u) {
        ok = ok && mbar_wait(bars + C::kBarS, step, ctl);
        tc_fence_after();
        // Q and dO are in TMEM once the first scores stand: their tiles are free for the next item
        if (j == 0 && threadIdx.x == 0) mbar_arrive(bars + C::kBarResFree);
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
            for (int h = 0; h < 2; ++h) {
              const uint32_t keep = low_bits(lim - 32 * h);
#pragma unroll
              for (int u = 0; u < 32; ++u)
                if ((keep & (1u << u)) == 0u) p[h][u] = -INFINITY;
            }
          }
#pragma unroll
          for (int u = 0; u < 32; ++u) {
            float* x = p[u >> 4] + 2 * (u & 15);
            const float2 e = ffma2(make_float2(x[0], x[1]), c2, nl2);
            x[0] = exp2_approx(e.x);
            x[1] = exp2_approx(e.y);
          }
        }
        ok = ok && mbar_wait(bars + C::kBarDp, step, ctl);
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
        if (lane == 0) mbar_arrive(bars + C::kBarDs);
      }
      if (n > 0) {
        ok = ok && mbar_wait(bars + C::kBarAcc, (item - 1u) & 1u, ctl);
        tc_fence_after();
      }
      // output: each half of the warps takes half of the columns; rows that see nothing get zeros
      store_lanes<X, D / 2>(t_dq + lane_off + (D / 2) * hf,
                            nl == -INFINITY ? 0.f : is_bf16<X>() ? a.scale : a.scale * power_of_two(-fit),
                            static_cast<X*>(a.dq) + (D / 2) * hf, at >= 0 ? at * D : -1, n > 0 && ok);
      tc_fence_before();
      ct.give();
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}
#undef CSA_BWD_SETUP

// ----------------------------------------------------------------- launches
template <typename X, int D>
cudaError_t run(const AttnParams& p, const AttnBwdPlan& plan, uint8_t* ws, cudaStream_t stream) {
  using C = BwdCfg<D>;
  BwdArgs f;
  f.a = p;
  f.tq = 128 / p.g;
  f.c = p.scale * 1.4426950408889634f;
  f.n_split = plan.n_split;
  f.part_dk = reinterpret_cast<float*>(ws + plan.off_part);
  f.part_dv = f.part_dk + static_cast<long long>(plan.n_split) * p.Tk * p.Hk * D;
  int32_t* order = plan.ordered ? reinterpret_cast<int32_t*>(ws + plan.off_order) : nullptr;
  f.order = order;
  static_assert(C::kOffA % 1024 == 0 && C::kTile % 1024 == 0, "swizzled tiles start on 1024 bytes");
  cudaError_t e;
  if (p.Tq == 0) {  // nothing is seen
    const size_t n = static_cast<size_t>(p.Tk) * p.Hk * D * sizeof(X);
    if ((e = cudaMemsetAsync(p.dk, 0, n, stream)) != cudaSuccess) return e;
    return cudaMemsetAsync(p.dv, 0, n, stream);
  }
  if ((e = smem_limit_once<attn_dq_kernel<X, D>>(C::kSmem)) != cudaSuccess) return e;
  CUtensorMap tq, to, tk, tv;
  if (!make_rows_map(&tq, p, p.q, p.q_st, p.q_sh, f.tq) ||
      !make_rows_map(&to, p, p.dout, static_cast<long long>(p.Hq) * D, D, f.tq) ||
      !make_keys_map(&tk, p, p.k, p.k_st, p.k_sh) || !make_keys_map(&tv, p, p.v, p.v_st, p.v_sh))
    return cudaErrorInvalidValue;
  const int nb_k = static_cast<int>((static_cast<long long>(p.Tk) + 127) / 128);
  const int nb_q = static_cast<int>((static_cast<long long>(p.Tq) + f.tq - 1) / f.tq);
  const long long runs_k = static_cast<long long>(nb_k) + p.N + 1, runs_q = static_cast<long long>(nb_q) + p.N + 1;
  if (runs_k * p.Hk * plan.n_split > 0x7FFFFFFFll || runs_q * p.Hk > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  const long long rows = static_cast<long long>(p.Tq) * p.Hq;
  constexpr int PER = 256 / (D / 8);
  if constexpr (is_bf16<X>()) {
    attn_delta_kernel<X, D><<<static_cast<unsigned>((rows + PER - 1) / PER + (order != nullptr)), 256, 0, stream>>>(
        p, order, static_cast<int>(runs_k), nb_k, f.tq);
  } else {
    if (p.N > 0 && (e = cudaMemsetAsync(p.range, 0, static_cast<size_t>(p.N) * p.Hk * 8, stream)) != cudaSuccess) return e;
    const long long row_blocks = runs_q * p.Hk, blocks = (order != nullptr) + row_blocks + runs_k * p.Hk;
    if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    attn_range_kernel<X, D><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(
        p, order, static_cast<int>(runs_k), nb_k, nb_q, f.tq, static_cast<unsigned>(row_blocks));
  }
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // dq first: it improves delta for the rows of few keys
  f.nb = nb_q;
  f.wait_ns = attn_wait_ns(attn_steps_keys(p.Tk));
  attn_dq_kernel<X, D><<<static_cast<unsigned>(runs_q * p.Hk), kThreads, C::kSmem, stream>>>(tq, to, tk, tv, f);
  if ((e = cudaGetLastError()) != cudaSuccess || p.Tk == 0) return e;
  f.nb = nb_k;
  f.wait_ns = attn_wait_ns(attn_steps_rows(p.Tq, f.tq));
  const unsigned grid = static_cast<unsigned>(runs_k * p.Hk * plan.n_split);
  if (plan.n_split > 1) {
    if ((e = smem_limit_once<attn_dkv_kernel<X, D, true>>(C::kSmem)) != cudaSuccess) return e;
    attn_dkv_kernel<X, D, true><<<grid, kThreads, C::kSmem, stream>>>(tq, to, tk, tv, f);
  } else {
    if ((e = smem_limit_once<attn_dkv_kernel<X, D, false>>(C::kSmem)) != cudaSuccess) return e;
    attn_dkv_kernel<X, D, false><<<grid, kThreads, C::kSmem, stream>>>(tq, to, tk, tv, f);
  }
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (plan.n_split > 1) {
    const long long keys = static_cast<long long>(p.Tk) * p.Hk;
    constexpr int PER_J = 256 / (D / 4);
    attn_join_dkv_kernel<X, D><<<static_cast<unsigned>((keys + PER_J - 1) / PER_J), 256, 0, stream>>>(
        p, f.part_dk, f.part_dv, plan.n_split);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_backward(const AttnParams& p, int dtype, void* workspace, cudaStream_t s) {
  const AttnBwdPlan plan = attn_bwd_plan(p.N, p.Tq, p.Tk, p.Hq, p.Hk, p.D, dtype == CSA_F16);
  AttnParams a = p;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.delta = reinterpret_cast<float*>(ws);
  a.norm2 = reinterpret_cast<float*>(ws + plan.off_norm2);
  a.range = reinterpret_cast<uint32_t*>(ws + plan.off_range);
  if (dtype == CSA_BF16)
    return p.D == 128 ? run<__nv_bfloat16, 128>(a, plan, ws, s) : run<__nv_bfloat16, 64>(a, plan, ws, s);
  return p.D == 128 ? run<__half, 128>(a, plan, ws, s) : run<__half, 64>(a, plan, ws, s);
}

cudaError_t take_status_attn_bwd(uint32_t* out, cudaStream_t stream) { return take_status(out, stream); }

}  // namespace csa
