// csa_sparse_fwd.cu -- attention over listed blocks of keys on the tensor cores.
//
//   s_j = scale q.k_j over the keys that a row lists, out = sum_j p_j v_j with
//   p = softmax(s), lse = log sum_j exp(s_j).
//
// An item is one query row, one key head and one share of the row's list.  Its
// g = Hq/Hk query heads are the rows of the products, and its list's slots, 128
// at a time, their columns; a slot that names no visible key keeps its place, reads
// as zero and weighs nothing:
//   S = Q . K^T      (A = queries, B = key tile, both in shared memory, to TMEM)
//   P = 2^(c (S - m) + shift) in the storage type, c = scale log2(e), over S
//   O += P . V       (A = P in TMEM, B = value tile read MN-major, O in TMEM)
// The products have 128 rows and g is often less: the queries stand there R =
// 128 / G times (G: 32, 64 or 128 rows), and copy r takes the columns r 128/R
// .. of each tile; P is zero in its others.  So each thread has 128/R scores
// instead of one thread having all, each copy keeps its own reference m and sum
// l, and the copies' outputs are joined once per item.
//
// m is raised (and O, l rescaled) only when a tile's largest score is 2^kRaise
// above it; fp16 weights are formed 2^kShift times their size, so that they
// count down to 2^-32 of the reference's.
//
// Roles (20 warps, R = 1 and 2: 24, one CTA per SM, walking items blockIdx.x + n
// gridDim.x):
//   warps 0-3    softmax, one thread per row of S; R = 1 and 2: warps 20-23 have the
//                second half of a copy's columns, and the two exchange the tile's
//                largest score (64 columns in one thread: 1750 cycles a tile, a
//                prompt of 16384 tokens with 64 heads 515 us; in two: 500)
//   warps 4-7    outputs: join, division, stores, while the next item runs
//   warps 8-11   loads of the listed keys' rows (and, by TMA, of the queries)
//   warps 12-15  the same of the values' rows
//   warps 16-17  issuers of the products with keys and with values, a thread each
//   warps 18-19  lists: each writes the rows of every second tile, up to kRing tiles
//                ahead
// Rows are gathered by cp.async, 16 bytes a lane, into the layout that TMA would
// write: hidden keys are never read, what fills up a tile is zero.  (Four warps get
// 91 bytes a ns that way out of L2, four with TMA's gathered loads 41 to 55: those
// take 40 to 70 cycles each to issue.)
// Shared memory: two query blocks, two key and two value tiles.  TMEM: S0 S1 O0 O1.
//
// Measured (bf16, D 128): 16384 rows of 64 heads and one key head over 512 listed
// entries, 425 us (606 TFLOP/s of counted work, twice that with the copies of the
// queries); 8192 rows of 2 x 16 heads over 256 blocks of 4 keys and a window of 128,
// 688 us (13 TB/s out of L2; 16 heads of 128 rows count); one token of 64 sequences, 8
// key heads, 512 blocks of 4 of a cache of 32768, 97 us (5.9 TB/s of HBM, 88 % of a
// copy); one token, 131072 cached, 12 us with the join.  Prompts are bound by what
// a tile costs in instructions (schedulers busy 63 % of the time, tensor cores 41 %)
// and in meetings of the roles, 200 to 300 cycles each; wide blocks by the gathered
// rows out of L2.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstring>
#include <type_traits>

#include "csa_sparse_list.cuh"

namespace csa {
namespace {

template <typename X>
constexpr float kShift = is_bf16<X>() ? 0.f : 8.f;
constexpr float kRaise = 6.f;  // P stays below 2^(kShift + kRaise)

constexpr int kLists = 2;
constexpr int kOutWarp = 4, kKeyWarp = 8, kValueWarp = 12, kScoreWarp = 16, kMmaWarp = 17, kListWarp = 18, kHalfWarp = 20;
template <int R>
constexpr int kHalves = R == 4 ? 1 : 2;  // softmax threads of a row
template <int R>
constexpr int kThreads = 32 * (kHalfWarp + 4 * (kHalves<R> - 1));
constexpr int kPitch = 36;    // floats between two rows of staged outputs (32 columns)

template <int D>
struct Cfg {
  static constexpr uint32_t kTile = kChunkBytes * (D / 64);  // 128 rows x D
  static constexpr uint32_t kOffQ = 0, kOffK = 2 * kTile, kOffV = 4 * kTile, kOffOut = 6 * kTile;
  static constexpr uint32_t kOffRing = kOffOut + 128 * kPitch * 4;
  static constexpr uint32_t kOffMl = kOffRing + kRing * sizeof(Tile);  // [2][3][128] floats: m, l of two items (l by halves)
  static constexpr uint32_t kOffTop = kOffMl + 2 * 3 * 128 * 4;          // [2][2][128] floats: a tile's largest scores
  static constexpr uint32_t kOffItem = kOffTop + 2 * 2 * 128 * 4;          // [2] items whose outputs are to come
  static constexpr uint32_t kOffBar = kOffItem + 64;
  static constexpr int kBarQ = 0, kBarQFree = 2, kBarK = 4, kBarV = 6, kBarS = 8, kBarP = 10, kBarPv = 12, kBarO = 14,
                       kBarMl = 16, kBarOFree = 18, kBarTile = 20, kBarTileFree = kBarTile + kRing,
                       kBarMeet = kBarTileFree + kRing, kBarPair = kBarMeet + 1, kBarDone = kBarPair + 4, kBars = kBarDone + 1;
  static constexpr uint32_t kOffMisc = kOffBar + 8 * kBars, kSmem = kOffMisc + 16;
};
static_assert(Cfg<128>::kSmem <= 227 * 1024, "one CTA per SM");

struct FwdArgs {
  SparseParams p;
  ListArgs l;
  int n_split;      // shares of a row's list
  float c;          // scale * log2(e)
  float* part_o;    // [n_split][Tq * Hq][D] (n_split > 1)
  float* part_lse;  // [n_split][Tq * Hq]
  unsigned long long wait_ns;
};

template <typename X, int D, int R, bool SPLIT>
__global__ void __launch_bounds__(kThreads<R>, 1)
    sparse_fwd_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ FwdArgs f) {
  using C = Cfg<D>;
  constexpr int G = 128 / R, CW = 128 / R;  // rows of a copy of the queries; columns that a copy takes
  constexpr int H = kHalves<R>, TW = CW / H;  // columns of a softmax thread
  extern __shared__ __align__(1024) uint8_t base[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + C::kOffBar);
  Tile* ring = reinterpret_cast<Tile*>(base + C::kOffRing);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + C::kOffMisc);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(base + C::kOffMisc + 4);
  const SparseParams& p = f.p;
  const int warp = threadIdx.x / 32;
  const uint32_t lane = lane_id();

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kBars; ++i) {
      int n = 1;
      if (i >= C::kBarP && i < C::kBarP + 2) n = 4 * H;
      if (i >= C::kBarMl && i < C::kBarMl + 2) n = 4 * H;
      if (i >= C::kBarPair && i < C::kBarPair + 4) n = 2;
      if (i >= C::kBarOFree && i < C::kBarOFree + 2) n = 4;
      if (i >= C::kBarK && i < C::kBarV + 2) n = 128;  // every lane that loads
      if (i >= C::kBarTileFree && i < C::kBarTileFree + kRing) n = 10 + 4 * H;
      if (i == C::kBarDone) n = 2;
      if (i == C::kBarMeet) n = 4;
      mbar_init(bars + i, n);
    }
    if ((smem_u32(base) & 1023u) != 0u) record_error(kErrDevice);  // the swizzled tiles would be misread
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == kKeyWarp && lane == 0) prefetch_tmap(&tmap_q);
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl ctl{abort_flag, f.wait_ns};
  volatile uint32_t dummy = 0;
  const WaitCtl drain{&dummy, f.wait_ns};  // for what has to be waited for even when a role gave up
  // the next tile; n < 0 after the last one or a wait that gave up
  Place at(f.l);
  auto next_head = [&]() -> TileHead {
    if (at.left == 0 || !bar_wait(bars + C::kBarTile + at.slot, at.parity, ctl)) return TileHead{-1, 0, 0, 0, 0, 0, 0};
    return ring[at.slot].h;
  };
  auto give_head = [&] {  // by a role's warp
    __syncwarp();
    if (lane == 0) mbar_arrive(bars + C::kBarTileFree + at.slot);
    at.next();
  };

  if (warp >= kListWarp && warp < kHalfWarp) {
    const int w = warp - kListWarp;
    list_tiles<kLists>(p, f.l, w, ring, bars + C::kBarTile, bars + C::kBarTileFree, ctl);
  } else if (warp >= kKeyWarp && warp < kScoreWarp) {
    // ------------------------------------------------------------------------- rows of keys, of values
    const bool keys = warp < kValueWarp;
    const int r0 = 32 * (warp & 3);
    const GatherRows& rows = keys ? p.k : p.v;
    uint64_t* full = bars + (keys ? C::kBarK : C::kBarV);
    // a stage is free when the product that read it has completed
    uint64_t* used = bars + (keys ? C::kBarS : C::kBarPv);
    uint8_t* stages = base + (keys ? C::kOffK : C::kOffV);
    uint32_t j = 0, nq = 0;
    bool first = true;  // no tile of this item yet
    while (true) {
      const TileHead h = next_head();
      if (h.n < 0) break;
      if (h.n > 0) {
        if (warp == kKeyWarp && first) {
          const uint32_t b = nq & 1u;
          if (!bar_wait(bars + C::kBarQFree + b, ((nq >> 1) & 1u) ^ 1u, ctl)) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(bars + C::kBarQ + b, static_cast<uint32_t>(R * p.g) * 128u * (D / 64));
            const uint64_t q_pol = l2_policy_evict_first();
            for (int r = 0; r < R; ++r)
              for (int ch = 0; ch < D / 64; ++ch)
                tma_load_3d_hint(base + C::kOffQ + b * C::kTile + ch * kChunkBytes + r * (G * 128), &tmap_q,
                                 bars + C::kBarQ + b, ch * 64, h.hk * p.g, h.t, q_pol);
          }
          __syncwarp();
          ++nq;
        }
        first = false;
        const uint32_t st = j & 1u;
        if (!bar_wait(used + st, ((j >> 1) & 1u) ^ 1u, ctl)) break;
        load_rows<D, 32>(stages + st * C::kTile, rows, keys ? ring[at.slot].k_row : ring[at.slot].v_row, r0, (h.n + 15) & ~15);
        report_rows(full + st);
        ++j;
      }
      if (h.last) first = true;
      give_head();
    }
    wait_rows();  // no copy is in flight when the CTA ends, a role's giving up included
    for (uint32_t i = nq > 2 ? nq - 2 : 0; i < nq; ++i) bar_wait(bars + C::kBarQ + (i & 1u), (i >> 1) & 1u, drain);
  } else if (warp == kScoreWarp || warp == kMmaWarp) {
    // ------------------------------------------------------------------------- issuers of the products
    // Each warp runs as one (uniform operands), one elected thread issues.  Two of
    // them, so that neither's waits hold up the other's products: with one for both, a
    // tile took 2400 cycles of which the tensor cores had work for 1000.  (They do not
    // poll: that takes the issue slots of the warps beside them, 598 us for 500.)
    const uint32_t tm = static_cast<uint32_t>(uniform(static_cast<int>(tmem)));
    constexpr uint32_t kT = C::kTile >> 4;
    bool alive = true, first = true;
    auto wait = [&](int bar, uint32_t parity) { alive = alive && bar_wait(bars + bar, parity, ctl); };
    uint32_t j = 0;
    if (warp == kScoreWarp) {
      const uint64_t qd = smem_desc_kmajor(smem_u32(base + C::kOffQ), 128);
      const uint64_t kd = smem_desc_kmajor(smem_u32(base + C::kOffK), 128);
      constexpr uint32_t kIdS = idesc_f16<X>(128, 128, false);
      uint32_t nq = 0;
      while (alive) {
        const TileHead h = next_head();
        const int n = uniform(h.n), last = uniform(h.last);
        if (n < 0) break;
        give_head();
        if (n > 0) {
          const uint32_t st = j & 1u;
          if (first) wait(C::kBarQ + static_cast<int>(nq & 1u), (nq >> 1) & 1u);
          first = false;
          wait(C::kBarPv + static_cast<int>(st), ((j >> 1) & 1u) ^ 1u);  // P in this S has been used
          wait(C::kBarK + static_cast<int>(st), (j >> 1) & 1u);
          fence_proxy_async_shared();
          tc_fence_after();
          if (elect_one()) {
            if (alive) {
              const uint64_t q = qd + static_cast<uint64_t>((nq & 1u) * kT), k = kd + static_cast<uint64_t>(st * kT);
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks) {
                const uint64_t o = static_cast<uint64_t>(((ks >> 2) * kChunkBytes + (ks & 3) * 32) >> 4);
                umma_bf16(tm + st * 128u, q + o, k + o, kIdS, ks != 0 ? 1u : 0u);
              }
            }
            umma_commit(bars + C::kBarS + st);
          }
          __syncwarp();
          ++j;
        }
        if (last && !first) {
          if (elect_one()) umma_commit(bars + C::kBarQFree + (nq & 1u));
          __syncwarp();
          ++nq;
          first = true;
        }
      }
    } else {
      const uint64_t vd = smem_desc_mn_sw128(smem_u32(base + C::kOffV), kChunkBytes, 1024u);
      constexpr uint32_t kIdO = idesc_f16<X>(128, D, true);
      uint32_t on = 0;
      while (alive) {
        const TileHead h = next_head();
        const int n = uniform(h.n), last = uniform(h.last);
        if (n < 0) break;
        give_head();
        if (first && (n > 0 || last)) wait(C::kBarOFree + static_cast<int>(on & 1u), ((on >> 1) & 1u) ^ 1u);
        if (n > 0) {
          const uint32_t st = j & 1u;
          wait(C::kBarV + static_cast<int>(st), (j >> 1) & 1u);
          wait(C::kBarP + static_cast<int>(st), (j >> 1) & 1u);
          fence_proxy_async_shared();
          tc_fence_after();
          const int steps = (n + 15) >> 4;
          if (elect_one()) {
            if (alive) {
#pragma unroll
              for (int ks = 0; ks < 8; ++ks)
                if (ks < steps)
                  umma_bf16_tmem_a(tm + 256u + (on & 1u) * 128u, tm + st * 128u + 8u * ks,
                                   vd + static_cast<uint64_t>(st * kT) + static_cast<uint64_t>(128 * ks), kIdO,
                                   (!first || ks != 0) ? 1u : 0u);
            }
            umma_commit(bars + C::kBarPv + st);
          }
          __syncwarp();
          first = false;
          ++j;
        }
        if (last) {
          if (elect_one()) umma_commit(bars + C::kBarO + (on & 1u));
          __syncwarp();
          ++on;
          first = true;
        }
      }
    }
    if (elect_one()) umma_commit(bars + C::kBarDone);
    __syncwarp();
    bar_wait(bars + C::kBarDone, 0u, drain);
  } else if (warp < kOutWarp || warp >= kHalfWarp) {
    // ------------------------------------------------------------------------- softmax
    const int half = warp < kOutWarp ? 0 : 1, quarter = warp & 3;
    const int row = quarter * 32 + static_cast<int>(lane), copy = row / G, col0 = copy * CW + half * TW;
    const bool used = row % G < p.g;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    float* ml = reinterpret_cast<float*>(base + C::kOffMl);
    float* tops = reinterpret_cast<float*>(base + C::kOffTop);
    TileHead* done_items = reinterpret_cast<TileHead*>(base + C::kOffItem);
    const float c = f.c;
    uint32_t j = 0, on = 0, met = 0;
    auto meet_half = [&] {  // with the warp that has the other half of these rows
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + C::kBarPair + quarter);
      const bool here = bar_wait(bars + C::kBarPair + quarter, met, ctl);
      met ^= 1u;
      return here;
    };
    float m = -INFINITY, l = 0.f;
    bool ok = true, first = true;
    while (ok) {
      const TileHead h = next_head();
      if (h.n < 0) break;
      if (h.n > 0) {
        const uint32_t st = j & 1u;
        ok = bar_wait(bars + C::kBarS + st, (j >> 1) & 1u, ctl);
        if (!ok) break;
        tc_fence_after();
        const uint32_t ts = tmem + lanes + st * 128u;
        const uint32_t* keys = ring[at.slot].keys + col0 / 32;
        float s[32];
        auto load = [&](int i) {  // 32 scores, those of no key at -inf
          tmem_ld32_start(ts + col0 + 32 * i, s);
          const uint32_t see = keys[i];
          tmem_wait32(s);
          if (see != 0xffffffffu) {
#pragma unroll
            for (int u = 0; u < 32; ++u)
              if (((see >> u) & 1u) == 0u) s[u] = -INFINITY;
          }
        };
        // the tile's largest score (NaN is passed over)
        float top = -INFINITY;
#pragma unroll 1
        for (int i = 0; i < TW / 32; ++i) {
          load(i);
          float a = fmaxf(s[0], s[1]), b = fmaxf(s[2], s[3]);
#pragma unroll
          for (int u = 4; u < 32; u += 4) {
            a = max3(a, s[u], s[u + 1]);
            b = max3(b, s[u + 2], s[u + 3]);
          }
          top = max3(top, a, b);
        }
        if (!used) top = -INFINITY;  // no query: what stands there asks for nothing
        if constexpr (H == 2) {
          tops[st * 256 + half * 128 + row] = top;
          if (!(ok = meet_half())) break;
          top = fmaxf(top, tops[st * 256 + (half ^ 1) * 128 + row]);
        }
        if (first) {
          m = top;
          l = 0.f;
        } else if (__any_sync(0xffffffffu, top * c > m * c + kRaise)) {
          // the former tile's product with V has to be through before O is rescaled
          ok = bar_wait(bars + C::kBarPv + (st ^ 1u), ((j - 1) >> 1) & 1u, ctl);
          if (!ok) break;
          tc_fence_after();
          const float mn = fmaxf(m, top), r = mn == -INFINITY ? 1.f : exp2_approx((m - mn) * c);
          m = mn;
          l *= r;
          const uint32_t to = tmem + lanes + 256u + (on & 1u) * 128u;
#pragma unroll 1
          for (int i = half; i < D / 16; i += H) tmem_scale16(to + 16 * i, r);
        }
        const float ref = (m == -INFINITY ? 0.f : m) * c, bias = kShift<X> - ref;
        float2 sum = make_float2(0.f, 0.f);
        // P lies over S: of this thread's columns when they have been read; of the other half's, with which the
        // reads of the first half's second 32 columns would collide, after a second meeting
        uint32_t pk[TW / 32][16];
        auto weights = [&](int i) {
#pragma unroll
          for (int u = 0; u < 16; ++u) {
            const float2 e = ffma2(make_float2(s[2 * u], s[2 * u + 1]), make_float2(c, c), make_float2(bias, bias));
            const float2 w = make_float2(exp2_approx(e.x), exp2_approx(e.y));
            sum = fadd2(sum, w);
            pk[i][u] = pack_pair<X>(w.x, w.y);
          }
        };
        if constexpr (TW == 32) {
          weights(0);
        } else {
#pragma unroll
          for (int i = 0; i < TW / 32; ++i) {
            load(i);
            weights(i);
          }
          if (!(ok = meet_half())) break;
        }
#pragma unroll
        for (int i = 0; i < TW / 32; ++i) tmem_st16(ts + (col0 + 32 * i) / 2, pk[i]);
        l += sum.x + sum.y;
        if (R > 1) {  // the other copies' columns, as far as the product reads
          const uint32_t zero[16] = {};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (32 * i / CW != copy && 32 * i < h.n && i % H == half) tmem_st16(ts + 16 * i, zero);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + C::kBarP + st);
        first = false;
        ++j;
      }
      if (h.last) {
        ok = bar_wait(bars + C::kBarOFree + (on & 1u), ((on >> 1) & 1u) ^ 1u, ctl);
        float* mine = ml + (on & 1u) * 384;
        if (half == 0) mine[row] = m;
        if (threadIdx.x == 0) done_items[on & 1u] = h;
        mine[128 + half * 128 + row] = l;
        m = -INFINITY;
        l = 0.f;
        first = true;
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + C::kBarMl + (on & 1u));
        ++on;
      }
      give_head();
    }
  } else {
    // ------------------------------------------------------------------------- outputs
    const int w = warp - kOutWarp, row = w * 32 + static_cast<int>(lane), head = row % G, tid = row;
    float* stage = reinterpret_cast<float*>(base + C::kOffOut);
    const float* ml = reinterpret_cast<const float*>(base + C::kOffMl);
    const long long rows = static_cast<long long>(p.Tq) * p.Hq;
    uint32_t on = 0, met = 0;
    auto all_here = [&] {  // a meeting of these four warps, bounded as every wait is
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + C::kBarMeet);
      bar_wait(bars + C::kBarMeet, met, ctl);
      met ^= 1u;
    };
    for (long long left = item_count(f.l); left > 0; --left) {
      {
        const uint32_t b = on & 1u;
        if (!bar_wait(bars + C::kBarMl + b, (on >> 1) & 1u, ctl) || !bar_wait(bars + C::kBarO + b, (on >> 1) & 1u, ctl)) break;
        const TileHead h = reinterpret_cast<const TileHead*>(base + C::kOffItem)[b];
        tc_fence_after();
        const float* mm = ml + b * 384;
        float top = -INFINITY, l = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) top = fmaxf(top, mm[r * G + head]);
        const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int r = 0; r < R; ++r)
          l += (mm[128 + r * G + head] + (H == 2 ? mm[256 + r * G + head] : 0.f)) * exp2_approx((mm[r * G + head] - ref) * f.c);
        const bool seen = l > 0.f || l != l;
        const float weight = seen ? exp2_approx((mm[row] - ref) * f.c) / l : 0.f;
        const long long at = static_cast<long long>(h.t) * p.Hq + static_cast<long long>(h.hk) * p.g;
        if (row < p.g) {
          const float lse = seen ? (ref * f.c + __log2f(l) - kShift<X>) * 0.6931471805599453f : -INFINITY;
          if constexpr (SPLIT)
            f.part_lse[h.z * rows + at + row] = lse;
          else
            p.lse[at + row] = lse;
        }
        const uint32_t acc = tmem + (static_cast<uint32_t>(w * 32) << 16) + 256u + b * 128u;
        using Out = std::conditional_t<SPLIT, float, X>;
        Out* to = (SPLIT ? reinterpret_cast<Out*>(f.part_o) + h.z * rows * D : static_cast<Out*>(p.out)) +
                  (at + (tid >> 3)) * D + (tid & 7) * 4;
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          float o[32];
          tmem_ld32_start(acc + 32 * ch, o);
          tmem_wait32(o);
          if (weight == 0.f) {  // no key: what stands there may be anything
#pragma unroll
            for (int u = 0; u < 32; ++u) o[u] = 0.f;
          }
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const float2 w2 = make_float2(weight, weight), lo = fmul2(make_float2(o[4 * u], o[4 * u + 1]), w2),
                         hi = fmul2(make_float2(o[4 * u + 2], o[4 * u + 3]), w2);
            *reinterpret_cast<float4*>(stage + row * kPitch + 4 * u) = make_float4(lo.x, lo.y, hi.x, hi.y);
          }
          all_here();
          // eight threads a head, 16 heads at a time
          const float* from = stage + (tid >> 3) * kPitch + (tid & 7) * 4;
#pragma unroll
          for (int k = 0; k < G / 16; ++k) {
            if ((tid >> 3) + 16 * k >= p.g) break;
            float4 v = *reinterpret_cast<const float4*>(from + 16 * k * kPitch);
#pragma unroll
            for (int r = 1; r < R; ++r) {
              const float4 x = *reinterpret_cast<const float4*>(from + (r * G + 16 * k) * kPitch);
              const float2 lo = fadd2(make_float2(v.x, v.y), make_float2(x.x, x.y)),
                           hi = fadd2(make_float2(v.z, v.w), make_float2(x.z, x.w));
              v = make_float4(lo.x, lo.y, hi.x, hi.y);
            }
            if constexpr (SPLIT)
              *reinterpret_cast<float4*>(to + static_cast<long long>(16 * k) * D + 32 * ch) = v;
            else
              *reinterpret_cast<uint2*>(to + static_cast<long long>(16 * k) * D + 32 * ch) =
                  make_uint2(pack_pair<X>(v.x, v.y), pack_pair<X>(v.z, v.w));
          }
          all_here();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + C::kBarOFree + b);
        ++on;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

template <typename X, int D, int R, bool SPLIT>
cudaError_t start(FwdArgs f, const CUtensorMap& tq, cudaStream_t stream) {
  constexpr auto kernel = sparse_fwd_kernel<X, D, R, SPLIT>;
  const cudaError_t e = smem_limit_once<kernel>(Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  const long long grid = std::min(f.l.items, 152ll);
  set_step(f.l, f.p.Hk, grid);
  kernel<<<static_cast<unsigned>(grid), kThreads<R>, Cfg<D>::kSmem, stream>>>(tq, f);
  return cudaGetLastError();
}

template <typename X, int D, int R>
cudaError_t run(const SparseParams& p, int dtype, void* workspace, cudaStream_t stream) {
  CUtensorMap tq;
  FwdArgs f;
  f.p = p;
  f.l.slots = static_cast<int>(sparse_slots(p));
  f.n_split = sparse_splits(p.Tq, p.Hk, f.l.slots);
  f.l.items = static_cast<long long>(p.Tq) * p.Hk * f.n_split;
  f.l.t0 = 0;
  f.l.n_z = f.n_split;
  f.l.split = 1;
  f.l.per = std::max(1, ((f.l.slots + 127) / 128 + f.n_split - 1) / f.n_split);
  f.c = p.scale * 1.4426950408889634f;
  f.part_o = static_cast<float*>(workspace);
  f.part_lse = f.part_o + static_cast<long long>(f.n_split) * p.Tq * p.Hq * D;
  f.wait_ns = attn_wait_ns(f.l.slots / 128 + 1);
  if (!make_heads_map(&tq, p, p.q, p.q_st, p.q_sh, p.g)) return cudaErrorInvalidValue;
  if (f.n_split == 1) return start<X, D, R, false>(f, tq, stream);
  cudaError_t e = start<X, D, R, true>(f, tq, stream);
  if (e != cudaSuccess) return e;
  AttnParams a;
  std::memset(&a, 0, sizeof(a));
  a.Tq = p.Tq;
  a.Hq = p.Hq;
  a.D = D;
  a.out = p.out;
  a.lse = p.lse;
  return launch_attn_join(a, dtype, f.part_o, f.part_lse, f.n_split, stream);
}

template <typename X, int D>
cudaError_t by_heads(const SparseParams& p, int dtype, void* ws, cudaStream_t s) {
  if (p.g <= 32) return run<X, D, 4>(p, dtype, ws, s);
  return p.g <= 64 ? run<X, D, 2>(p, dtype, ws, s) : run<X, D, 1>(p, dtype, ws, s);
}

}  // namespace

cudaError_t launch_sparse_forward(const SparseParams& p, int dtype, void* workspace, cudaStream_t s) {
  if (dtype == CSA_BF16)
    return p.D == 128 ? by_heads<__nv_bfloat16, 128>(p, dtype, workspace, s)
                      : by_heads<__nv_bfloat16, 64>(p, dtype, workspace, s);
  return p.D == 128 ? by_heads<__half, 128>(p, dtype, workspace, s) : by_heads<__half, 64>(p, dtype, workspace, s);
}

cudaError_t take_status_sparse_fwd(uint32_t* out, cudaStream_t stream) { return take_status(out, stream); }

}  // namespace csa
