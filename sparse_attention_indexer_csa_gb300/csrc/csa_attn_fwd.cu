// csa_attn_fwd.cu -- causal attention over packed sequences on the tensor
// cores: forward, and the join of split keys.
//
//   s_j = scale q.k_j over the keys a row sees, out = sum_j p_j v_j with
//   p = softmax(s), lse = log sum_j exp(s_j).
//
// An item is TILES blocks of 128 query rows of one sequence and one key head; a
// CTA walks the keys in tiles of 128, in one pass with a running reference m
// and sum l:
//   S = Q . K^T     (A = q block, B = k tile, both in shared memory, to TMEM)
//   P = 2^(c (S - m)) in the storage type, c = scale log2(e), written over S
//   O += P . V      (A = P in TMEM, B = v tile read MN-major, O in TMEM)
// and at the end out = O / l, lse = scale m + ln l.
//
// Rows: the g = Hq/Hk query heads that share a key head are rows of the same
// block (row = token * g + head), so a block holds 128/g consecutive tokens,
// K and V are read once per group, and one token of g heads (decoding) is a
// block like any other.
//
// m is a reference, not the running maximum: the maximum of the first tile,
// raised to the maximum so far (with O and l rescaled and the tile's P formed
// again) only when a tile's sum of P exceeds kRaise.  Up to there P is in range of
// fp16 too, its relative precision is the same and so is the quotient O / l; no
// maximum is taken in the tiles that follow.  Where a first tile's scores are
// all -inf, m is f.lowest, so that the first score above gives an infinite P
// and raises it (asking each tile for rows without a reference took 2 %).
//
// Roles (TILES = 2: 12 warps, one CTA per SM; TILES = 1: 8 warps, two CTAs
// per SM):
//   warps 0..4 TILES-1  softmax: one thread per row, all 128 scores of a tile
//                       in registers; then the division and the stores
//   next warp           issuer of the products, one thread
//   next warp           TMA producer, one thread
//   next warp           items: a CTA that has one more item to come takes it from
//                       the blocks of the grid that have not started (cluster
//                       launch control), so its rows, first tiles and query
//                       block are on their way while the former item ends
//   next warp           value tiles that hold keys hidden from some row
// With two blocks the tensor cores form S and O of one while the softmax of
// the other runs; TMEM holds S0 S1 O0 O1 (512 columns).  With one block the
// second CTA on the SM does the same.
//
// Keys may be split over n_split items (few rows, long caches): each writes
// its normalised O and lse in fp32, and a second kernel joins them.
//
// Measured (bf16, 64 + 8 heads of 128): a prompt of 16384 tokens 2.75 ms, 1600
// TFLOP/s of 1885 (a library product's rate): tensor cores.  32768 tokens in 22
// documents 1.31 ms, 1289 TFLOP/s: an SM takes 55 items of 13 key tiles, and between the
// last product of one and the first P of the next some 5 us pass (diagonal tiles
// add 5 % of products that do not count).  One token of 64
// sequences over 2048 to 8192 cached ones 0.248 ms, 5.4 TB/s of 6.7; of one
// sequence over 131072, 0.095 ms, 5.7 TB/s: memory, and the join's launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "csa_attn_internal.h"
#include "csa_attn_tiles.cuh"

namespace csa {
namespace {

// P is formed 2^kShift times its size, so that fp16 holds weights down to 2^-33 of the reference's (at 2^-25, as they
// come, 131072 keys of that weight would be in l and not in O); O and l share the factor.  The reference is raised
// when a tile's sum of P exceeds kRaise: P stays in range, and a first tile (128 at most, unshifted) never asks for it.
template <typename X>
constexpr int kShift = is_bf16<X>() ? 0 : 8;
template <typename X>
constexpr float kRaise = is_bf16<X>() ? 4096.f : 32768.f;

// ROWS: rows of a block that may be used.  32 (with TILES = 1) keeps a smaller
// query block in shared memory and a third key or value tile in its place; the
// products read 128 rows all the same, and what they read past the block
// reaches only the unused rows of S.
template <int D, int TILES, int ROWS>
struct FwdCfg {
  static constexpr uint32_t kTile = kChunkBytes * (D / 64);  // 128 rows x D, 64 columns per 16 KB chunk
  static constexpr uint32_t kQChunk = ROWS * 128, kQTile = kQChunk * (D / 64);  // 64 columns of the query block; all
  static constexpr int kStages = TILES == 2 ? (D == 128 ? 4 : 8) : ROWS == 32 ? (D == 128 ? 3 : 6) : (D == 128 ? 2 : 5);
  static constexpr int kWarps = TILES == 2 ? 12 : 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kMmaWarp = 4 * TILES, kTmaWarp = kMmaWarp + 1, kItemWarp = kMmaWarp + 2;
  static constexpr uint32_t kOffQ = 0, kOffKv = kOffQ + TILES * kQTile;
  // TILES = 2: 64 columns of each block's output on their way to memory
  static constexpr uint32_t kOffOut = kOffKv + kStages * kTile;
  static constexpr uint32_t kOffBar = kOffOut + (TILES == 2 ? 2 * kChunkBytes : 0);
  static constexpr int kSlots = 2;  // items ahead
  static constexpr int kBarQ = 0, kBarQFree = TILES, kBarFull = 2 * TILES, kBarEmpty = kBarFull + kStages,
                       kBarS = kBarEmpty + kStages, kBarP = kBarS + TILES, kBarO = kBarP + TILES,
                       kBarItem = kBarO + TILES, kBarItemFree = kBarItem + kSlots, kBarNext = kBarItemFree + kSlots,
                       kBarSoon = kBarNext + 1, kBarMeet = kBarSoon + 1, kBarLast = kBarMeet + TILES,
                       kBarDone = kBarLast + kStages, kBars = kBarDone + 1;
  static constexpr uint32_t kOffMisc = (kOffBar + 8 * kBars + 15) / 16 * 16, kOffItem = kOffMisc + 32;
  static constexpr uint32_t kSmem = kOffItem + kSlots * 64;
  static constexpr uint32_t kTmemCols = TILES == 2 ? 512 : 256;
  static constexpr uint32_t kO = 128 * TILES;  // first column of O
};
static_assert(FwdCfg<128, 2, 128>::kSmem <= 227 * 1024 && FwdCfg<64, 2, 128>::kSmem <= 227 * 1024, "one CTA per SM");
constexpr bool two_fit(uint32_t smem) { return 2 * (smem + 1024) <= 228 * 1024; }
static_assert(two_fit(FwdCfg<128, 1, 128>::kSmem) && two_fit(FwdCfg<64, 1, 128>::kSmem) &&
                  two_fit(FwdCfg<128, 1, 32>::kSmem) && two_fit(FwdCfg<64, 1, 32>::kSmem),
              "two CTAs per SM");

struct FwdArgs {
  AttnParams a;
  int tq;        // tokens per block of 128 rows
  int nb;        // ceil(Tq / (TILES * tq))
  int n_split;
  float c;       // scale * log2(e)
  float lowest;  // the least reference of a row: c * lowest is finite
  float* part_o;    // [n_split][Tq * Hq][D] (n_split > 1)
  float* part_lse;  // [n_split][Tq * Hq]
  unsigned long long wait_ns;
};

// One item: a run of at most TILES * tq query rows of one sequence (or of rows
// outside all of them: lk = 0), one key head, one share of the keys.
struct FwdItem {
  SeqExt s;
  int t0, t1;     // rows; t0 >= t1: no more items
  int lo, hi[2];  // block w walks the key tiles lo .. hi[w]-1
  int n_tok[2];   // tokens of each block
  int hk, z;      // key head, share
  int open;       // keys that all rows see: the value tiles past them are mended before their products
  int seen;       // keys that some row sees
  int odd;        // first key tile of which values were taken out (see mend_values)
};
static_assert(sizeof(FwdItem) <= 64, "a slot");

// A warp; every lane gets the result.
template <int TILES>
__device__ __forceinline__ FwdItem make_item(const FwdArgs& f, uint32_t id) {
  const AttnParams& a = f.a;
  FwdItem it;
  const uint32_t rest = id / static_cast<uint32_t>(a.Hk);
  it.hk = static_cast<int>(id - rest * static_cast<uint32_t>(a.Hk));
  const uint32_t x = rest / static_cast<uint32_t>(f.n_split);
  it.z = static_cast<int>(rest - x * static_cast<uint32_t>(f.n_split));
  // rows are taken from the last ones on: those that see most keys first
  const RowItem r = find_row_item(a, TILES * f.tq, f.nb, f.nb + a.N - static_cast<int>(x));
  it.s = r.s;
  it.t0 = r.t0;
  it.t1 = r.t1;
  it.odd = INT32_MAX;
  it.open = r.t0 < r.t1 ? keys_seen(a, r.s, r.t0 - r.s.q0) : 0;
  it.lo = 0;
  int top = 0;
  it.seen = 0;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    it.n_tok[w] = w < TILES ? min(f.tq, max(0, r.t1 - r.t0 - w * f.tq)) : 0;
    const int see = it.n_tok[w] > 0 ? keys_seen(a, r.s, r.t0 + w * f.tq + it.n_tok[w] - 1 - r.s.q0) : 0;
    it.hi[w] = (see + 127) >> 7;
    top = max(top, it.hi[w]);
    it.seen = max(it.seen, see);
  }
  if (f.n_split > 1) {
    const int share = (top + f.n_split - 1) / f.n_split;
    it.lo = it.z * share;
#pragma unroll
    for (int w = 0; w < 2; ++w) it.hi[w] = max(it.lo, min(it.hi[w], it.lo + share));
  }
  return it;
}

// What the products of a value tile may not meet, since a hidden key's P of 0
// does not cancel it.  Rows from `held` on are the sequence's no more, or hidden
// from every row of the item: cleared.  Those from `open` on are hidden from some: what is infinite
// or NaN among them is taken out, and `odd` remembers the tile (patch_row adds
// it to the rows that see it).  By a warp of its own, between the tile's arrival
// and the products: 2.72 -> 2.77 ms for a prompt of 16384 tokens, 1.26 -> 1.33
// for 22 documents; in the softmax warps it cost 5 to 8 % of a prompt's time.
template <typename X, int D>
__device__ __forceinline__ void mend_values(uint8_t* tile, int held, int open, int* odd, int j) {
  constexpr uint32_t kExp = is_bf16<X>() ? 0x7f807f80u : 0x7c007c00u, kOne = is_bf16<X>() ? 0x00800080u : 0x04000400u;
  constexpr int P = D / 8;  // 16-byte pieces of a row; piece `q` of row `row` (whatever the swizzle makes of it)
  auto at = [&](int row, int q) {
    return reinterpret_cast<uint4*>(tile + (q >> 3) * kChunkBytes + row * 128 + ((q & 7) * 16));
  };
  const int lane = static_cast<int>(lane_id()), first = max(0, min(open, held)), last = min(held, 128);
  // an exponent of all ones carries into the sign's place when one is added to it
  uint32_t found = 0u;
#pragma unroll 4
  for (int i = lane; i < (last - first) * P; i += 32) {
    const uint4 v = *at(first + i / P, i % P);
    found |= ((v.x & kExp) + kOne) | ((v.y & kExp) + kOne) | ((v.z & kExp) + kOne) | ((v.w & kExp) + kOne);
  }
  if (__any_sync(0xffffffffu, (found & 0x80008000u) != 0u)) {
    if (lane == 0) atomicMin(odd, j);
    auto finite = [&](uint32_t x) {
      const uint32_t bad = ((x & kExp) + kOne) & 0x80008000u;  // a bit for each half to take out
      return x & ~((bad >> 15) * 0xffffu);
    };
#pragma unroll 1
    for (int i = lane; i < (last - first) * P; i += 32) {
      uint4* p = at(first + i / P, i % P);
      const uint4 v = *p;
      *p = make_uint4(finite(v.x), finite(v.y), finite(v.z), finite(v.w));
    }
  }
#pragma unroll 4
  for (int i = lane; i < (128 - max(0, held)) * P; i += 32) *at(max(0, held) + i / P, i % P) = make_uint4(0u, 0u, 0u, 0u);
}

// Adds to a row's stored output (type Y) what mend_values took out and the row
// sees: the infinite and NaN values of its keys first .. see-1.  (In line: a
// call would take registers from the loop over the tiles.)
template <typename X, int D, typename Y>
__device__ __forceinline__ void patch_row(const X* v, long long v_st, int first, int see, Y* out) {
  constexpr uint32_t kExp = is_bf16<X>() ? 0x7f80u : 0x7c00u;
#pragma unroll 1
  for (int key = first; key < see; ++key) {
#pragma unroll 1
    for (int d = 0; d < D; ++d) {
      const X* x = v + key * v_st + d;
      if ((*reinterpret_cast<const uint16_t*>(x) & kExp) != kExp) continue;
      out[d] = static_cast<Y>(static_cast<float>(out[d]) + static_cast<float>(*x));
    }
  }
}

// SPLIT: items are shares of the keys, and their outputs go to the workspace.
template <typename X, int D, int TILES, int ROWS, bool SPLIT>
__global__ void __launch_bounds__(FwdCfg<D, TILES, ROWS>::kThreads, TILES == 2 ? 1 : 2)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                    const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_out,
                    const FwdArgs f) {
  using C = FwdCfg<D, TILES, ROWS>;
  extern __shared__ __align__(1024) uint8_t base[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + C::kOffBar);
  uint8_t* next_slot = base + C::kOffMisc;  // 16 bytes: the answer to a request for the next item
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + C::kOffMisc + 16);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(base + C::kOffMisc + 20);
  const AttnParams& a = f.a;
  const int warp = threadIdx.x / 32;
  const uint32_t lane = lane_id();

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kBars; ++i) {
      int n = 1;
      if ((i >= C::kBarP && i < C::kBarP + TILES) || (i >= C::kBarMeet && i < C::kBarMeet + TILES)) n = 4;
      if (i >= C::kBarItemFree && i < C::kBarItemFree + C::kSlots) n = 3 + 4 * TILES;
      mbar_init(bars + i, n);
    }
    if ((smem_u32(base) & 1023u) != 0u) record_error(kErrDevice);  // the swizzled tiles would be misread
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == C::kTmaWarp && lane == 0) {
    prefetch_tmap(&tmap_q);
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
    if (TILES == 2 && !SPLIT) prefetch_tmap(&tmap_out);
  }
  if (warp == C::kMmaWarp) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl ctl{abort_flag, f.wait_ns};
  // the role's next item; null after the last one or a wait that gave up.  Its slot is the role's until
  // give_item(): fields are read where they are needed instead of being held in registers
  uint32_t n_item = 0;
  auto next_item = [&]() -> const volatile FwdItem* {
    const uint32_t sl = n_item & 1u;
    if (!mbar_wait(bars + C::kBarItem + sl, (n_item >> 1) & 1u, ctl)) return nullptr;
    const volatile FwdItem* it = reinterpret_cast<const volatile FwdItem*>(base + C::kOffItem + 64 * sl);
    return it->t0 < it->t1 ? it : nullptr;
  };
  auto give_item = [&] {
    mbar_arrive(bars + C::kBarItemFree + (n_item & 1u));
    ++n_item;
  };

  if (warp == C::kItemWarp) {
    reg_shrink();
    // ----------------------------------------------------------------------- items
    // Prepared ahead of the other roles: the search for a run of rows is a chain of global loads.
    if (blockIdx.x == 0)
      for (int i = static_cast<int>(lane); i < a.N; i += 32) seq_extent(a, i);
    uint32_t id = blockIdx.x, n = 0, asked = 0;
    bool more = true;
    while (more) {
      const FwdItem it = make_item<TILES>(f, id);
      if (it.t0 < it.t1) {  // two borders may fall together: no row
        if (lane == 0) *reinterpret_cast<FwdItem*>(base + C::kOffItem + 64 * (n & 1u)) = it;
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + C::kBarItem + (n & 1u));
        ++n;
        // Another one is asked for when the copies of this one have all been started, two or three tiles before
        // its end: an item that a CTA holds ahead is one that no idle CTA can take.
        more = mbar_wait(bars + C::kBarSoon, (n - 1u) & 1u, ctl) &&
               mbar_wait(bars + C::kBarItemFree + (n & 1u), ((n >> 1) & 1u) ^ 1u, ctl);
      }
      if (!more) break;
      if (lane == 0) request_next(next_slot, bars + C::kBarNext);
      volatile uint32_t dummy = 0;  // the answer is waited for even when a role gave up: it writes shared memory
      const WaitCtl dctl{&dummy, ctl.limit_ns};
      const bool got = mbar_wait(bars + C::kBarNext, asked & 1u, dctl);
      ++asked;
      more = got && answer_next(next_slot, id);
    }
    if (*abort_flag == 0u) {
      const uint32_t sl = n & 1u;
      mbar_wait(bars + C::kBarItemFree + sl, ((n >> 1) & 1u) ^ 1u, ctl);
      if (lane == 0) reinterpret_cast<FwdItem*>(base + C::kOffItem + 64 * sl)->t1 = INT32_MIN;
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + C::kBarItem + sl);
    }
  } else if (warp == C::kTmaWarp) {
    reg_shrink();
    if (lane == 0) {  // --------------------------------------------------- TMA producer
      const uint64_t q_pol = l2_policy_evict_first(), kv_pol = l2_policy_evict_last();
      uint32_t at = 0, phase = 1, nq[TILES] = {};
      Copies copies;
      while (const volatile FwdItem* it = next_item()) {
        const int lo = it->lo, hi[2] = {it->hi[0], it->hi[1]}, top = max(hi[0], hi[1]);
        const int t0 = it->t0, k0 = it->s.k0, hk = it->hk, open = it->open;
        give_item();
        for (int w = 0; w < TILES; ++w) {
          if (hi[w] <= lo) continue;
          if (!mbar_wait(bars + C::kBarQFree + w, (nq[w] & 1u) ^ 1u, ctl)) continue;
          ++nq[w];
          mbar_arrive_expect_tx(bars + C::kBarQ + w, static_cast<uint32_t>(f.tq * a.g) * 128u * (D / 64));
          for (int ch = 0; ch < D / 64; ++ch)
            tma_load_4d_hint(base + C::kOffQ + w * C::kQTile + ch * C::kQChunk, &tmap_q, bars + C::kBarQ + w, ch * 64, 0,
                             t0 + w * f.tq, hk, q_pol);
        }
        for (int j = lo; j < top; ++j)
          for (int kv = 0; kv < 2; ++kv) {
            const uint32_t st = at, ph = phase;
            if (++at == static_cast<uint32_t>(C::kStages)) {
              at = 0;
              phase ^= 1u;
            }
            if (!mbar_wait(bars + C::kBarEmpty + st, ph, ctl)) continue;
            // a value tile that is mended lands on the stage's other barrier; who mends it completes the first
            const bool mend = kv && (j + 1) * 128 > open;
            uint64_t* bar = bars + (mend ? C::kBarLast : C::kBarFull) + st;
            copies.start(static_cast<int>(st), mend, ph ^ 1u);
            mbar_arrive_expect_tx(bar, C::kTile);
            for (int ch = 0; ch < D / 64; ++ch)
              tma_load_3d_hint(base + C::kOffKv + st * C::kTile + ch * kChunkBytes, kv ? &tmap_v : &tmap_k, bar, ch * 64,
                               k0 + j * 128, hk, kv_pol);
          }
        mbar_arrive(bars + C::kBarSoon);
      }
      // no copy is in flight when the CTA ends, a role's giving up included
      volatile uint32_t dummy = 0;
      const WaitCtl dctl{&dummy, ctl.limit_ns};
      for (int w = 0; w < TILES; ++w)
        if (nq[w] > 0) mbar_wait(bars + C::kBarQ + w, (nq[w] - 1u) & 1u, dctl);
      copies.drain([&](int st, bool mend, uint32_t parity) {
        mbar_wait(bars + (mend ? C::kBarLast : C::kBarFull) + st, parity, dctl);
      });
    }
  } else if (warp == C::kMmaWarp) {
    reg_shrink();
    // ----------------------------------------------------------------------- issuer of the products
    // The warp runs as one (uniform operands: a descriptor moved to uniform registers for each product made the
    // products wait for their issue), one elected thread issues.
    const uint32_t tm = static_cast<uint32_t>(uniform(static_cast<int>(tmem)));
    const uint64_t qd = smem_desc_kmajor(smem_u32(base + C::kOffQ), 128);
    const uint64_t kd = smem_desc_kmajor(smem_u32(base + C::kOffKv), 128);
    const uint64_t vd = smem_desc_mn_sw128(smem_u32(base + C::kOffKv), kChunkBytes, 1024u);
    constexpr uint32_t kIdS = idesc_f16<X>(128, 128, false), kIdO = idesc_f16<X>(128, D, true), kT = C::kTile >> 4;
    bool alive = true;
    auto wait = [&](int bar, uint32_t parity) { alive = alive && mbar_spin_warp(bars + bar, parity, ctl); };
    // S_w = Q_w . K^T
    auto scores = [&](int w, uint32_t st) {
      tc_fence_after();
      if (elect_one()) {
        if (alive) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint64_t o = static_cast<uint64_t>(((ks >> 2) * kChunkBytes + (ks & 3) * 32) >> 4);
            const uint64_t oq = static_cast<uint64_t>(((ks >> 2) * C::kQChunk + (ks & 3) * 32) >> 4);
            umma_bf16(tm + w * 128, qd + static_cast<uint64_t>(w * (C::kQTile >> 4)) + oq, kd + static_cast<uint64_t>(st * kT) + o, kIdS,
                      ks != 0 ? 1u : 0u);
          }
        }
        umma_commit(bars + C::kBarS + w);
      }
      __syncwarp();
    };
    // positions in the ring, kept without divisions; `seen` is what the look ahead found
    uint32_t at = 0, phase = 0;
    auto full = [&](bool seen) -> uint32_t {  // waits for the ring's next tile and returns its stage
      const uint32_t st = at;
      if (!seen) wait(C::kBarFull + static_cast<int>(st), phase);
      if (++at == static_cast<uint32_t>(C::kStages)) {
        at = 0;
        phase ^= 1u;
      }
      return st;
    };
    uint32_t p_par[TILES] = {}, q_par[TILES] = {};  // parities of P and Q
    while (const volatile FwdItem* it = next_item()) {
      const int lo = uniform(it->lo), hi[2] = {uniform(it->hi[0]), uniform(it->hi[1])}, top = max(hi[0], hi[1]);
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + C::kBarItemFree + (n_item & 1u));
      ++n_item;
      if (top <= lo) continue;
      uint32_t sk = full(false);
#pragma unroll
      for (int w = 0; w < TILES; ++w)
        if (hi[w] > lo) {
          wait(C::kBarQ + w, q_par[w]);
          q_par[w] ^= 1u;
          scores(w, sk);
        }
      for (int j = lo; j < top; ++j) {
        const uint32_t sv = full(false);
        if (j + 1 < top) sk = full(false);
#pragma unroll
        for (int w = 0; w < TILES; ++w) {
          if (j >= hi[w]) continue;
          wait(C::kBarP + w, p_par[w]);
          p_par[w] ^= 1u;
          tc_fence_after();
          if (elect_one()) {
            if (alive) {
#pragma unroll
              for (int ks = 0; ks < 8; ++ks)
                umma_bf16_tmem_a(tm + C::kO + w * 128, tm + w * 128 + 8u * ks,
                                 vd + static_cast<uint64_t>(sv * kT) + static_cast<uint64_t>(128 * ks), kIdO,
                                 (j != lo || ks != 0) ? 1u : 0u);
            }
            if (j + 1 >= hi[w]) umma_commit(bars + C::kBarO + w);
          }
          __syncwarp();
          if (j + 1 < hi[w]) scores(w, sk);
        }
      }
    }
    if (elect_one()) umma_commit(bars + C::kBarDone);
    __syncwarp();
    volatile uint32_t dummy = 0;
    const WaitCtl dctl{&dummy, ctl.limit_ns};
    mbar_wait(bars + C::kBarDone, 0u, dctl);
  } else if (warp < 4 * TILES) {  // ----------------------------------------- softmax, output
    reg_grow<TILES>();
    const int w = warp >> 2, row = (warp & 3) * 32 + static_cast<int>(lane);
    const int tok = row / a.g, head = row - tok * a.g;
    const uint32_t ts = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + w * 128;
    const uint32_t to = ts + (C::kO - w * 128) + w * 128;
    const float c = f.c;
    const bool has_rows = (warp & 3) * 32 < ROWS;  // of a warp without rows nothing is used
    uint32_t s_phase = 0, o_phase = 0, met = 0, ring = 0;  // ring: tiles of the ring before this item
    bool ok = true;
    while (const volatile FwdItem* it = next_item()) {
      const int lo = it->lo, my_hi = it->hi[w], top = max(it->hi[0], it->hi[1]), lk = it->s.lk;
      const bool row_ok = tok < it->n_tok[w];
      int see = 0, see_all = 0;  // keys this row sees; keys every row of the block sees
      if (my_hi > lo) {
        const SeqExt e{it->s.q0, it->s.q1, it->s.k0, lk};
        const int r = it->t0 + w * f.tq - e.q0;
        see_all = keys_seen(a, e, r);
        if (row_ok) see = keys_seen(a, e, r + tok);
      }
      float m = -INFINITY, l = 0.f;
      // The last block's scores of a tile are formed last: when they stand, all products with this key tile and
      // the former value tile are done, and one thread gives both back to the producer.  (A commit of the issuing
      // thread for each would hold up its next products.)
      const bool first_thread = (threadIdx.x & 127) == 0;
      const bool frees = my_hi == top && (w == TILES - 1 || it->n_tok[TILES - 1] <= 0) && first_thread;
      for (int j = lo; j < my_hi; ++j) {
        ok = ok && mbar_wait(bars + C::kBarS + w, s_phase, ctl);
        s_phase ^= 1u;
        tc_fence_after();
        const uint32_t nk = ring + 2u * static_cast<uint32_t>(j - lo);
        if (frees) {
          mbar_arrive(bars + C::kBarEmpty + nk % C::kStages);
          if (j > lo) mbar_arrive(bars + C::kBarEmpty + (nk - 1) % C::kStages);
        }
        if (j == my_hi - 1 && first_thread) mbar_arrive(bars + C::kBarQFree + w);  // the last product with Q
          if (ok && has_rows) {
          float tile;
          uint32_t pk[4][16];
          // the row's 128 scores, those it does not see at -inf
          auto load = [&](float (&s)[4][32]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) tmem_ld32_start(ts + 32 * i, s[i]);
#pragma unroll
            for (int i = 0; i < 4; ++i) tmem_wait32(s[i]);
            if ((j + 1) * 128 > see_all) {
              const int lim = see - j * 128;
#pragma unroll
              for (int i = 0; i < 128; ++i)
                if (i >= lim) s[i >> 5][i & 31] = -INFINITY;
            }
          };
          auto probs = [&](const float (&s)[4][32]) {
            const float b = static_cast<float>(kShift<X>) - m * c;
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int u = 0; u < 64; ++u) {
              const float* x = s[u >> 4] + 2 * (u & 15);
              const float2 e = ffma2(make_float2(x[0], x[1]), make_float2(c, c), make_float2(b, b));
              const float2 p = make_float2(exp2_approx(e.x), exp2_approx(e.y));
              sum[u & 1] = fadd2(sum[u & 1], p);
              pk[u >> 4][u & 15] = pack_pair<X>(p.x, p.y);
            }
            tile = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          };
          {
            float s[4][32];
            load(s);
            if (j == lo) m = fmaxf(row_max(s), f.lowest);
            probs(s);
          }
          if (__any_sync(0xffffffffu, tile > kRaise<X>)) {
            float s[4][32];
            load(s);
            // the former tiles' product with V has completed: its commit preceded this tile's scores
            const float mn = fmaxf(m, row_max(s));
            const float r = exp2_approx((m - mn) * c);
            m = mn;
            l *= r;
            if (j != lo) {
#pragma unroll
              for (int i = 0; i < D / 16; ++i) tmem_scale16(to + 16 * i, r);
            }
            probs(s);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_st16(ts + 16 * i, pk[i]);
          l += tile;
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + C::kBarP + w);
      }
      ring += 2u * static_cast<uint32_t>(max(0, top - lo));
      // ---------------------------------------------------------------- output
      const bool any = my_hi > lo;
      if (any) {
        ok = ok && mbar_wait(bars + C::kBarO + w, o_phase, ctl);
        o_phase ^= 1u;
        tc_fence_after();
        if (frees) mbar_arrive(bars + C::kBarEmpty + (ring - 1u) % C::kStages);
      }
      const bool seen = any && ok && (l > 0.f || l != l);
      const float inv = seen ? 1.f / l : 0.f;
      const float lse = seen ? (m * c + __log2f(l * (1.f / (1 << kShift<X>)))) * 0.6931471805599453f : -INFINITY;
      const long long rows = static_cast<long long>(a.Tq) * a.Hq;
      // element offset of row `r` of the block (and -1 for a row it does not hold)
      const int t_blk = it->t0 + w * f.tq, hk = it->hk, z = it->z;
      const long long at = row_ok ? static_cast<long long>(t_blk + tok) * a.Hq + hk * a.g + head : -1;
      if (at >= 0) {
        if constexpr (SPLIT)
          f.part_lse[z * rows + at] = lse;
        else
          a.lse[at] = lse;
      }
      if constexpr (TILES == 2 && !SPLIT) {
        // A full block goes through shared memory, 64 columns at a time, and is stored by TMA: a quarter of the
        // instructions of the stores below, which run once per item and wait for being fetched.
        if (it->n_tok[w] == f.tq) {
          uint8_t* mine = base + C::kOffOut + w * kChunkBytes;
#pragma unroll 1
          for (int ch = 0; ch < D / 64; ++ch) {
            if (first_thread) bulk_wait_group_read<0>();  // what was staged before has been read
            meet(bars + C::kBarMeet + w, met, ctl);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float o[32];
              if (any) {
                tmem_ld32_start(to + 64 * ch + 32 * h, o);
                tmem_wait32(o);
              }
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                uint4 q = make_uint4(0u, 0u, 0u, 0u);
                if (seen)
                  q = make_uint4(pack_pair<X>(o[8 * u] * inv, o[8 * u + 1] * inv),
                                 pack_pair<X>(o[8 * u + 2] * inv, o[8 * u + 3] * inv),
                                 pack_pair<X>(o[8 * u + 4] * inv, o[8 * u + 5] * inv),
                                 pack_pair<X>(o[8 * u + 6] * inv, o[8 * u + 7] * inv));
                *reinterpret_cast<uint4*>(mine + row * 128 + (((4 * h + u) ^ (row & 7)) * 16)) = q;
              }
            }
            fence_proxy_async_shared();
            meet(bars + C::kBarMeet + w, met, ctl);
            if (first_thread) {
              tma_store_4d(&tmap_out, mine, ch * 64, 0, t_blk, hk);
              bulk_commit_group();
            }
          }
          if (it->odd < my_hi) {
            if (first_thread) bulk_wait_group_all();
            meet(bars + C::kBarMeet + w, met, ctl);
            if (seen && at >= 0)
              patch_row<X, D>(static_cast<const X*>(a.v) + it->s.k0 * a.v_st + hk * a.v_sh, a.v_st, it->odd * 128, see,
                              static_cast<X*>(a.out) + at * D);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bars + C::kBarItemFree + (n_item & 1u));
          ++n_item;
          continue;
        }
      }
      // Lanes 4 i .. 4 i + 3 exchange their rows' 16-byte pieces, so that four lanes store 64 bytes of one row:
      // a store of 16 bytes by each of 32 rows takes as many passes through L1 as it has rows.
      long long at4[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) at4[u] = __shfl_sync(0xffffffffu, at, (lane & ~3u) + u);
      // (not unrolled: this runs once per item, and its time is that of fetching its instructions)
#pragma unroll 1
      for (int i = 0; i < D / 32; ++i) {
        float o[32];
        __syncwarp();
        if (any) {
          tmem_ld32_start(to + 32 * i, o);
          tmem_wait32(o);
        }
#pragma unroll
        for (int u = 0; u < 32; ++u) o[u] = seen ? o[u] * inv : 0.f;
        if constexpr (SPLIT) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // 16 fp32 values: four pieces
            uint4 q[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
              q[u] = make_uint4(__float_as_uint(o[16 * h + 4 * u]), __float_as_uint(o[16 * h + 4 * u + 1]),
                                __float_as_uint(o[16 * h + 4 * u + 2]), __float_as_uint(o[16 * h + 4 * u + 3]));
            transpose4(q, lane);
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (at4[u] >= 0)
                reinterpret_cast<uint4*>(f.part_o + (z * rows + at4[u]) * D + 32 * i + 16 * h)[lane & 3] = q[u];
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
            if (at4[u] >= 0) reinterpret_cast<uint4*>(static_cast<X*>(a.out) + at4[u] * D + 32 * i)[lane & 3] = q[u];
        }
      }
      if (it->odd < my_hi) {
        __syncwarp();  // the row's stores may have been another lane's
        __threadfence_block();
        if (seen && at >= 0) {
          const X* v = static_cast<const X*>(a.v) + it->s.k0 * a.v_st + hk * a.v_sh;
          if constexpr (SPLIT)
            patch_row<X, D>(v, a.v_st, it->odd * 128, min(see, my_hi * 128), f.part_o + (z * rows + at) * D);
          else
            patch_row<X, D>(v, a.v_st, it->odd * 128, see, static_cast<X*>(a.out) + at * D);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + C::kBarItemFree + (n_item & 1u));
      ++n_item;
    }
    if (TILES == 2 && !SPLIT && (threadIdx.x & 127) == 0) bulk_wait_group_all();
  } else {  // ---------------------------------------------------------------- mender
    reg_shrink();
    uint32_t ring = 0, last_par = 0;
    while (const volatile FwdItem* it = next_item()) {
      const int lo = it->lo, top = max(it->hi[0], it->hi[1]), open = it->open, seen = it->seen;
      for (int j = max(lo, open >> 7); j < top; ++j) {
        const uint32_t st = (ring + 2u * static_cast<uint32_t>(j - lo) + 1u) % C::kStages;
        if (mbar_wait(bars + C::kBarLast + st, (last_par >> st) & 1u, ctl))
          mend_values<X, D>(base + C::kOffKv + st * C::kTile, seen - j * 128, open - j * 128, const_cast<int*>(&it->odd), j);
        last_par ^= 1u << st;
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + C::kBarFull + st);
      }
      ring += 2u * static_cast<uint32_t>(max(0, top - lo));
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + C::kBarItemFree + (n_item & 1u));
      ++n_item;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C::kMmaWarp) tmem_dealloc(tmem, C::kTmemCols);
}

// out = sum_z w_z O_z / sum_z w_z with w_z = exp(lse_z - max lse).  A block per
// row and head: 256 / (D/4) groups of threads take every so many shares, four
// values a thread, and their sums are added in order.  Bytes: n_split (D + 1)
// fp32 read per row and head.  (One group for all shares took longer than the
// attention itself where a single sequence is cut into many.)
template <typename X, int D>
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnParams a, const float* part_o, const float* part_lse,
                                                       int n_split) {
  constexpr int LANES = D / 4, GROUPS = 256 / LANES;
  __shared__ float w[kMaxSplit], top[8], total[8];
  __shared__ float4 acc[GROUPS][LANES];
  const long long rows = static_cast<long long>(a.Tq) * a.Hq, r = blockIdx.x;
  const int tid = threadIdx.x, warp = tid / 32;
  const float lz = tid < n_split ? part_lse[tid * rows + r] : -INFINITY;  // n_split <= kMaxSplit = 256
  float m = lz;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((tid & 31) == 0) top[warp] = m;
  __syncthreads();
  m = top[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmaxf(m, top[i]);
  const float ms = m == -INFINITY ? 0.f : m;
  const float wz = exp2_approx((lz - ms) * 1.4426950408889634f);  // 0 for a share that saw nothing
  float s = wz;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (tid < n_split) w[tid] = wz;
  if ((tid & 31) == 0) total[warp] = s;
  __syncthreads();
  s = ((total[0] + total[1]) + (total[2] + total[3])) + ((total[4] + total[5]) + (total[6] + total[7]));
  const int g = tid / LANES, l = tid % LANES;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int z = g; z < n_split; z += GROUPS) {
    const float f = w[z];
    const float4 o = reinterpret_cast<const float4*>(part_o + (z * rows + r) * D)[l];
    if (f != 0.f) {
      v.x = fmaf(f, o.x, v.x);
      v.y = fmaf(f, o.y, v.y);
      v.z = fmaf(f, o.z, v.z);
      v.w = fmaf(f, o.w, v.w);
    }
  }
  acc[g][l] = v;
  __syncthreads();
  if (g != 0) return;
#pragma unroll
  for (int i = 1; i < GROUPS; ++i) {
    const float4 o = acc[i][l];
    v.x += o.x;
    v.y += o.y;
    v.z += o.z;
    v.w += o.w;
  }
  const float inv = s == 0.f ? 0.f : 1.f / s;
  uint2 u;
  u.x = pack_pair<X>(v.x * inv, v.y * inv);
  u.y = pack_pair<X>(v.z * inv, v.w * inv);
  reinterpret_cast<uint2*>(static_cast<X*>(a.out) + r * D)[l] = u;
  if (l == 0) a.lse[r] = s == 0.f ? -INFINITY : ms + logf(s);
}

template <typename X, int D, int TILES, int ROWS>
cudaError_t run(const AttnParams& p, int n_split, void* workspace, cudaStream_t stream) {
  using C = FwdCfg<D, TILES, ROWS>;
  CUtensorMap tq, tk, tv, to;
  FwdArgs f;
  f.a = p;
  f.tq = ROWS / p.g;
  f.nb = static_cast<int>((static_cast<long long>(p.Tq) + TILES * f.tq - 1) / (TILES * f.tq));
  f.n_split = n_split;
  f.c = p.scale * 1.4426950408889634f;
  f.lowest = -3.3e38f / std::max(1.f, f.c);
  f.part_o = static_cast<float*>(workspace);
  f.part_lse = f.part_o + static_cast<long long>(n_split) * p.Tq * p.Hq * D;
  f.wait_ns = attn_wait_ns(attn_steps_keys(p.Tk));
  if (!make_rows_map(&tq, p, p.q, p.q_st, p.q_sh, f.tq) || !make_keys_map(&tk, p, p.k, p.k_st, p.k_sh) ||
      !make_keys_map(&tv, p, p.v, p.v_st, p.v_sh) ||
      !make_rows_map(&to, p, p.out, static_cast<long long>(p.Hq) * D, D, f.tq))
    return cudaErrorInvalidValue;
  const long long grid = (static_cast<long long>(f.nb) + p.N + 1) * p.Hk * n_split;
  const long long rows = static_cast<long long>(p.Tq) * p.Hq;
  if (grid > 0x7FFFFFFFll || (n_split > 1 && rows > 0x7FFFFFFFll)) return cudaErrorInvalidValue;
  cudaError_t e;
  if (n_split == 1) {
    constexpr auto kernel = attn_fwd_kernel<X, D, TILES, ROWS, false>;
    if ((e = smem_limit_once<kernel>(C::kSmem)) != cudaSuccess) return e;
    kernel<<<static_cast<unsigned>(grid), C::kThreads, C::kSmem, stream>>>(tq, tk, tv, to, f);
    return cudaGetLastError();
  }
  constexpr auto kernel = attn_fwd_kernel<X, D, TILES, ROWS, true>;
  if ((e = smem_limit_once<kernel>(C::kSmem)) != cudaSuccess) return e;
  kernel<<<static_cast<unsigned>(grid), C::kThreads, C::kSmem, stream>>>(tq, tk, tv, to, f);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  attn_join_kernel<X, D><<<static_cast<unsigned>(rows), 256, 0, stream>>>(p, f.part_o, f.part_lse, n_split);
  return cudaGetLastError();
}

template <typename X, int D>
cudaError_t by_plan(const AttnParams& p, void* ws, cudaStream_t s) {
  const AttnPlan plan = attn_plan(p.N, p.Tq, p.Tk, p.Hk, p.g);
  if (plan.tiles == 2) return run<X, D, 2, 128>(p, plan.n_split, ws, s);
  return plan.rows == 32 ? run<X, D, 1, 32>(p, plan.n_split, ws, s) : run<X, D, 1, 128>(p, plan.n_split, ws, s);
}

}  // namespace

cudaError_t launch_attn_forward(const AttnParams& p, int dtype, void* workspace, cudaStream_t s) {
  if (dtype == CSA_BF16)
    return p.D == 128 ? by_plan<__nv_bfloat16, 128>(p, workspace, s) : by_plan<__nv_bfloat16, 64>(p, workspace, s);
  return p.D == 128 ? by_plan<__half, 128>(p, workspace, s) : by_plan<__half, 64>(p, workspace, s);
}

cudaError_t launch_attn_join(const AttnParams& p, int dtype, const float* part_o, const float* part_lse, int n_split,
                             cudaStream_t s) {
  const long long rows = static_cast<long long>(p.Tq) * p.Hq;
  if (rows > 0x7FFFFFFFll || n_split > kMaxSplit) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(rows);
  if (dtype == CSA_BF16) {
    if (p.D == 128)
      attn_join_kernel<__nv_bfloat16, 128><<<grid, 256, 0, s>>>(p, part_o, part_lse, n_split);
    else
      attn_join_kernel<__nv_bfloat16, 64><<<grid, 256, 0, s>>>(p, part_o, part_lse, n_split);
  } else if (p.D == 128) {
    attn_join_kernel<__half, 128><<<grid, 256, 0, s>>>(p, part_o, part_lse, n_split);
  } else {
    attn_join_kernel<__half, 64><<<grid, 256, 0, s>>>(p, part_o, part_lse, n_split);
  }
  return cudaGetLastError();
}

cudaError_t take_status_attn_fwd(uint32_t* out, cudaStream_t stream) { return take_status(out, stream); }

}  // namespace csa
