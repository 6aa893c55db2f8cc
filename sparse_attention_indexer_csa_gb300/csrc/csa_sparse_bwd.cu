// csa_sparse_bwd.cu -- gradients of attention over listed blocks of keys.
//
//   delta = dout.out (per row and head),  p_j = exp(s_j - lse),
//   ds_j = p_j (dout.v_j - delta),  dq = scale sum_j ds_j k_j,
//   dk_j = scale sum_rows ds_j q,  dv_j = sum_rows p_j dout.
//
// The rows that list a key are not its neighbours, and each contributes a matrix
// product with its g heads to dk and dv.  So the work goes by rows, and every
// row's share of dk and dv for each slot of its list goes to memory, where a
// second kernel adds up the shares of a key in the order of the rows: no
// atomics on values, the same bits on every call.
//
//   sparse_rows_kernel  an item is a row, a key head and up to 64 of its query
//     heads; its listed keys, 128 at a time, are the rows of the products:
//       S^T = K Q^T, dP^T = V dO^T         (operands in shared memory)
//       P^T, dS^T in the storage type over S^T, dP^T in TMEM, dS^T to shared memory
//       dV = P^T dO, dK = dS^T Q           (A in TMEM, B read MN-major): the shares
//       dQ += dS K                         (A and B read MN-major)
//     so that a group of up to 64 heads costs no more than its heads; a larger one is two
//     items, each with shares of its own.
//   lists (sparse_count, _scan, _fill)  for each block the rows that
//     list it, in ascending order: a counting sort, the counts kept by groups of
//     rows so that the place of each entry does not depend on timing.
//   sparse_sum_kernel  a block of threads per key and key head adds the shares.
//
// Bytes: a share of dk and one of dv, D values each, per listed key, written once
// and read once.  For bf16 a share is kept in fp16 at a power of two of its own, from
// the bound sum over heads of |ds| |q| (p |dout|) that its key's thread adds up on the
// way: 11 bits, finer than ds and p have, at half of fp32's bytes (in bf16 it cost
// the gradients half of their precision, 0.0029 of their size for 0.0024).  For fp16,
// whose own roundings are no larger, it is fp32.  The scale meets dk when its shares have
// been added: a large one would take the power of two of a share whose bound is zero
// past fp32's range (0 * inf from a scale of 8 on).  As many rows at a time as
// kShareBytes hold.
//
// Where a list is one tile, delta is taken as sum_j p_j dout.v_j from the products at
// hand, in fp32: the rounding of out, which the forward stored, is an error of delta
// for all keys of the row at once, and shows where these are few.  That holds while the
// list is all that the softmax has, sum_j p_j = 1, and dout.out differs by no more than out's
// rounding: with out and lse of several calls joined, delta is dout.out, as it is for longer lists.
//
// Measured (bf16, D 128): 8192 rows of 64 heads and one key head, 256 listed entries
// each, 670 us: delta 60 to 69, lists 36, rows 355, sums 205 (1 GB of shares, which
// rows writes at 2.8 TB/s, forming 161 GFLOP, and sums reads at 5.0 TB/s).  4096 rows of 2 x
// 16 heads, 16 blocks of 16 and a window of 64: 550 us, of which rows 331 (4 TB/s of
// shares) and sums 181.
// With 64 heads the rows kernel is bound by its roles' steps one behind the other (P and dS of a tile
// wait for its scores, its shares for both, and one buffer holds each: tensor cores 22
// %, schedulers 43 %, HBM 39 %).
//
// fp16: dS is formed times a power of two that brings its bound 2 |dout| max|v| to
// 2^15 (|dout| over the item's heads, |v| over the finite values of the row's keys), or
// |dout| max|v| + |delta| where that is larger (out of joined calls), and P^T, at most
// 1, at 2^15 times its size; both are taken back in fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <type_traits>

#include "csa_sparse_list.cuh"

namespace csa {
namespace {

constexpr size_t kShareBytes = 4ull << 30;
constexpr int kHeads = 64;  // query heads of an item at most
constexpr int kGroups = 1024;  // groups of rows in the lists' sort at most
constexpr int kLists = 2;
constexpr int kDrainWarp = 4, kKeyWarp = 8, kValueWarp = 10, kMmaWarp = 12, kItemWarp = 13, kListWarp = 14, kDrain2Warp = 16, kMma2Warp = 20;
template <bool TWO>
constexpr int kThreads = 32 * (kMma2Warp + (TWO ? 1 : 0));

template <typename X>
constexpr int kProbExp = is_bf16<X>() ? 0 : 15;  // power of two of P^T

// What a share is kept in.
template <typename X>
struct ShareType {
  using T = __half;
};
template <>
struct ShareType<__half> {
  using T = float;
};

// TWO: items of up to 32 heads, whose scores and dS have two buffers each.
template <int D, bool TWO>
struct Cfg {
  static constexpr int kBufs = TWO ? 2 : 1, kFactors = TWO ? 4 : 2;
  static constexpr uint32_t kTile = kChunkBytes * (D / 64);           // 128 rows x D
  static constexpr uint32_t kHeadChunk = (TWO ? 32 : kHeads) * 128, kHeadTile = kHeadChunk * (D / 64);
  static constexpr uint32_t kOffK = 0, kOffV = 2 * kTile, kOffDs = 4 * kTile;  // dS^T: 128 keys x 64 heads
  // (the product that reads dS has 128 rows: what stands behind its 64 heads is read too and not used)
  static constexpr uint32_t kOffQ = kOffDs + kBufs * kChunkBytes, kOffDo = kOffQ + 2 * kHeadTile;
  static constexpr uint32_t kOffRing = kOffDo + 2 * kHeadTile;
  static constexpr uint32_t kOffStat = kOffRing + kRing * sizeof(Tile);  // [2][64] lse, delta, |dout|, |q|
  static constexpr uint32_t kOffFactor = kOffStat + 2 * kHeads * 16;     // [kFactors][128] factors of a key's shares
  static constexpr uint32_t kOffSum = kOffFactor + kFactors * 128 * 8;  // [2][4][64] sums of p dout.v, of p over a warp's keys
  static constexpr uint32_t kOffTol = kOffSum + 8 * kHeads * 4;         // [2][64] what out's rounding is in delta
  static constexpr uint32_t kOffFit = kOffTol + 2 * kHeads * 4;         // [2] power of two of dS
  static constexpr uint32_t kOffBar = kOffFit + 16;
  static constexpr int kBarQ = 0, kBarQFree = 2, kBarStat = 4, kBarStatFree = 6, kBarK = 8, kBarV = 10, kBarS = 12,
                       kBarKFree = 14, kBarP = 16, kBarD = 18, kBarDFree = 20, kBarDq = 21, kBarDqFree = 22,
                       kBarSum = 23, kBarTile = 24, kBarTileFree = kBarTile + kRing, kBarDone = kBarTileFree + kRing,
                       kBars = kBarDone + 1;
  static constexpr uint32_t kOffMisc = kOffBar + 8 * kBars, kSmem = kOffMisc + 16;
};
template <typename C>
constexpr bool fits_layout() {
  return C::kSmem <= 227 * 1024 && C::kOffRing >= C::kOffDs + (C::kBufs + 1) * kChunkBytes && C::kOffStat % 16 == 0;
}
static_assert(fits_layout<Cfg<128, false>>() && fits_layout<Cfg<128, true>>() && fits_layout<Cfg<64, false>>() &&
                  fits_layout<Cfg<64, true>>(),
              "one CTA per SM; the second half of dS' product stays in bounds; statistics are read 16 bytes at a time");

struct RowsArgs {
  SparseParams p;
  ListArgs l;      // n_z: parts of a key head's query heads
  int heads, padded;  // of a part; the same rounded up to 16
  int s_pad;       // slots of a row's list, rounded up to 128
  float c;         // scale * log2(e)
  const float *delta, *norm_do, *norm_q, *tol;  // [Tq][Hq] (tol: lists of one tile)
  const float* range;  // [Tq][Hk]: the largest |v|^2 of a row's keys (fp16)
  void* share;     // [rows][Hk][n_z][2][s_pad][D] (ShareType)
  uint16_t* power; // [rows][Hk][n_z][s_pad]: the share of dk / scale is its values times 2^(low byte - 143), dv: high byte
  unsigned long long wait_ns;
};

// First head of a key head's part z.  All parts have as many; the last of an odd group begins with the last head of the
// part before, which counts there and weighs nothing here.
__device__ __forceinline__ int first_head(const RowsArgs& f, int z) { return min(z * f.heads, f.p.g - f.heads); }

__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }
// E with x < 2^E for x >= 0, within lo .. hi.
__device__ __forceinline__ int exponent_above(float x, int lo, int hi) {
  return min(max(static_cast<int>((__float_as_uint(x) >> 23) & 255u) - 126, lo), hi);
}

// Sixteen columns of this warp's lanes, requested; and eight written.
__device__ __forceinline__ void tmem_ld16_start(uint32_t taddr, float (&v)[16]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait16(float (&v)[16]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// 32 columns of a warp's 32 rows, each times its lane's f, stored as T: lanes 4 i
// .. 4 i + 3 exchange 16-byte pieces, so that four lanes store 64 bytes of one row.
// Row r goes to dst + r * D where bit r of `rows` is set.  (Streaming stores: what is written is
// read once, much later; 722 -> 716 us and 853 -> 848.)
template <typename T, int D>
__device__ __forceinline__ void store_columns(const float (&o)[32], float f, T* dst, uint32_t rows) {
  const uint32_t lane = lane_id();
#pragma unroll
  for (int h = 0; h < static_cast<int>(sizeof(T)) / 2; ++h) {
    uint4 q[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if constexpr (sizeof(T) == 4) {
        const float* x = o + 16 * h + 4 * u;
        q[u] = make_uint4(__float_as_uint(x[0] * f), __float_as_uint(x[1] * f), __float_as_uint(x[2] * f),
                          __float_as_uint(x[3] * f));
      } else {
        const float* x = o + 8 * u;
        q[u] = make_uint4(pack_pair<T>(x[0] * f, x[1] * f), pack_pair<T>(x[2] * f, x[3] * f),
                          pack_pair<T>(x[4] * f, x[5] * f), pack_pair<T>(x[6] * f, x[7] * f));
      }
    }
    transpose4(q, lane);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t r = (lane & ~3u) + u;
      if ((rows >> r) & 1u) __stcs(reinterpret_cast<uint4*>(dst + static_cast<size_t>(r) * D + 16 * h) + (lane & 3u), q[u]);
    }
  }
}

// ONE: the lists are one tile.  TWO: see Cfg.  Then a tile's scores are formed while the
// tile before is in its softmax, which mends what a row of few heads waits for most: the
// way from P through its products to the next scores (3100 cycles of 4500 a tile).
// (4096 rows of 2 x 16 heads, 16 blocks of 16, window 64: this kernel 348 -> 336 us, where
// its shares go out at 4 TB/s; 517 rows of 2 x 5 heads of 64: 28 -> 24; with one issuer 375 and 23.)
template <typename X, int D, bool ONE, bool TWO>
__global__ void __launch_bounds__(kThreads<TWO>, 1)
    sparse_rows_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_do,
                       const __grid_constant__ RowsArgs f) {
  using C = Cfg<D, TWO>;
  using T = typename ShareType<X>::T;
  extern __shared__ __align__(1024) uint8_t base[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + C::kOffBar);
  Tile* ring = reinterpret_cast<Tile*>(base + C::kOffRing);
  float4* stat = reinterpret_cast<float4*>(base + C::kOffStat);
  float2* factor = reinterpret_cast<float2*>(base + C::kOffFactor);
  float* tols = reinterpret_cast<float*>(base + C::kOffTol);
  int* fits = reinterpret_cast<int*>(base + C::kOffFit);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + C::kOffMisc);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(base + C::kOffMisc + 4);
  const SparseParams& p = f.p;
  const int warp = threadIdx.x / 32;
  const uint32_t lane = lane_id();

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kBars; ++i) {
      int n = 1;
      if (i >= C::kBarK && i < C::kBarV + 2) n = 64;  // every lane that loads
      if (i >= C::kBarStatFree && i < C::kBarStatFree + 2) n = 12;
      if (i == C::kBarP || i == C::kBarP + 1 || i == C::kBarSum) n = 4;
      if (i == C::kBarDFree || i == C::kBarDqFree) n = 8;
      if (i >= C::kBarTileFree && i < C::kBarTileFree + kRing) n = TWO ? 19 : 18;
      if (i == C::kBarDone) n = TWO ? 2 : 1;
      mbar_init(bars + i, n);
    }
    if ((smem_u32(base) & 1023u) != 0u) record_error(kErrDevice);  // the swizzled tiles would be misread
    *abort_flag = 0u;
    fence_mbar_init();
  }
  // rows of no head: the products over heads read them, and the loads leave them as they are
  for (uint32_t i = threadIdx.x; i < 4 * C::kHeadTile / 16; i += kThreads<TWO>)
    reinterpret_cast<uint4*>(base + C::kOffQ)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_shared();
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  constexpr uint32_t kColS = 0, kColDp = TWO ? 32 : 64, kColBuf = TWO ? 64 : 0, kColDv = 128, kColDk = 256, kColDq = 384;
  const WaitCtl ctl{abort_flag, f.wait_ns};
  volatile uint32_t dummy = 0;
  const WaitCtl drain{&dummy, f.wait_ns};  // for what has to be waited for even when a role gave up
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

  if (warp >= kListWarp && warp < kDrain2Warp) {
    list_tiles<kLists>(p, f.l, warp - kListWarp, ring, bars + C::kBarTile, bars + C::kBarTileFree, ctl);
  } else if (warp == kItemWarp) {
    // ------------------------------------------------------------------------- an item's queries, cotangents, statistics
    uint32_t ni = 0;
    bool first = true;
    while (true) {
      const TileHead h = next_head();
      if (h.n < 0) break;
      if (h.n > 0 && first) {
        const uint32_t b = ni & 1u, turn = ((ni >> 1) & 1u) ^ 1u;
        const int own = first_head(f, h.z), head = h.hk * p.g + own, skip = h.z * f.heads - own;
        // on their way while the buffers become free (loaded one behind the other after that, they were what short items
        // waited for: 4096 rows of 8 x 8 heads of 64, 256 entries each, 1229 us; so 1188)
        const long long at = static_cast<long long>(h.t) * p.Hq + head;
        float l[kHeads / 32], de[kHeads / 32], n[kHeads / 32], nq[kHeads / 32], tol[kHeads / 32], range = 0.f;
#pragma unroll
        for (int u = 0; u < kHeads / 32; ++u) {
          const int i = static_cast<int>(lane) + 32 * u;
          l[u] = -INFINITY;
          de[u] = n[u] = nq[u] = tol[u] = 0.f;
          if (i >= skip && i < f.heads) {
            l[u] = p.lse[at + i];
            de[u] = f.delta[at + i];
            n[u] = f.norm_do[at + i];
            nq[u] = f.norm_q[at + i];
            if constexpr (ONE) tol[u] = f.tol[at + i];
          }
        }
        if constexpr (!is_bf16<X>()) range = f.range[static_cast<long long>(h.t) * p.Hk + h.hk];
        if (!bar_wait(bars + C::kBarQFree + b, turn, ctl)) break;
        if (lane == 0) {
          const uint64_t pol = l2_policy_evict_first();
          mbar_arrive_expect_tx(bars + C::kBarQ + b, static_cast<uint32_t>(f.heads) * 256u * (D / 64));
          for (int ch = 0; ch < D / 64; ++ch) {
            tma_load_3d_hint(base + C::kOffQ + b * C::kHeadTile + ch * C::kHeadChunk, &tmap_q, bars + C::kBarQ + b, ch * 64,
                             head, h.t, pol);
            tma_load_3d_hint(base + C::kOffDo + b * C::kHeadTile + ch * C::kHeadChunk, &tmap_do, bars + C::kBarQ + b,
                             ch * 64, head, h.t, pol);
          }
        }
        __syncwarp();
        ++ni;
        if (!bar_wait(bars + C::kBarStatFree + b, turn, ctl)) break;
        float top = 0.f, most = 0.f;  // of |dout|, |delta|
#pragma unroll
        for (int u = 0; u < kHeads / 32; ++u) {
          const int i = static_cast<int>(lane) + 32 * u;
          if (i < f.padded) {
            const bool some = l[u] != -INFINITY;  // else no head, or a row without a weight: P = 0
            if (!some) de[u] = 0.f;
            stat[b * kHeads + i] = some ? make_float4(l[u] * 1.4426950408889634f, de[u], n[u], nq[u])
                                        : make_float4(INFINITY, 0.f, 0.f, 0.f);
            if constexpr (ONE) tols[b * kHeads + i] = tol[u];
            top = fmaxf(top, n[u]);
            most = fmaxf(most, fabsf(de[u]));
          }
        }
        if constexpr (!is_bf16<X>()) {
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
          }
          const float dp = top * sqrtf(range);
          if (lane == 0) fits[b] = 15 - exponent_above(dp + fmaxf(dp, most), -60, 60);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + C::kBarStat + b);
        first = false;
      }
      if (h.last) first = true;
      give_head();
    }
    for (uint32_t i = ni > 2 ? ni - 2 : 0; i < ni; ++i) bar_wait(bars + C::kBarQ + (i & 1u), (i >> 1) & 1u, drain);
  } else if (warp >= kKeyWarp && warp < kMmaWarp) {
    // ------------------------------------------------------------------------- rows of keys, of values
    const bool keys = warp < kValueWarp;
    const int r0 = 64 * (warp & 1);
    const GatherRows& rows = keys ? p.k : p.v;
    uint64_t* full = bars + (keys ? C::kBarK : C::kBarV);
    uint64_t* used = bars + (keys ? C::kBarKFree : C::kBarS);  // a stage is free when the last product that reads it is through
    uint8_t* stages = base + (keys ? C::kOffK : C::kOffV);
    uint32_t j = 0;
    while (true) {
      const TileHead h = next_head();
      if (h.n < 0) break;
      if (h.n > 0) {
        const uint32_t st = j & 1u;
        if (!bar_wait(used + st, ((j >> 1) & 1u) ^ 1u, ctl)) break;
        load_rows<D, 64>(stages + st * C::kTile, rows, keys ? ring[at.slot].k_row : ring[at.slot].v_row, r0, (h.n + 15) & ~15);
        report_rows(full + st);
        ++j;
      }
      give_head();
    }
    wait_rows();  // no copy is in flight when the CTA ends, a role's giving up included
  } else if (warp == kMmaWarp || warp >= kMma2Warp) {
    // ------------------------------------------------------------------------- issuers of the products
    const uint32_t tm = static_cast<uint32_t>(uniform(static_cast<int>(tmem)));
    const uint64_t qd = smem_desc_kmajor(smem_u32(base + C::kOffQ), 128), dod = smem_desc_kmajor(smem_u32(base + C::kOffDo), 128);
    const uint64_t qn = smem_desc_mn_sw128(smem_u32(base + C::kOffQ), C::kHeadChunk, 1024u);
    const uint64_t don = smem_desc_mn_sw128(smem_u32(base + C::kOffDo), C::kHeadChunk, 1024u);
    const uint64_t kd = smem_desc_kmajor(smem_u32(base + C::kOffK), 128), vd = smem_desc_kmajor(smem_u32(base + C::kOffV), 128);
    const uint64_t kn = smem_desc_mn_sw128(smem_u32(base + C::kOffK), kChunkBytes, 1024u);
    const uint64_t ds = smem_desc_mn_sw128(smem_u32(base + C::kOffDs), kChunkBytes, 1024u);
    const uint32_t id_s = idesc_f16<X>(128, f.padded, false);
    constexpr uint32_t kIdD = idesc_f16<X>(128, D, true), kIdDq = idesc_f16<X>(128, D, true) | (1u << 15);  // A MN-major too
    constexpr uint32_t kT = C::kTile >> 4, kH = C::kHeadTile >> 4;
    const int head_steps = uniform(f.padded >> 4);
    bool alive = true, first = true, got_dq = false;
    struct {  // the tile whose P and dS are to come: its last key (0: none), whether it is the item's first; gives dQ
      int n;
      bool first, last;
      uint32_t j, q;  // its number, its item's
    } pend{0, false, false, 0, 0};
    uint32_t j = 0, nq = 0, on = 0;
    auto wait = [&](int bar, uint32_t parity) { alive = alive && bar_wait(bars + bar, parity, ctl); };
    auto scores = [&] {  // S^T, dP^T of tile j, whose rows have been waited for
      const uint32_t st = j & 1u;
      fence_proxy_async_shared();
      tc_fence_after();
      if (elect_one()) {
        if (alive) {
          const uint64_t q = static_cast<uint64_t>((nq & 1u) * kH), t = static_cast<uint64_t>(st * kT);
          const uint32_t to = tm + st * kColBuf;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            umma_bf16(to + kColS, kd + t + static_cast<uint64_t>(((ks >> 2) * kChunkBytes + (ks & 3) * 32) >> 4),
                      qd + q + static_cast<uint64_t>(((ks >> 2) * C::kHeadChunk + (ks & 3) * 32) >> 4), id_s, ks != 0 ? 1u : 0u);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            umma_bf16(to + kColDp, vd + t + static_cast<uint64_t>(((ks >> 2) * kChunkBytes + (ks & 3) * 32) >> 4),
                      dod + q + static_cast<uint64_t>(((ks >> 2) * C::kHeadChunk + (ks & 3) * 32) >> 4), id_s, ks != 0 ? 1u : 0u);
        }
        umma_commit(bars + C::kBarS + st);
      }
      __syncwarp();
    };
    auto shares = [&] {  // dV, dK
      const uint32_t i = pend.j;
      wait(C::kBarP + static_cast<int>(i & 1u), (i >> 1) & 1u);
      wait(C::kBarDFree, (i & 1u) ^ 1u);
      tc_fence_after();
      if (elect_one()) {
        if (alive) {
          const uint64_t o = static_cast<uint64_t>((pend.q & 1u) * kH);
          const uint32_t from = tm + (i & 1u) * kColBuf;
          for (int ks = 0; ks < head_steps; ++ks)
            umma_bf16_tmem_a(tm + kColDv, from + kColS + 8u * ks, don + o + static_cast<uint64_t>(128 * ks), kIdD, ks != 0 ? 1u : 0u);
          for (int ks = 0; ks < head_steps; ++ks)
            umma_bf16_tmem_a(tm + kColDk, from + kColDp + 8u * ks, qn + o + static_cast<uint64_t>(128 * ks), kIdD, ks != 0 ? 1u : 0u);
        }
        umma_commit(bars + C::kBarD + (i & 1u));
      }
      __syncwarp();
    };
    auto take_dq = [&] {
      if (!got_dq) wait(C::kBarDqFree, (on & 1u) ^ 1u);
      got_dq = true;
    };
    auto give_dq = [&](bool any, uint32_t q) {  // the item's dQ is complete, and so is what its queries are read for
      take_dq();
      got_dq = false;
      if (elect_one()) {
        umma_commit(bars + C::kBarDq);
        if (any) umma_commit(bars + C::kBarQFree + (q & 1u));
      }
      __syncwarp();
      ++on;
    };
    auto query = [&] {  // dQ += dS K
      const uint32_t st = pend.j & 1u;
      take_dq();
      tc_fence_after();
      const int steps = (pend.n + 15) >> 4;
      if (elect_one()) {
        if (alive)
          for (int ks = 0; ks < steps; ++ks)
            umma_bf16(tm + kColDq, ds + static_cast<uint64_t>((TWO ? st * (kChunkBytes >> 4) : 0u) + 128 * ks),
                      kn + static_cast<uint64_t>(st * kT + 128 * ks), kIdDq, (!pend.first || ks != 0) ? 1u : 0u);
        umma_commit(bars + C::kBarKFree + st);
      }
      __syncwarp();
      pend.n = 0;
      if (pend.last) give_dq(true, pend.q);
    };
    // One issuer: the products of a tile's P and dS are issued when the next tile has come
    while (alive) {
      const TileHead h = next_head();
      const int n = uniform(h.n), last = uniform(h.last);
      if (n < 0) break;
      give_head();
      const uint32_t st = j & 1u, par = (j >> 1) & 1u;
      if (TWO && warp == kMmaWarp) {
        if (n > 0) {
          if (first) wait(C::kBarQ + static_cast<int>(nq & 1u), (nq >> 1) & 1u);
          wait(C::kBarD + static_cast<int>(st), par ^ 1u);  // P and dS of the tile before the last have been used
          wait(C::kBarK + static_cast<int>(st), par);
          wait(C::kBarV + static_cast<int>(st), par);
          scores();
        }
      } else if (TWO) {
        if (n > 0) {
          pend = {n, first, last != 0, j, nq};
          wait(C::kBarK + static_cast<int>(st), par);
          fence_proxy_async_shared();
          shares();
          query();
        } else if (last != 0) {
          give_dq(!first, nq);
        }
      } else {
        if (n > 0) {
          if (pend.n != 0) {
            shares();  // reads P and dS where the scores will be
            // the next scores go first, unless they would have to wait for their tile
            if (!mbar_look_warp(bars + C::kBarK + st, par) || !mbar_look_warp(bars + C::kBarV + st, par)) query();
          }
          if (first) wait(C::kBarQ + static_cast<int>(nq & 1u), (nq >> 1) & 1u);
          wait(C::kBarK + static_cast<int>(st), par);
          wait(C::kBarV + static_cast<int>(st), par);
          scores();
          if (pend.n != 0) query();
          pend = {n, first, false, j, nq};
        }
        if (last != 0) {
          if (pend.n != 0) {
            shares();
            query();
          }
          give_dq(n > 0 || !first, nq);
        }
      }
      if (n > 0) {
        first = false;
        ++j;
      }
      if (last != 0) {
        if (!first) ++nq;
        first = true;
      }
    }
    if (elect_one()) umma_commit(bars + C::kBarDone);
    __syncwarp();
    bar_wait(bars + C::kBarDone, 0u, drain);
  } else if (warp < kDrainWarp) {
    // ------------------------------------------------------------------------- P and dS: a thread per key
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const int key = warp * 32 + static_cast<int>(lane);
    const float2 c2 = make_float2(f.c, f.c);
    uint32_t j = 0, ni = 0;
    bool first = true;
    float fit = 1.f;        // power of two of dS over that of P
    float back = 1.f, back_v = 1.f;  // what undoes the powers of two
    uint32_t met = 0;
    auto meet_all = [&] {  // these four warps, bounded as every wait is
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + C::kBarSum);
      const bool here = bar_wait(bars + C::kBarSum, met, ctl);
      met ^= 1u;
      return here;
    };
    while (true) {
      const TileHead h = next_head();
      if (h.n < 0) break;
      if (h.n > 0) {
        const uint32_t st = j & 1u;
        if (first) {
          if (!bar_wait(bars + C::kBarStat + (ni & 1u), (ni >> 1) & 1u, ctl)) break;
          if constexpr (!is_bf16<X>()) {
            fit = power_of_two(fits[ni & 1u] - kProbExp<X>);
            back = power_of_two(-fits[ni & 1u]);
            back_v = power_of_two(-kProbExp<X>);
          }
        }
        first = false;
        if (!bar_wait(bars + C::kBarS + st, (j >> 1) & 1u, ctl)) break;
        // the former tile's product with K has read dS (TWO: the one before that has, or K would not be here)
        if (!TWO && j > 0 && !bar_wait(bars + C::kBarKFree + (st ^ 1u), ((j - 1) >> 1) & 1u, ctl)) break;
        tc_fence_after();
        const bool see = (ring[at.slot].keys[warp] >> lane) & 1u;
        uint8_t* row = base + C::kOffDs + (TWO ? st * kChunkBytes : 0u) + key * 128;
        const uint32_t ts = tmem + lanes + kColS + st * kColBuf, td = tmem + lanes + kColDp + st * kColBuf;
        const float4* ls = stat + (ni & 1u) * kHeads;
        if constexpr (ONE) {  // delta, see above
          float* sums = reinterpret_cast<float*>(base + C::kOffSum);
#pragma unroll 1
          for (int i = 0; i < f.padded / 16; ++i) {
            float t[16], dp[16];
            tmem_ld16_start(ts + 16 * i, t);
            tmem_ld16_start(td + 16 * i, dp);
            tmem_wait16(t);
            tmem_wait16(dp);
#pragma unroll
            for (int u = 0; u < 16; ++u) {
              t[u] = see ? exp2_approx(fmaf(t[u], f.c, -ls[16 * i + u].x)) : 0.f;
              dp[u] = see ? t[u] * dp[u] : 0.f;
            }
            // each step adds half of the heads over half of the lanes; lanes 2 h and 2 h + 1 end with head h
#pragma unroll
            for (int n = 8; n > 0; n >>= 1) {
              const bool up = (lane & (2u * n)) != 0u;
#pragma unroll
              for (int u = 0; u < n; ++u) {
                const float give = up ? dp[u] : dp[u + n], keep = up ? dp[u + n] : dp[u];
                const float give2 = up ? t[u] : t[u + n], keep2 = up ? t[u + n] : t[u];
                dp[u] = keep + __shfl_xor_sync(0xffffffffu, give, 2 * n);
                t[u] = keep2 + __shfl_xor_sync(0xffffffffu, give2, 2 * n);
              }
            }
            // (even lanes end with sums of p dP, odd ones with those of p; sums of p by integer reductions took 10 us more)
            const bool odd = (lane & 1u) != 0u;
            const float give = odd ? dp[0] : t[0], keep = odd ? t[0] : dp[0];
            sums[(4 * (lane & 1u) + warp) * kHeads + 16 * i + (lane >> 1)] = keep + __shfl_xor_sync(0xffffffffu, give, 1);
          }
          if (!meet_all()) break;
          if (key < f.heads) {
            auto all = [&](const auto* x) { return (x[0] + x[kHeads]) + (x[2 * kHeads] + x[3 * kHeads]); };
            float4& x = stat[(ni & 1u) * kHeads + key];
            const float sum = all(sums + key), left = fabsf(all(sums + 4 * kHeads + key) - 1.f);
            // the weights add up to 1 within the errors of scores and lse (2^-23 of their size each) and of the sum
            if (left <= 0x1p-16f + 0x1p-21f * fabsf(x.x) && fabsf(sum - x.y) <= tols[(ni & 1u) * kHeads + key]) x.y = sum;
          }
          if (!meet_all()) break;
        }
        float2 bk = make_float2(0.f, 0.f), bv = bk;  // bounds of the key's shares
#pragma unroll 1
        for (int i = 0; i < f.padded / 16; ++i) {
          float s[16], dp[16];
          tmem_ld16_start(ts + 16 * i, s);
          tmem_ld16_start(td + 16 * i, dp);
          tmem_wait16(s);
          tmem_wait16(dp);
          uint32_t pw[8], dw[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const float4 x = ls[16 * i + 2 * u], y = ls[16 * i + 2 * u + 1];  // of two heads
            const float2 e = ffma2(make_float2(s[2 * u], s[2 * u + 1]), c2,
                                   make_float2(static_cast<float>(kProbExp<X>) - x.x, static_cast<float>(kProbExp<X>) - y.x));
            const float2 w = make_float2(exp2_approx(e.x), exp2_approx(e.y));
            float2 d = fmul2(w, fadd2(make_float2(dp[2 * u], dp[2 * u + 1]), make_float2(-x.y, -y.y)));
            if constexpr (!is_bf16<X>()) d = fmul2(d, make_float2(fit, fit));
            bv = ffma2(w, make_float2(x.z, y.z), bv);
            bk = ffma2(make_float2(fabsf(d.x), fabsf(d.y)), make_float2(x.w, y.w), bk);
            pw[u] = see ? pack_pair<X>(w.x, w.y) : 0u;
            dw[u] = see ? pack_pair<X>(d.x, d.y) : 0u;
          }
          tmem_st8(ts + 8 * i, pw);
          tmem_st8(td + 8 * i, dw);
#pragma unroll
          for (int u = 0; u < 2; ++u)
            *reinterpret_cast<uint4*>(row + (((2 * i + u) ^ (key & 7)) * 16)) =
                make_uint4(dw[4 * u], dw[4 * u + 1], dw[4 * u + 2], dw[4 * u + 3]);
        }
        int ek = 15, ev = 15;  // (fp32: as they are)
        if constexpr (sizeof(T) == 2) {
          // (down to where 2^(15 - E) is finite; up to the largest that a byte holds)
          ek = exponent_above((bk.x + bk.y) * back, -110, 127);
          ev = exponent_above((bv.x + bv.y) * back_v, -110, 127);
        }
        factor[(j % C::kFactors) * 128 + key] = make_float2(back * power_of_two(15 - ek), back_v * power_of_two(15 - ev));
        const long long item = (static_cast<long long>(h.t - f.l.t0) * p.Hk + h.hk) * f.l.n_z + h.z;
        f.power[item * f.s_pad + h.c * 128 + key] = static_cast<uint16_t>((ek + 128) | ((ev + 128) << 8));
        tmem_wait_st();
        fence_proxy_async_shared();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + C::kBarP + st);
        ++j;
      }
      if (h.last && !first) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + C::kBarStatFree + (ni & 1u));
        ++ni;
        first = true;
      }
      give_head();
    }
  } else {
    // ------------------------------------------------------------------------- shares of dk, of dv; half of dq each
    const bool dk = warp < kDrain2Warp;
    const int w = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(w * 32) << 16;
    uint32_t j = 0, ni = 0, on = 0;
    bool first = true;
    while (true) {
      const TileHead h = next_head();
      if (h.n < 0) break;
      if (h.n > 0) {
        first = false;
        const uint32_t see = ring[at.slot].keys[w];
        if (!bar_wait(bars + C::kBarD + (j & 1u), (j >> 1) & 1u, ctl)) break;
        tc_fence_after();
        const long long item = (static_cast<long long>(h.t - f.l.t0) * p.Hk + h.hk) * f.l.n_z + h.z;
        T* dst = static_cast<T*>(f.share) + ((2 * item + (dk ? 0 : 1)) * f.s_pad + h.c * 128 + w * 32) * D;
        if (see != 0u) {
          const float2 both = factor[(j % C::kFactors) * 128 + w * 32 + lane];
          const float mine = dk ? both.x : both.y;
#pragma unroll 1
          for (int ch = 0; ch < D / 32; ++ch) {
            float o[32];
            tmem_ld32_start(tmem + lanes + (dk ? kColDk : kColDv) + 32 * ch, o);
            tmem_wait32(o);
            store_columns<T, D>(o, mine, dst + 32 * ch, see);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + C::kBarDFree);
        ++j;
      }
      if (h.last) {
        if (!bar_wait(bars + C::kBarDq, on & 1u, ctl)) break;
        tc_fence_after();
        ++on;
        if (w * 32 < f.heads) {
          float back = p.scale;  // (finite: no inf meets a zero)
          if (!is_bf16<X>() && !first) back = fminf(back * power_of_two(-fits[ni & 1u]), 0x1.fffffep127f);
          const int own = first_head(f, h.z), skip = h.z * f.heads - own;
          const uint32_t rows = low_bits(f.heads - w * 32) & ~low_bits(max(0, skip - w * 32));
          X* dst = static_cast<X*>(p.dq) + (static_cast<long long>(h.t) * p.Hq + h.hk * p.g + own + w * 32) * D;
#pragma unroll 1
          for (int ch = dk ? 0 : D / 64; ch < (dk ? D / 64 : D / 32); ++ch) {
            float o[32];
            tmem_ld32_start(tmem + lanes + kColDq + 32 * ch, o);
            tmem_wait32(o);
            if (first) {
#pragma unroll
              for (int u = 0; u < 32; ++u) o[u] = 0.f;  // no key
            }
            store_columns<X, D>(o, back, dst + 32 * ch, rows);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bars + C::kBarDqFree);
          if (!first) mbar_arrive(bars + C::kBarStatFree + (ni & 1u));
        }
        if (!first) ++ni;
        first = true;
      }
      give_head();
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// ----------------------------------------------------------------- statistics of rows, range of values
// delta = dout.out of each row and head, |dout| and |q|: D/8 lanes a head.  The norms bound the shares whose powers of
// two they give, so they hold over all of bf16's range: squares that leave fp32's (of values below 2^-48 or above 2^48)
// are formed again of the values times a power of two.  tol (where given): 4 u sum |dout||out|, where
// rounding out to X adds at most u sum |dout||out| to delta; the rest is room for the rounded weights.
template <typename X, int D>
__global__ void __launch_bounds__(256) sparse_delta_kernel(const SparseParams p, float* delta, float* norm_do, float* norm_q,
                                                           float* tol) {
  constexpr int G = D / 8;
  constexpr float kLow = 0x1p-96f, kHigh = 0x1p96f, kUp = 0x1p80f, kDown = 0x1p-80f;
  const long long r = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) / G;
  const int l = threadIdx.x % G;
  const bool ok = r < static_cast<long long>(p.Tq) * p.Hq;
  constexpr float kTol = is_bf16<X>() ? 0x1p-6f : 0x1p-9f;
  float d = 0.f, n = 0.f, m = 0.f, s = 0.f;
  uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a, c = a;
  if (ok) {
    const long long t = r / p.Hq, h = r - t * p.Hq;
    a = reinterpret_cast<const uint4*>(static_cast<const X*>(p.dout) + r * D)[l];
    b = reinterpret_cast<const uint4*>(static_cast<const X*>(p.out) + r * D)[l];
    c = reinterpret_cast<const uint4*>(static_cast<const X*>(p.q) + t * p.q_st + h * p.q_sh)[l];
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w}, z[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 u = unpack_pair<X>(x[i]), v = unpack_pair<X>(y[i]), w = unpack_pair<X>(z[i]);
      d = fmaf(u.x, v.x, fmaf(u.y, v.y, d));
      s = fmaf(fabsf(u.x), fabsf(v.x), fmaf(fabsf(u.y), fabsf(v.y), s));
      n = fmaf(u.x, u.x, fmaf(u.y, u.y, n));
      m = fmaf(w.x, w.x, fmaf(w.y, w.y, m));
    }
  }
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) {
    d += __shfl_xor_sync(0xffffffffu, d, o);
    n += __shfl_xor_sync(0xffffffffu, n, o);
    m += __shfl_xor_sync(0xffffffffu, m, o);
    if (tol != nullptr) s += __shfl_xor_sync(0xffffffffu, s, o);
  }
  float back_n = 1.f, back_m = 1.f;
  const bool far = !(n >= kLow && n <= kHigh) || !(m >= kLow && m <= kHigh);
  if (is_bf16<X>() && __any_sync(0xffffffffu, ok && far)) {
    auto again = [&](const uint4& v, float& s, float& back) {
      const float by = s < kLow ? kUp : s <= kHigh ? 1.f : kDown;
      const uint32_t x[4] = {v.x, v.y, v.z, v.w};
      s = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 u = unpack_pair<X>(x[i]);
        s = fmaf(u.x * by, u.x * by, fmaf(u.y * by, u.y * by, s));
      }
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      back = 1.f / by;
    };
    again(a, n, back_n);
    again(c, m, back_m);
  }
  if (ok && l == 0) {
    delta[r] = d;
    norm_do[r] = sqrtf(n) * back_n;
    norm_q[r] = sqrtf(m) * back_m;
    if (tol != nullptr) tol[r] = kTol * s;
  }
}

// The sequence of key t, by one thread: the largest i with cu_k[i] <= t (-1: none).
__device__ __forceinline__ int key_sequence(const SparseParams& p, int t) {
  int lo = 0, hi = p.N;
  if (p.N <= 0 || p.cu_k[0] > t) return -1;
  while (lo < hi) {
    const int i = (lo + hi + 1) >> 1;
    if (p.cu_k[i] <= t)
      lo = i;
    else
      hi = i - 1;
  }
  return lo < p.N ? lo : -1;
}

// norm[key][key head] = |v|^2 over the finite ones of a key's values.  A warp per key.
template <typename X, int D>
__global__ void __launch_bounds__(256) sparse_value_kernel(const SparseParams p, float* norm) {
  const long long w = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) / 32;
  const int lane = threadIdx.x & 31;
  const long long key = w / p.Hk;
  if (key >= p.Tk) return;
  const int hk = static_cast<int>(w - key * p.Hk);
  const X* v = reinterpret_cast<const X*>(
      static_cast<const char*>(p.v.base) +
      static_cast<uint64_t>(key * p.v.rt + static_cast<long long>(hk) * p.v.rh) * p.v.unit_bytes);
  float n = 0.f;
  for (int i = lane; i < D; i += 32) {
    const float x = static_cast<float>(v[i]);
    if (fabsf(x) < INFINITY) n = fmaf(x, x, n);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  if (lane == 0) norm[w] = n;
}
// range[row][key head] = the largest of them over the keys that the row sees: what else its sequence holds does not
// count.  A warp for a row and four key heads, a lane per slot of its list (4096 rows of 256 keys, 8 heads: 11.5 us, a
// warp for each head 32).
__global__ void __launch_bounds__(256) sparse_range_kernel(const SparseParams p, const float* norm, float* range) {
  const int parts = (p.Hk + 3) / 4;
  const long long w = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) / 32, t = w / parts;
  if (t >= p.Tq) return;
  const int lane = threadIdx.x & 31, h0 = 4 * static_cast<int>(w - t * parts);
  const ListRow row = find_list_row(p, load_borders(p), static_cast<int>(t));
  float4 top = make_float4(0.f, 0.f, 0.f, 0.f);
  if (row.lk > 0 && row.pos >= 0) {
    const int slots = p.window + (p.top_k << p.block_shift), lim = min(row.lk - 1, row.pos - p.window);
    const int32_t* list = p.idx + t * p.idx_st;
    const bool four = (p.Hk & 3) == 0;
#pragma unroll 4
    for (int s = lane; s < slots; s += 32) {
      int j = row.pos - s;
      if (s >= p.window) {
        const int b = list[(s - p.window) >> p.block_shift];
        j = -1;
        if (static_cast<unsigned>(b) <= static_cast<unsigned>((row.lk - 1) >> p.block_shift)) {
          const int key = (b << p.block_shift) + ((s - p.window) & ((1 << p.block_shift) - 1));
          if (key <= lim) j = key;
        }
      }
      if (j < 0) continue;
      const float* n = norm + static_cast<long long>(row.k0 + j) * p.Hk + h0;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (four) {
        x = *reinterpret_cast<const float4*>(n);
      } else {
        x.x = n[0];
        if (h0 + 1 < p.Hk) x.y = n[1];
        if (h0 + 2 < p.Hk) x.z = n[2];
        if (h0 + 3 < p.Hk) x.w = n[3];
      }
      top = make_float4(fmaxf(top.x, x.x), fmaxf(top.y, x.y), fmaxf(top.z, x.z), fmaxf(top.w, x.w));
    }
  }
  auto largest = [](float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
  };
  const float all[4] = {largest(top.x), largest(top.y), largest(top.z), largest(top.w)};
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (lane == u && h0 + u < p.Hk) range[t * p.Hk + h0 + u] = all[u];
}

// ----------------------------------------------------------------- who lists a block
// Blocks of all sequences in one numbering: block b of sequence i is number
// (k0 >> shift) + i + b, of n_blocks = (Tk >> shift) + N + 1.
struct WhoArgs {
  SparseParams p;
  int t0, rows;          // rows t0 .. t0 + rows - 1
  int groups, per;       // groups of `per` rows whose counts are kept apart
  int n_blocks;
  int u_bits;            // an entry is (row - t0) << u_bits | place in the row's list
  uint32_t *count, *total, *start, *entry;  // [groups][n_blocks], [n_blocks], [n_blocks + 1], [rows * top_k]
  uint32_t* ticket;                         // zero before sparse_scan_kernel, as the counts
};
// Number of the listed block b of a row, where the row sees some of its keys; -1 else.
__device__ __forceinline__ int listed_block(const SparseParams& p, const ListRow& r, int b) {
  if (r.lk <= 0 || static_cast<unsigned>(b) > static_cast<unsigned>((r.lk - 1) >> p.block_shift)) return -1;
  if ((b << p.block_shift) > static_cast<long long>(r.pos) - p.window) return -1;
  return (r.k0 >> p.block_shift) + r.seq + b;
}
__global__ void __launch_bounds__(256) sparse_count_kernel(const WhoArgs f) {
  const int r = (blockIdx.x * 256 + threadIdx.x) / 32, lane = threadIdx.x & 31;
  if (r >= f.rows) return;
  const ListRow row = find_list_row(f.p, load_borders(f.p), f.t0 + r);
  uint32_t* count = f.count + static_cast<long long>(r / f.per) * f.n_blocks;
  for (int u = lane; u < f.p.top_k; u += 32) {
    const int id = listed_block(f.p, row, f.p.idx[(f.t0 + r) * f.p.idx_st + u]);
    if (id >= 0) atomicAdd(count + id, 1u);
  }
}
// Counts become places within the block's entries.  32 blocks of keys and 32 runs of
// groups per block of threads: each thread adds up its run of groups, the runs before it
// give where it starts.  The last block of threads to be through forms start, the running sum of
// the totals (a launch of its own took 4 us).
__global__ void __launch_bounds__(1024) sparse_scan_kernel(const WhoArgs f) {
  __shared__ uint32_t sums[32][33];
  __shared__ bool last;
  const int tid = threadIdx.x, lane = tid & 31, run = tid / 32, id = blockIdx.x * 32 + lane;
  const int per = (f.groups + 31) / 32, g0 = min(f.groups, run * per), g1 = min(f.groups, g0 + per);
  uint32_t* c = f.count + static_cast<long long>(g0) * f.n_blocks + id;
  uint32_t n = 0, x[kGroups / 32];
#pragma unroll
  for (int g = 0; g < kGroups / 32; ++g)
    x[g] = id < f.n_blocks && g < g1 - g0 ? c[static_cast<long long>(g) * f.n_blocks] : 0u;
#pragma unroll
  for (int g = 0; g < kGroups / 32; ++g) n += x[g];
  sums[run][lane] = n;
  __syncthreads();
  if (id < f.n_blocks) {
    n = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) n += i < run ? sums[i][lane] : 0u;
#pragma unroll
    for (int g = 0; g < kGroups / 32; ++g) {
      if (g < g1 - g0) c[static_cast<long long>(g) * f.n_blocks] = n;
      n += x[g];
    }
    if (run == 31) {
      f.total[id] = n;
      __threadfence();
    }
  }
  __syncthreads();
  if (tid == 0) last = atomicAdd(f.ticket, 1u) == gridDim.x - 1u;
  __syncthreads();
  if (!last) return;
  __threadfence();
  uint32_t before = 0;
  for (int base = 0; base < f.n_blocks; base += 4096) {
    uint32_t x[4], mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = base + 4 * tid + i;
      x[i] = at < f.n_blocks ? __ldcg(f.total + at) : 0u;
      mine += x[i];
    }
    uint32_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) sums[0][run] = upto;
    __syncthreads();
    uint32_t off = before, all = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if (i < run) off += sums[0][i];
      all += sums[0][i];
    }
    upto += off - mine;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = base + 4 * tid + i;
      if (at < f.n_blocks) f.start[at] = upto;
      upto += x[i];
    }
    before += all;
    __syncthreads();
  }
  if (tid == 0) f.start[f.n_blocks] = before;
}
// A block of threads per group takes its rows in order, so that entries of a block
// of keys ascend by row (one listed twice by a row: its two shares are equal).
__global__ void __launch_bounds__(256) sparse_fill_kernel(const WhoArgs f) {
  const int g = blockIdx.x;
  uint32_t* place = f.count + static_cast<long long>(g) * f.n_blocks;
  const int last = min(f.rows, (g + 1) * f.per);
  const Borders border = load_borders(f.p);
  const int u0 = threadIdx.x;
  auto list = [&](int r, int u) { return u < f.p.top_k && r < last ? f.p.idx[(f.t0 + r) * f.p.idx_st + u] : -1; };
  int next = list(g * f.per, u0);  // of the coming row, on its way while this one's places are taken
  for (int r = g * f.per; r < last; ++r) {
    const ListRow row = find_list_row(f.p, border, f.t0 + r);
    const int here = next;
    next = list(r + 1, u0);
    for (int u = u0; u < f.p.top_k; u += 256) {
      const int id = listed_block(f.p, row, u == u0 ? here : list(r, u));
      if (id >= 0) f.entry[f.start[id] + atomicAdd(place + id, 1u)] = (static_cast<uint32_t>(r) << f.u_bits) | u;
    }
    __syncthreads();
  }
}

// ----------------------------------------------------------------- sums of the shares
struct SumArgs {
  SparseParams p;
  int t0, rows, u_bits, n_z, s_pad;
  const uint32_t *start, *entry;
  const void* share;
  const uint16_t* power;
  float* acc;           // [2][Tk][Hk][D]: sums of the rounds before (more than one round), dk's without the scale
  int opens, closes;    // the first round, the last
};

// dk, dv of key blockIdx.x, key head blockIdx.y.  256 shares at a time: each
// thread finds one, with its powers of two, then eight warps add 32 each, four
// values a lane (D = 64: half a warp a share); the warps' sums are joined in order.
template <typename X, int D>
__global__ void __launch_bounds__(256) sparse_sum_kernel(const SumArgs f) {
  using T = typename ShareType<X>::T;
  constexpr int L = D / 4, PER = 32 / L, W = 8 * PER, U = sizeof(T) == 2 ? 8 : 4;  // lanes of a share; shares a warp, a block adds at once; in flight
  struct Found {
    long long at;  // first value of the share of dk; negative: none
    float k, v;    // factors
  };
  __shared__ Found found[256];
  __shared__ float4 red[2][W][L];
  const SparseParams& p = f.p;
  const int key = blockIdx.x, hk = blockIdx.y, tid = threadIdx.x, sub = tid / L, col = (tid % L) * 4;
  float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
  const int seq = key_sequence(p, key);
  SeqExt s{0, 0, 0, 0};
  if (seq >= 0) s = sparse_extent(p, seq);
  const int j = key - s.k0, shift = s.lk - (s.q1 - s.q0) - s.q0;  // position of row t: t + shift
  if (seq >= 0 && j >= 0 && j < s.lk) {
    const int in = j & ((1 << p.block_shift) - 1);
    uint32_t a = 0, n = 0;
    if (p.top_k > 0) {
      const int id = (s.k0 >> p.block_shift) + seq + (j >> p.block_shift);
      a = f.start[id];
      n = f.start[id + 1] - a;
    }
    // rows in whose window the key lies: positions j .. j + window - 1
    const long long first = max(static_cast<long long>(max(s.q0, f.t0)), static_cast<long long>(j) - shift);
    const long long end = min(static_cast<long long>(min(s.q1, f.t0 + f.rows)), static_cast<long long>(j) - shift + p.window);
    const long long near = max(0ll, end - first), all = (static_cast<long long>(n) + near) * f.n_z;
    const long long dv = static_cast<long long>(f.s_pad) * D;  // from a share of dk to that of dv
    for (long long base = 0; base < all; base += 256) {
      Found x{-1, 0.f, 0.f};
      if (base + tid < all) {
        // listed rows first, then those of the window; the groups of heads of a row one after the other
        const long long e = (base + tid) / f.n_z;
        const int z = static_cast<int>(base + tid - e * f.n_z);
        int r, slot;
        bool ok = true;
        if (e < n) {
          const uint32_t entry = f.entry[a + static_cast<uint32_t>(e)];
          r = static_cast<int>(static_cast<uint64_t>(entry) >> f.u_bits);
          slot = p.window + ((entry & ((1u << f.u_bits) - 1u)) << p.block_shift) + in;
          ok = p.causal == 0 || j <= static_cast<long long>(f.t0 + r) + shift - p.window;
        } else {
          const long long t = first + (e - n);
          r = static_cast<int>(t - f.t0);
          slot = static_cast<int>(t + shift) - j;
        }
        if (ok) {
          const long long item = (static_cast<long long>(r) * p.Hk + hk) * f.n_z + z;
          const uint32_t e2 = f.power[item * f.s_pad + slot];
          x.at = 2 * item * dv + static_cast<long long>(slot) * D;
          x.k = power_of_two(static_cast<int>(e2 & 255u) - 143);
          x.v = power_of_two(static_cast<int>(e2 >> 8) - 143);
        }
      }
      __syncthreads();
      found[tid] = x;
      __syncthreads();
      const int most = static_cast<int>(min(256ll, all - base));
#pragma unroll 1
      for (int i = sub; i < most; i += W * U) {
        using Raw = std::conditional_t<sizeof(T) == 2, uint2, uint4>;  // four values
        Raw rk[U], rv[U];
        float fk[U], fv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int at = i + u * W;
          rk[u] = rv[u] = Raw{};
          fk[u] = fv[u] = 0.f;
          if (at < most) {
            const Found y = found[at];
            if (y.at >= 0) {
              const T* src = static_cast<const T*>(f.share) + y.at + col;
              rk[u] = __ldcs(reinterpret_cast<const Raw*>(src));
              rv[u] = __ldcs(reinterpret_cast<const Raw*>(src + dv));
              fk[u] = y.k;
              fv[u] = y.v;
            }
          }
        }
        auto add = [](float4& to, const Raw& r, float by) {
          float2 lo, hi;
          if constexpr (sizeof(T) == 2) {
            lo = unpack_pair<__half>(r.x);
            hi = unpack_pair<__half>(r.y);
          } else {
            lo = make_float2(__uint_as_float(r.x), __uint_as_float(r.y));
            hi = make_float2(__uint_as_float(r.z), __uint_as_float(r.w));
          }
          to.x = fmaf(lo.x, by, to.x);
          to.y = fmaf(lo.y, by, to.y);
          to.z = fmaf(hi.x, by, to.z);
          to.w = fmaf(hi.y, by, to.w);
        };
#pragma unroll
        for (int u = 0; u < U; ++u) {
          add(k, rk[u], fk[u]);
          add(v, rv[u], fv[u]);
        }
      }
    }
  }
  red[0][sub][tid % L] = k;
  red[1][sub][tid % L] = v;
  __syncthreads();
  if (tid >= 2 * L) return;
  const int which = tid / L;
  float4 x = red[which][0][tid % L];
  auto join = [&](const float4& b) {
    x.x += b.x;
    x.y += b.y;
    x.z += b.z;
    x.w += b.w;
  };
#pragma unroll
  for (int i = 1; i < W; ++i) join(red[which][i][tid % L]);
  const long long at = (static_cast<long long>(key) * p.Hk + hk) * D + (tid % L) * 4;
  float* acc = f.acc + which * static_cast<long long>(p.Tk) * p.Hk * D + at;
  if (!f.opens) join(*reinterpret_cast<const float4*>(acc));
  if (!f.closes) {
    *reinterpret_cast<float4*>(acc) = x;
    return;
  }
  if (which == 0) {
    x.x *= p.scale;
    x.y *= p.scale;
    x.z *= p.scale;
    x.w *= p.scale;
  }
  uint2 u;
  u.x = pack_pair<X>(x.x, x.y);
  u.y = pack_pair<X>(x.z, x.w);
  *reinterpret_cast<uint2*>(static_cast<X*>(which ? p.dv : p.dk) + at) = u;
}

// ----------------------------------------------------------------- plan and launches
struct Plan {
  int heads, n_z, s_pad, rows, rounds, groups, per, n_blocks, u_bits;
  size_t norm_do, norm_q, tol, range, count, total, start, entry, power, acc, share, bytes;
};
Plan make_plan(const SparseParams& p, int dtype) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  Plan a;
  const bool fp16 = dtype == CSA_F16;
  a.n_z = (p.g + kHeads - 1) / kHeads;
  a.heads = (p.g + a.n_z - 1) / a.n_z;
  a.s_pad = static_cast<int>((sparse_slots(p) + 127) / 128 * 128);
  const size_t row = static_cast<size_t>(p.Hk) * a.n_z * 2 * a.s_pad * p.D * (fp16 ? 4 : 2);  // bytes of a row's shares
  a.u_bits = 0;
  while ((1ll << a.u_bits) < p.top_k) ++a.u_bits;
  long long rows = row == 0 ? p.Tq : static_cast<long long>(std::max<size_t>(1, kShareBytes / row));
  rows = std::min({rows, static_cast<long long>(p.Tq), 1ll << (32 - a.u_bits)});
  if (p.top_k > 0) rows = std::min(rows, std::max(1ll, 0x7FFFFFFFll / p.top_k));
  a.rows = static_cast<int>(std::max(1ll, rows));
  a.rounds = (p.Tq + a.rows - 1) / a.rows;
  a.rows = (p.Tq + std::max(1, a.rounds) - 1) / std::max(1, a.rounds);  // of equal size
  a.n_blocks = (p.Tk >> p.block_shift) + p.N + 1;
  // sparse_fill_kernel takes a group's rows one after the other, 2 us each; the counts of a group are cleared, added to,
  // read and written once each, 16 bytes for a block of keys, at 6 bytes a ps.  Both cost the same where groups^2 = rows *
  // 750000 / n_blocks.  (Of 16384 rows over 131072 blocks of one key: 308 groups, 110 us each; as many groups as 8 MB of
  // counts hold, 16, would take 2 ms.)  1024 groups fill the SMs (8192 rows, 256 listed entries, with the forward: 863 us, 2048:
  // 895, 304: 870), and 1 GiB of counts is the most there is for them.
  const double even = std::sqrt(static_cast<double>(a.rows) * 750000.0 / a.n_blocks);
  const long long most = std::max(1ll, static_cast<long long>(std::min({even, static_cast<double>(kGroups), 268435456.0 / a.n_blocks})));
  a.per = std::max(1, static_cast<int>((a.rows + most - 1) / most));  // (no rows: one group of none)
  a.groups = (a.rows + a.per - 1) / a.per;
  const size_t per_row = up(static_cast<size_t>(p.Tq) * p.Hq * 4);
  const bool lists = p.top_k > 0;
  a.norm_do = per_row;
  a.norm_q = 2 * per_row;
  a.tol = 3 * per_row;
  a.range = a.tol + (a.s_pad <= 128 ? per_row : 0);
  a.count = up(a.range + (fp16 ? (static_cast<size_t>(p.Tq) + p.Tk) * p.Hk * 4 : 0));  // the norms of keys, and of rows
  a.total = up(a.count + (lists ? (static_cast<size_t>(a.groups) * a.n_blocks + 1) * 4 : 0));  // and the ticket
  a.start = up(a.total + (lists ? static_cast<size_t>(a.n_blocks) * 4 : 0));
  a.entry = up(a.start + (lists ? static_cast<size_t>(a.n_blocks + 1) * 4 : 0));
  a.power = up(a.entry + static_cast<size_t>(a.rows) * p.top_k * 4);
  a.acc = up(a.power + static_cast<size_t>(a.rows) * p.Hk * a.n_z * a.s_pad * 2);
  a.share = a.acc + (a.rounds > 1 ? up(static_cast<size_t>(p.Tk) * p.Hk * p.D * 8) : 0);
  a.bytes = a.share + row * a.rows;
  return a;
}

template <typename X, int D>
cudaError_t run(const SparseParams& p, int dtype, void* workspace, cudaStream_t stream) {
  const Plan a = make_plan(p, dtype);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  constexpr bool fp16 = !is_bf16<X>();
  float* delta = reinterpret_cast<float*>(ws);
  float *norm_v = reinterpret_cast<float*>(ws + a.range), *range = norm_v + static_cast<long long>(p.Tk) * p.Hk;
  cudaError_t e;
  const size_t dkv = static_cast<size_t>(p.Tk) * p.Hk * D * sizeof(X);
  if (p.Tq == 0) {
    if ((e = cudaMemsetAsync(p.dk, 0, dkv, stream)) != cudaSuccess) return e;
    return cudaMemsetAsync(p.dv, 0, dkv, stream);
  }
  const long long rows = static_cast<long long>(p.Tq) * p.Hq, blocks = (rows * (D / 8) + 255) / 256;
  if (blocks > 0x7FFFFFFFll || p.Hk > 65535) return cudaErrorInvalidValue;
  float *norm_do = reinterpret_cast<float*>(ws + a.norm_do), *norm_q = reinterpret_cast<float*>(ws + a.norm_q);
  float* tol = a.s_pad <= 128 ? reinterpret_cast<float*>(ws + a.tol) : nullptr;
  sparse_delta_kernel<X, D><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(p, delta, norm_do, norm_q, tol);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (fp16 && p.N > 0 && p.Tk > 0) {
    const long long nk = (static_cast<long long>(p.Tk) * p.Hk + 7) / 8, nq = (static_cast<long long>(p.Tq) * ((p.Hk + 3) / 4) + 7) / 8;
    if (nk > 0x7FFFFFFFll || nq > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    sparse_value_kernel<X, D><<<static_cast<unsigned>(nk), 256, 0, stream>>>(p, norm_v);
    sparse_range_kernel<<<static_cast<unsigned>(nq), 256, 0, stream>>>(p, norm_v, range);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  RowsArgs f;
  f.p = p;
  f.l.n_z = a.n_z;
  f.l.split = 0;
  f.l.slots = static_cast<int>(sparse_slots(p));
  f.l.per = std::max(1, a.s_pad / 128);
  f.heads = a.heads;
  f.padded = (a.heads + 15) / 16 * 16;
  f.s_pad = a.s_pad;
  f.c = p.scale * 1.4426950408889634f;
  f.delta = delta;
  f.norm_do = norm_do;
  f.norm_q = norm_q;
  f.tol = tol;
  f.range = range;
  f.share = ws + a.share;
  f.power = reinterpret_cast<uint16_t*>(ws + a.power);
  f.wait_ns = attn_wait_ns(f.l.slots / 128 + 1);
  CUtensorMap tq, tdo;
  if (!make_heads_map(&tq, p, p.q, p.q_st, p.q_sh, a.heads) ||
      !make_heads_map(&tdo, p, p.dout, static_cast<long long>(p.Hq) * D, D, a.heads))
    return cudaErrorInvalidValue;
  const bool one = f.l.per == 1;
  void (*kernel)(CUtensorMap, CUtensorMap, RowsArgs) = nullptr;
  uint32_t smem = 0, threads = 0;
  const bool two = f.padded <= 32;
  auto take = [&](auto k1, auto k2) {
    constexpr bool ONE = decltype(k1)::value, TWO = decltype(k2)::value;
    constexpr auto k = sparse_rows_kernel<X, D, ONE, TWO>;
    kernel = k;
    smem = Cfg<D, TWO>::kSmem;
    threads = kThreads<TWO>;
    return smem_limit_once<k>(smem);
  };
  constexpr std::true_type yes;
  constexpr std::false_type no;
  e = one ? (two ? take(yes, yes) : take(yes, no)) : (two ? take(no, yes) : take(no, no));
  if (e != cudaSuccess) return e;
  WhoArgs who;
  who.p = p;
  who.per = a.per;
  who.n_blocks = a.n_blocks;
  who.u_bits = a.u_bits;
  who.count = reinterpret_cast<uint32_t*>(ws + a.count);
  who.total = reinterpret_cast<uint32_t*>(ws + a.total);
  who.start = reinterpret_cast<uint32_t*>(ws + a.start);
  who.entry = reinterpret_cast<uint32_t*>(ws + a.entry);
  SumArgs sum;
  sum.p = p;
  sum.u_bits = a.u_bits;
  sum.n_z = a.n_z;
  sum.s_pad = a.s_pad;
  sum.start = who.start;
  sum.entry = who.entry;
  sum.share = f.share;
  sum.power = f.power;
  sum.acc = reinterpret_cast<float*>(ws + a.acc);
  for (int i = 0; i < a.rounds; ++i) {
    const int t0 = i * a.rows, n = std::min(a.rows, p.Tq - t0);
    f.l.t0 = who.t0 = sum.t0 = t0;
    who.rows = sum.rows = n;
    who.groups = (n + a.per - 1) / a.per;
    f.l.items = static_cast<long long>(n) * p.Hk * a.n_z;
    if (p.Tk > 0 && p.top_k > 0) {
      const size_t counts = static_cast<size_t>(who.groups) * a.n_blocks;
      who.ticket = who.count + counts;
      if ((e = cudaMemsetAsync(who.count, 0, (counts + 1) * 4, stream)) != cudaSuccess) return e;
      sparse_count_kernel<<<static_cast<unsigned>((static_cast<long long>(n) * 32 + 255) / 256), 256, 0, stream>>>(who);
      sparse_scan_kernel<<<(a.n_blocks + 31) / 32, 1024, 0, stream>>>(who);
      sparse_fill_kernel<<<who.groups, 256, 0, stream>>>(who);
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    const long long grid = std::min(f.l.items, 152ll);
    set_step(f.l, p.Hk, grid);
    kernel<<<static_cast<unsigned>(grid), threads, smem, stream>>>(tq, tdo, f);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (p.Tk == 0) continue;
    sum.opens = i == 0;
    sum.closes = i + 1 == a.rounds;
    sparse_sum_kernel<X, D><<<dim3(static_cast<unsigned>(p.Tk), static_cast<unsigned>(p.Hk)), 256, 0, stream>>>(sum);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t sparse_backward_workspace(const SparseParams& p, int dtype) { return make_plan(p, dtype).bytes; }

cudaError_t launch_sparse_backward(const SparseParams& p, int dtype, void* workspace, cudaStream_t s) {
  if (dtype == CSA_BF16)
    return p.D == 128 ? run<__nv_bfloat16, 128>(p, dtype, workspace, s) : run<__nv_bfloat16, 64>(p, dtype, workspace, s);
  return p.D == 128 ? run<__half, 128>(p, dtype, workspace, s) : run<__half, 64>(p, dtype, workspace, s);
}

cudaError_t take_status_sparse_bwd(uint32_t* out, cudaStream_t stream) { return take_status(out, stream); }

}  // namespace csa
