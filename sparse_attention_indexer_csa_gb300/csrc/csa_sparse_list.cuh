// csa_sparse_list.cuh -- what the kernels of attention over listed blocks share:
// the keys that a row lists, and the maps of its queries.
#pragma once

#include "csa_attn_tiles.cuh"
#include "csa_sparse_internal.h"

namespace csa {

// ----------------------------------------------------------------- TMA maps (host)
// Heads of q (or dout): dims (D, Hq, Tq), box {64, heads, 1}.
inline bool make_heads_map(CUtensorMap* m, const SparseParams& p, const void* x, long long st, long long sh, int heads) {
  auto fn = attn_encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[3] = {(cuuint64_t)p.D, (cuuint64_t)p.Hq, (cuuint64_t)p.Tq};
  cuuint64_t strides[2] = {(cuuint64_t)sh * 2, (cuuint64_t)st * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)heads, 1}, estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(x), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// ----------------------------------------------------------------- lists
// The sequence of a query row: keys k0 .. k0+lk-1 (counted from 0 in a paged
// cache), the row's position, the sequence's number (-1: none, lk = 0).
struct ListRow {
  int seq, k0, lk, pos;
};

// Extents of sequence i, clamped to the tensors; what was clamped is recorded.
__device__ __forceinline__ SeqExt sparse_extent(const SparseParams& p, int i) {
  SeqExt s;
  const int a = p.cu_q[i], b = p.cu_q[i + 1];
  s.q0 = min(max(a, 0), p.Tq);
  s.q1 = min(max(b, s.q0), p.Tq);
  bool bad = a != s.q0 || b != s.q1;
  long long most;
  if (p.page > 0) {
    s.k0 = 0;
    most = static_cast<long long>(p.table_width) * p.page;
  } else {
    const int c = p.cu_k[i], d = p.cu_k[i + 1];
    s.k0 = min(max(c, 0), p.Tk);
    const int k1 = min(max(d, s.k0), p.Tk);
    bad |= c != s.k0 || d != k1;
    most = k1 - s.k0;
  }
  s.lk = static_cast<int>(min(most, 0x7FFFFFFFll));
  if (p.k_len != nullptr) {
    const int n = p.k_len[i], m = min(max(n, 0), s.lk);
    bad |= n != m;
    s.lk = m;
  }
  if (bad) record_error(kErrDevice);
  return s;
}

// The row's sequence, by a warp: the largest i with cu_q[i] <= t.  Sequences of
// equal lengths (one token each, when decoding) are met at the first look, others
// by 32 probes at a time.  Entries out of order give some sequence or none.
__device__ __forceinline__ ListRow find_list_row(const SparseParams& p, int t) {
  const int lane = static_cast<int>(lane_id());
  ListRow r{-1, 0, 0, -1};
  if (p.N <= 0) return r;
  int lo = static_cast<int>(static_cast<long long>(t) * p.N / p.Tq);
  if (t < p.cu_q[lo] || t >= p.cu_q[lo + 1]) {
    lo = 0;
    int hi = p.N;
    while (lo < hi) {
      const int span = hi - lo, stride = (span + 31) / 32;
      const int i = lo + min(span, (lane + 1) * stride);
      const unsigned out = __ballot_sync(0xffffffffu, p.cu_q[i] > t);
      if (out == 0u) {
        lo = hi;
      } else {
        const int n = __ffs(static_cast<int>(out)) - 1;
        hi = lo + min(span, (n + 1) * stride) - 1;
        lo = lo + min(span, n * stride);
      }
    }
    if (lo >= p.N) return r;
  }
  const SeqExt s = sparse_extent(p, lo);
  if (t < s.q0 || t >= s.q1) return r;
  r.seq = lo;
  r.k0 = s.k0;
  r.lk = s.lk;
  r.pos = p.causal ? t - s.q0 + s.lk - (s.q1 - s.q0) : s.lk - 1;
  return r;
}

// The slots of a row's list: first the window, newest key first, then top_k
// blocks.  A slot in three steps, so that the loads of the coming slots are in
// flight while the present ones are dealt with.  `bad` gathers what is out of range.
struct Slot {
  int j;     // key of the sequence; -1: none
  int page;  // its page (paged keys)
};
__device__ __forceinline__ int slot_block(const SparseParams& p, const int32_t* list, int s, int slots) {
  return s >= p.window && s < slots ? list[(s - p.window) >> p.block_shift] : -1;
}
__device__ __forceinline__ Slot slot_key(const SparseParams& p, const ListRow& r, int s, int slots, int b, bool& bad) {
  Slot x{-1, 0};
  if (s < p.window) {
    x.j = r.pos - s;  // negative: before the first key
  } else if (s < slots) {
    if (static_cast<unsigned>(b) <= static_cast<unsigned>((r.lk - 1) >> p.block_shift)) {
      const int j = (b << p.block_shift) + ((s - p.window) & ((1 << p.block_shift) - 1));
      if (j < r.lk && j <= r.pos - p.window) x.j = j;
    } else {
      bad |= b != -1;
    }
  }
  if (p.page > 0 && x.j >= 0) x.page = p.table[r.seq * p.table_st + x.j / p.page];
  return x;
}
// Rows of keys and values of slot x (key head 0); false: it has none.
__device__ __forceinline__ bool slot_rows(const SparseParams& p, const ListRow& r, const Slot& x, int& kr, int& vr,
                                          bool& bad) {
  if (x.j < 0) return false;
  if (p.page > 0) {
    if (static_cast<unsigned>(x.page) >= static_cast<unsigned>(p.pages)) {
      bad = true;
      return false;
    }
    const int off = x.j % p.page;
    kr = x.page * p.k.rp + off * p.k.rt;
    vr = x.page * p.v.rp + off * p.v.rt;
  } else {
    kr = (r.k0 + x.j) * p.k.rt;
    vr = (r.k0 + x.j) * p.v.rt;
  }
  return true;
}

constexpr int kLists = 2, kRing = 8;  // warps that write lists; tiles of rows ahead

// What the CTAs of a launch walk: items blockIdx.x + n gridDim.x, an item being
// row t0 + item / (n_z Hk), a key head and one of n_z parts.
struct ListArgs {
  long long items;
  int t0, n_z;
  int split;        // the parts are shares of the row's list (tiles z, z + n_z, ..); else all have the whole list
  int slots, per;   // of a row's list; its tiles (of an item)
};

// 128 slots of an item's list: the rows of those that are keys (-1: none), a bit
// for each of them, and n: one more than the last of them (0: none).  A hidden or
// empty slot keeps its place, as lists have few of them but at the end.
struct TileHead {
  int n, last, t, hk, z, c, seq;  // last: the item's last tile; c: its place in the row's list; n < 0: no more tiles
};
struct Tile {
  int k_row[128], v_row[128];
  uint32_t keys[4];
  TileHead h;
  int pad[1];
};

static_assert(sizeof(Tile) % 16 == 0, "tiles of a ring");

// As mbar_wait, its slow part out of line: sixteen warps in seven roles run here,
// and what they wait for is instructions.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, const WaitCtl& ctl) {
  return mbar_wait_u32(smem_u32(bar), parity, ctl);
}

// The tiles of a CTA: items blockIdx.x + n gridDim.x, `per` tiles each.
__device__ __forceinline__ long long tile_count(const ListArgs& f) {
  return (f.items - blockIdx.x + gridDim.x - 1) / gridDim.x * f.per;
}

// Writes the tiles w, w + kLists, .. of this CTA into the ring.  A warp.
__device__ __forceinline__ void list_tiles(const SparseParams& p, const ListArgs& f, int w, Tile* ring, uint64_t* full, uint64_t* free_bar,
                                           const WaitCtl& ctl) {
  const int lane = static_cast<int>(lane_id());
  bool bad = false;
  if (blockIdx.x == 0 && w == 0)
    for (int i = lane; i < p.N; i += 32) sparse_extent(p, i);  // what is out of order or range is recorded
  const long long tiles = tile_count(f);
  // the coming tile: its item, its place in the item, its row and the blocks that its slots list
  long long item = blockIdx.x + static_cast<long long>(w / f.per) * gridDim.x;
  int at = w % f.per, t = 0, hk = 0, z = 0, b[4];
  auto tile = [&] { return f.split ? at * f.n_z + z : at; };
  auto blocks = [&] {
    const long long rest = item / f.n_z, token = rest / p.Hk;
    z = static_cast<int>(item - rest * f.n_z);
    t = f.t0 + static_cast<int>(token);
    hk = static_cast<int>(rest - token * p.Hk);
    const int32_t* list = p.idx + t * p.idx_st;
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = slot_block(p, list, tile() * 128 + 32 * i + lane, f.slots);
  };
  ListRow row{-1, 0, 0, -1};
  int row_t = -1;
  if (w < tiles) blocks();
  for (long long n = w; n < tiles; n += kLists) {
    const uint32_t st = static_cast<uint32_t>(n % kRing), turn = static_cast<uint32_t>(n / kRing) & 1u;
    if (t != row_t) row = find_list_row(p, t);
    row_t = t;
    Slot x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = Slot{-1, 0};
      if (row.lk > 0 && row.pos >= 0)
        x[i] = slot_key(p, row, tile() * 128 + 32 * i + lane, f.slots, b[i], bad);
    }
    TileHead h{0, at == f.per - 1, t, hk, z, tile(), row.seq};
    const int k0 = hk * p.k.rh, v0 = hk * p.v.rh;
    at += kLists;
    while (at >= f.per) {
      at -= f.per;
      item += gridDim.x;
    }
    if (n + kLists < tiles) blocks();
    if (!bar_wait(free_bar + st, turn ^ 1u, ctl)) break;
    uint32_t mine = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int kr = 0, vr = 0;
      const bool see = slot_rows(p, row, x[i], kr, vr, bad);
      const unsigned all = __ballot_sync(0xffffffffu, see);
      if (all != 0u) h.n = 32 * i + 32 - __clz(static_cast<int>(all));
      if (lane == i) mine = all;
      ring[st].k_row[32 * i + lane] = see ? kr + k0 : -1;
      ring[st].v_row[32 * i + lane] = see ? vr + v0 : -1;
    }
    if (lane < 4) ring[st].keys[lane] = mine;
    if (lane == 0) ring[st].h = h;
    __syncwarp();
    if (lane == 0) mbar_arrive(full + st);
  }
  if (bad) record_error(kErrDevice);
}

// 64 rows of a tile (from row r0 on, as far as n of the tile) by a warp.  Whole
// stretches go without a branch or a size of their own, eight copies in a row: a
// copy that waits for its registers' former use takes 140 cycles instead of 40.
template <int D>
__device__ __forceinline__ void load_rows(uint8_t* tile, const GatherRows& g, const int* rows, int r0, int n) {
  constexpr int P = D / 8, PER = 32 / P;  // 16-byte pieces of a row; rows an instruction takes
  const int lane = static_cast<int>(lane_id());
  const int mine[2] = {r0 + lane < n ? rows[r0 + lane] : -1, r0 + 32 + lane < n ? rows[r0 + 32 + lane] : -1};
  const int piece = lane % P, sub = lane / P;
  const char* base = static_cast<const char*>(g.base) + piece * 16;
  const uint32_t dst = smem_u32(tile) + (piece >> 3) * kChunkBytes + (r0 + sub) * 128;
  uint32_t at[8 / PER];  // the swizzle repeats every eight rows
#pragma unroll
  for (int i = 0; i < 8 / PER; ++i) at[i] = dst + (((piece & 7) ^ ((PER * i + sub) & 7)) * 16);
  if (__all_sync(0xffffffffu, (mine[0] | mine[1]) >= 0)) {
#pragma unroll 1
    for (int h = 0; h < 64; h += 8 * PER) {
      const char* src[8];
      const int from = h < 32 ? mine[0] : mine[1];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = __shfl_sync(0xffffffffu, from, (h + PER * i + sub) & 31);
        src[i] = base + static_cast<uint64_t>(static_cast<uint32_t>(row)) * g.unit_bytes;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at[i % (8 / PER)] + (h + PER * i) * 128), "l"(src[i])
                     : "memory");
    }
  } else {
#pragma unroll 1
    for (int i = 0; i < 64 / PER && r0 + PER * i < n; ++i) {  // n is a multiple of 16
      const int r = PER * i + sub;
      const int row = __shfl_sync(0xffffffffu, PER * i < 32 ? mine[0] : mine[1], r & 31);
      const char* src = base + static_cast<uint64_t>(static_cast<uint32_t>(max(row, 0))) * g.unit_bytes;
      const uint32_t to = dst + PER * i * 128 + (((piece & 7) ^ (r & 7)) * 16);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src), "r"(row < 0 ? 0 : 16) : "memory");
    }
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void loaded() {  // all but the last N groups of rows are there, for the tensor cores too
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
  fence_proxy_async_shared();
  __syncwarp();
}

}  // namespace csa
