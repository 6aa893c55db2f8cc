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
  int q0, q1;  // the sequence's rows
};

// Extents of a sequence with rows a .. b-1, keys c .. d-1 and n of them (where given),
// clamped to the tensors; `bad` where anything was.
__device__ __forceinline__ SeqExt clamp_extent(const SparseParams& p, int a, int b, int c, int d, int n, bool& bad) {
  SeqExt s;
  s.q0 = min(max(a, 0), p.Tq);
  s.q1 = min(max(b, s.q0), p.Tq);
  bad |= a != s.q0 || b != s.q1;
  long long most;
  if (p.page > 0) {
    s.k0 = 0;
    most = static_cast<long long>(p.table_width) * p.page;
  } else {
    s.k0 = min(max(c, 0), p.Tk);
    const int k1 = min(max(d, s.k0), p.Tk);
    bad |= c != s.k0 || d != k1;
    most = k1 - s.k0;
  }
  s.lk = static_cast<int>(min(most, 0x7FFFFFFFll));
  if (p.k_len != nullptr) {
    const int m = min(max(n, 0), s.lk);
    bad |= n != m;
    s.lk = m;
  }
  return s;
}
// Those of sequence i; what was clamped is recorded.
__device__ __forceinline__ SeqExt sparse_extent(const SparseParams& p, int i) {
  bool bad = false;
  const SeqExt s = clamp_extent(p, p.cu_q[i], p.cu_q[i + 1], p.page > 0 ? 0 : p.cu_k[i], p.page > 0 ? 0 : p.cu_k[i + 1],
                                p.k_len != nullptr ? p.k_len[i] : 0, bad);
  if (bad) record_error(kErrDevice);
  return s;
}

// Borders and lengths of up to 31 sequences, a lane each, read once: rows of several
// sequences in turn would wait for them three times over (1021 rows in 13
// sequences: 41.8 us, so 38.4).
struct Borders {
  int q, k, n;
};
__device__ __forceinline__ Borders load_borders(const SparseParams& p) {
  Borders b{0, 0, 0};
  const int lane = static_cast<int>(lane_id());
  if (p.N > 0 && p.N <= 31) {
    b.q = p.cu_q[min(lane, p.N)];
    if (p.page == 0) b.k = p.cu_k[min(lane, p.N)];
    if (p.k_len != nullptr && lane < p.N) b.n = p.k_len[lane];
  }
  return b;
}

// By 32 probes at a time.
__device__ __forceinline__ int find_far(const SparseParams& p, int t) {
  const int lane = static_cast<int>(lane_id());
  int lo = 0, hi = p.N;
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
  return lo;
}
// The row's sequence, by a warp: the largest i with cu_q[i] <= t.  More than 31
// sequences of equal lengths (one token each, when decoding) are met at the first look,
// others are searched.  Entries out of order give some sequence or none.
__device__ __forceinline__ ListRow find_list_row(const SparseParams& p, const Borders& border, int t) {
  const int lane = static_cast<int>(lane_id());
  ListRow r{-1, 0, 0, -1, 0, 0};
  if (p.N <= 0) return r;
  int lo;
  SeqExt s;
  if (p.N <= 31) {
    const int next = __shfl_down_sync(0xffffffffu, border.q, 1);
    const unsigned in = __ballot_sync(0xffffffffu, lane < p.N && border.q <= t && t < next);
    if (in == 0u) return r;
    lo = 31 - __clz(static_cast<int>(in));
    auto of = [&](int x, int i) { return __shfl_sync(0xffffffffu, x, i); };
    bool bad = false;  // (recorded for all sequences at once)
    s = clamp_extent(p, of(border.q, lo), of(border.q, lo + 1), of(border.k, lo), of(border.k, lo + 1), of(border.n, lo), bad);
  } else {
    lo = static_cast<int>(static_cast<long long>(t) * p.N / p.Tq);
    if (t < p.cu_q[lo] || t >= p.cu_q[lo + 1]) lo = find_far(p, t);
    if (lo >= p.N) return r;
    s = sparse_extent(p, lo);
  }
  if (t < s.q0 || t >= s.q1) return r;
  r.seq = lo;
  r.q0 = s.q0;
  r.q1 = s.q1;
  r.k0 = s.k0;
  r.lk = s.lk;
  r.pos = p.causal ? t - s.q0 + s.lk - (s.q1 - s.q0) : s.lk - 1;
  return r;
}

// The slots of a row's list: first the window, newest key first, then top_k
// blocks.  Slot s's block (-1: none).
__device__ __forceinline__ int slot_block(const SparseParams& p, const int32_t* list, int s, int slots) {
  return s >= p.window && s < slots ? list[(s - p.window) >> p.block_shift] : -1;
}
// The page of key j >= 0 of a sequence: j * ceil(2^n / page) / 2^n with 2^(n - 31) >= page, which is exact below 2^31.
__device__ __forceinline__ int page_of(const SparseParams& p, int j) {
  return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(j)) * p.page_mul) >> p.page_shift);
}

constexpr int kRing = 8;  // tiles of rows ahead

// What the CTAs of a launch walk: items blockIdx.x + n gridDim.x, an item being
// row t0 + item / (n_z Hk), a key head and one of n_z parts.
struct ListArgs {
  long long items;
  int t0, n_z;
  int split;        // the parts are shares of the row's list (tiles z, z + n_z, ..); else all have the whole list
  int slots, per;   // of a row's list; its tiles (of an item)
  int dt, dh, dz;   // from an item to the CTA's next one: gridDim.x in rows, key heads and parts
};
inline void set_step(ListArgs& l, int Hk, long long grid) {
  l.dz = static_cast<int>(grid % l.n_z);
  l.dh = static_cast<int>(grid / l.n_z % Hk);
  l.dt = static_cast<int>(grid / l.n_z / Hk);
}

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

// As mbar_wait, its slow part out of line (twenty warps and more in seven roles
// run here, and what they wait for is instructions), and without a time for which
// the thread may be suspended: a thread that gives one comes back later.
static __device__ __noinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity, const WaitCtl& ctl) {
  uint64_t t0 = 0;
  for (uint32_t n = 1;; ++n) {
    if (mbar_try_wait_u32(bar, parity)) return true;
    if (*ctl.abort_flag) return false;
    if ((n & 15u) == 0u) {
      const uint64_t t = globaltimer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > ctl.limit_ns) {
        *ctl.abort_flag = 1u;
        record_error(kErrTimeout);
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, const WaitCtl& ctl) {
  return mbar_try_wait_u32(smem_u32(bar), parity) || bar_wait_slow(smem_u32(bar), parity, ctl);
}

// The items and tiles of a CTA: items blockIdx.x + n gridDim.x, `per` tiles each.
__device__ __forceinline__ long long item_count(const ListArgs& f) {
  return (f.items - blockIdx.x + gridDim.x - 1) / gridDim.x;
}
__device__ __forceinline__ long long tile_count(const ListArgs& f) { return item_count(f) * f.per; }

// A role's place in the ring of tiles.
struct Place {
  long long left;  // tiles to come
  uint32_t slot = 0, parity = 0;
  __device__ __forceinline__ explicit Place(const ListArgs& f) : left(tile_count(f)) {}
  __device__ __forceinline__ void next() {
    --left;
    slot = (slot + 1u) & (kRing - 1u);
    if (slot == 0u) parity ^= 1u;
  }
};
static_assert((kRing & (kRing - 1)) == 0, "Place");

// Writes the tiles w, w + LISTS, .. of this CTA into the ring.  A warp; a lane has
// four consecutive slots, whose keys follow one another where blocks and window
// allow it (one block, one page for the four).  A list warp must keep up with the
// tensor cores: with a block, a page and 64-bit divisions for each slot, two of them
// took 1700 cycles a tile, all that a prompt of 8192 tokens had.
template <int LISTS>
__device__ __forceinline__ void list_tiles(const SparseParams& p, const ListArgs& f, int w, Tile* ring, uint64_t* full,
                                           uint64_t* free_bar, const WaitCtl& ctl) {
  const int lane = static_cast<int>(lane_id());
  bool bad = false;
  if (w == 0)  // what is out of order or range is recorded, also of sequences without rows
    for (long long i = blockIdx.x * 32 + lane; i < p.N; i += 32 * gridDim.x) sparse_extent(p, static_cast<int>(i));
  const long long tiles = tile_count(f);
  const bool quads = p.block_shift >= 2 && (p.window & 3) == 0 && (p.page == 0 || ((p.page & 3) == 0 && p.window == 0));
  // the coming tile: its row, key head and part, its place in the item, the blocks that its slots list
  int at = w % f.per, t, hk, z, b[4];
  {
    const long long item = blockIdx.x + static_cast<long long>(w / f.per) * gridDim.x, rest = item / f.n_z, token = rest / p.Hk;
    z = static_cast<int>(item - rest * f.n_z);
    hk = static_cast<int>(rest - token * p.Hk);
    t = f.t0 + static_cast<int>(token);
  }
  auto tile = [&] { return f.split ? at * f.n_z + z : at; };
  auto blocks = [&] {
    const int32_t* list = p.idx + t * p.idx_st;
    const int s = tile() * 128 + 4 * lane;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i == 0 || !quads) b[i] = slot_block(p, list, s + i, f.slots);
  };
  ListRow row{-1, 0, 0, -1, 0, 0};
  const Borders border = load_borders(p);
  if (w < tiles) blocks();
  uint32_t st = static_cast<uint32_t>(w) % kRing, turn = static_cast<uint32_t>(w) / kRing & 1u;
  for (long long n = w; n < tiles; n += LISTS) {
    if (t >= row.q0 && t < row.q1)  // mostly the sequence of the row before
      row.pos = p.causal ? t - row.q0 + row.lk - (row.q1 - row.q0) : row.lk - 1;
    else
      row = find_list_row(p, border, t);
    TileHead h{0, at == f.per - 1, t, hk, z, tile(), row.seq};
    const int s = h.c * 128 + 4 * lane, k0 = hk * p.k.rh, v0 = hk * p.v.rh;
    int kr[4], vr[4];
    uint32_t see = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) kr[i] = vr[i] = -1;
    if (row.lk > 0 && row.pos >= 0) {
      if (quads) {
        int j = 0, first = 0, last = 0, step = 1;  // slot i is key j + i * step where first <= i < last
        if (s < p.window) {
          j = row.pos - s;
          last = j + 1;
          step = -1;
        } else if (s < f.slots) {
          if (static_cast<unsigned>(b[0]) <= static_cast<unsigned>((row.lk - 1) >> p.block_shift)) {
            j = (b[0] << p.block_shift) + ((s - p.window) & ((1 << p.block_shift) - 1));
            last = min(row.lk, row.pos - p.window + 1) - j;
          } else {
            bad |= b[0] != -1;
          }
        }
        int kb = row.k0 + j, vb = kb;
        if (p.page > 0) {
          kb = vb = 0;
          if (last > 0) {
            const int n_page = page_of(p, j), pg = p.table[row.seq * p.table_st + n_page], off = j - n_page * p.page;
            if (static_cast<unsigned>(pg) >= static_cast<unsigned>(p.pages)) {
              bad = true;
              last = 0;
            } else {
              kb = pg * p.k.rp + off * p.k.rt;
              vb = pg * p.v.rp + off * p.v.rt;
            }
          }
        } else {
          kb *= p.k.rt;
          vb *= p.v.rt;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i >= first && i < last) {
            kr[i] = kb + i * step * p.k.rt + k0;
            vr[i] = vb + i * step * p.v.rt + v0;
            see |= 1u << i;
          }
      } else {
        // straight on, a select for each border: branches for each slot took 2000 cycles a tile (38.4 us for 33.3, as above)
        const int lim = min(row.lk - 1, row.pos - p.window), mask = (1 << p.block_shift) - 1;
        const unsigned most = static_cast<unsigned>((row.lk - 1) >> p.block_shift);
        int j[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool listed = static_cast<unsigned>(b[i]) <= most;
          const int key = static_cast<int>(static_cast<unsigned>(b[i]) << p.block_shift) + ((s + i - p.window) & mask);
          bad |= !listed && b[i] != -1;
          j[i] = listed && key <= lim ? key : -1;
          if (s + i < p.window) j[i] = row.pos - s - i;
        }
        if (p.page > 0) {
          const int32_t* table = p.table + row.seq * p.table_st;
          int n_page[4], pg[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            n_page[i] = page_of(p, j[i]);
            pg[i] = j[i] >= 0 ? table[n_page[i]] : 0;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int off = j[i] - n_page[i] * p.page;
            const bool has = static_cast<unsigned>(pg[i]) < static_cast<unsigned>(p.pages);
            bad |= j[i] >= 0 && !has;
            if (j[i] >= 0 && has) {
              kr[i] = pg[i] * p.k.rp + off * p.k.rt + k0;
              vr[i] = pg[i] * p.v.rp + off * p.v.rt + v0;
              see |= 1u << i;
            }
          }
        } else {
          const int kb = row.k0 * p.k.rt + k0, vb = row.k0 * p.v.rt + v0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (j[i] >= 0) {
              kr[i] = kb + j[i] * p.k.rt;
              vr[i] = vb + j[i] * p.v.rt;
              see |= 1u << i;
            }
          }
        }
      }
    }
    at += LISTS;
    while (at >= f.per) {
      at -= f.per;
      z += f.dz;
      hk += f.dh;
      t += f.dt;
      if (z >= f.n_z) {
        z -= f.n_z;
        ++hk;
      }
      if (hk >= p.Hk) {
        hk -= p.Hk;
        ++t;
      }
    }
    if (n + LISTS < tiles) blocks();
    uint32_t word = see << (4 * (lane & 7));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) word |= __shfl_xor_sync(0xffffffffu, word, o);
    const unsigned some = __ballot_sync(0xffffffffu, see != 0u);
    if (some != 0u) {
      const int top = 31 - __clz(static_cast<int>(some));
      h.n = 4 * top + 32 - __clz(__shfl_sync(0xffffffffu, static_cast<int>(see), top));
    }
    if (!bar_wait(free_bar + st, turn ^ 1u, ctl)) break;
    Tile& to = ring[st];
    reinterpret_cast<int4*>(to.k_row)[lane] = make_int4(kr[0], kr[1], kr[2], kr[3]);
    reinterpret_cast<int4*>(to.v_row)[lane] = make_int4(vr[0], vr[1], vr[2], vr[3]);
    if ((lane & 7) == 0) to.keys[lane >> 3] = word;
    if (lane == 0) to.h = h;
    __syncwarp();
    if (lane == 0) mbar_arrive(full + st);
    st += LISTS;
    if (st >= kRing) {
      st -= kRing;
      turn ^= 1u;
    }
  }
  if (bad) record_error(kErrDevice);
}

// ROWS rows of a tile (from row r0 on, as far as n) by a warp: P lanes a row, each
// group of lanes its own stretch of rows, whose numbers it reads four at a time.
// Eight copies in a row: a copy that waits for its registers' former use takes 140
// cycles instead of 40.  What counts beyond that are instructions (all roles of a CTA
// together had the schedulers busy for 63 % of the time): three for a copy.  Empty slots read as
// zero; copies that may have one have a size of their own, which costs them a quarter more.
template <int D, int ROWS>
__device__ __forceinline__ void load_rows(uint8_t* tile, const GatherRows& g, const int* rows, int r0, int n) {
  constexpr int P = D / 8, SPAN = ROWS * P / 32;  // 16-byte pieces of a row; rows of a group of lanes
  const int lane = static_cast<int>(lane_id()), piece = lane % P, first = r0 + SPAN * (lane / P);
  const char* base = static_cast<const char*>(g.base) + piece * 16;
  uint32_t at[8];  // of the swizzle's eight rows
#pragma unroll
  for (int i = 0; i < 8; ++i)
    at[i] = smem_u32(tile) + (piece >> 3) * kChunkBytes + (first + i) * 128 + (((piece & 7) ^ i) * 16);
#pragma unroll 1
  for (int h = 0; h < SPAN; h += 8) {
    int4 a = reinterpret_cast<const int4*>(rows + first + h)[0], b = reinterpret_cast<const int4*>(rows + first + h)[1];
    int row[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (__all_sync(0xffffffffu, (row[0] | row[1] | row[2] | row[3] | row[4] | row[5] | row[6] | row[7]) >= 0)) {
      const char* src[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) src[i] = base + static_cast<uint64_t>(static_cast<uint32_t>(row[i])) * g.unit_bytes;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at[i]), "l"(src[i]) : "memory");
    } else if (__any_sync(0xffffffffu, first + h < n)) {  // (rows past n are not read by the products)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at[i]),
                     "l"(base + static_cast<uint64_t>(static_cast<uint32_t>(max(row[i], 0))) * g.unit_bytes),
                     "r"(row[i] < 0 ? 0 : 16)
                     : "memory");
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) at[i] += 8 * 128;
  }
}
// Each lane arrives at `full` when its copies so far have landed; who waits there
// has to order them before the tensor cores' reads (fence_proxy_async_shared).
__device__ __forceinline__ void report_rows(uint64_t* full) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(full)) : "memory");
}
__device__ __forceinline__ void wait_rows() { asm volatile("cp.async.wait_all;" ::: "memory"); }

}  // namespace csa
