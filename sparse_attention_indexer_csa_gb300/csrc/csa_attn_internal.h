// csa_attn_internal.h -- host-side interface between the C ABI of csa_attn.h
// (csa_attn_api.cu) and the translation units that launch the kernels.
#pragma once

#include "csa_attn.h"
#include "csa_attn_limits.h"
#include "csa_internal.h"

namespace csa {

// ----------------------------------------------------------------- norm + rotation
// How the rows (token, head) of q or of k are dealt to groups of lanes: unit n
// (R consecutive rows) goes to group n % groups, so that all groups together
// read and write one window that moves through memory.
struct RowDeal {
  int groups, R, rounds;
  int skip, dt, dh;  // rows between two units of a group; the same in tokens and heads
};
struct NormRopeParams {
  int T, Hq, Hk, D, rot, off, w_dtype;
  float eps, inv_d;
  const void *q, *k, *qw, *kw;
  long long q_st, q_sh, k_st, k_sh;  // element strides
  const int64_t* pos;
  const uint64_t* freqs;
  void *yq, *yk;              // outputs (forward) or gradients of q and k (backward)
  const void *gq, *gk;        // cotangents (backward)
  float *dqw, *dkw;           // gradients of the weights (backward)
  float* part;                // partial sums of them, [blocks][D] (backward)
  int q_blocks;               // blocks that work on q; the others work on k
  RowDeal deal_q, deal_k;
};
constexpr int kNormRopeBlocks = 152 * 4;  // blocks (and partial sums) of the backward at most
cudaError_t launch_norm_rope(const NormRopeParams& p, int dtype, bool inter, cudaStream_t stream);
cudaError_t launch_norm_rope_backward(const NormRopeParams& p, int dtype, bool inter, cudaStream_t stream);

// The checks of csa_norm_rope's arguments, and its parameters without the outputs (unset when T is 0).
csa_status norm_rope_call(const csa_norm_rope_problem* p, const void* q, const void* k, const void* q_weight,
                          const void* k_weight, const int64_t* positions, const uint64_t* freqs, const void* q_out,
                          const void* k_out, NormRopeParams* n);

// ----------------------------------------------------------------- attention
struct AttnParams {
  int N, Tq, Tk, Hq, Hk, g, D;  // g = Hq / Hk
  int causal;
  float scale;
  const void *q, *k, *v;
  long long q_st, q_sh, k_st, k_sh, v_st, v_sh;
  const int32_t *cu_q, *cu_k, *k_len;
  void* out;
  float* lse;
  // backward
  const void* dout;
  float* delta;  // [Tq,Hq]: sum over D of dout * out
  // fp16: what dS can reach (see ds_exponent)
  float* norm2;     // [Tq,Hq]: sum over D of dout^2
  uint32_t* range;  // [N,Hk,2]: the largest of a sequence's rows of dout, and of v (bits of fp32)
  void *dq, *dk, *dv;
};
cudaError_t launch_attn_forward(const AttnParams& p, int dtype, void* workspace, cudaStream_t stream);
cudaError_t launch_attn_backward(const AttnParams& p, int dtype, void* workspace, cudaStream_t stream);
// out and lse from the outputs [n_split][Tq * Hq][D] and lse [n_split][Tq * Hq] of the shares of each row's keys (fp32).
cudaError_t launch_attn_join(const AttnParams& p, int dtype, const float* part_o, const float* part_lse, int n_split,
                             cudaStream_t stream);
cudaError_t take_status_attn_fwd(uint32_t* out, cudaStream_t stream);
cudaError_t take_status_attn_bwd(uint32_t* out, cudaStream_t stream);

// How the forward cuts its work, from the sizes the host knows (the lengths
// stand on the device).
constexpr int kMaxSplit = 256;
struct AttnPlan {
  int tiles;    // blocks of rows per CTA (2: one CTA per SM, 1: two)
  int rows;     // rows of a block: 128, or 32 (tiles = 1)
  int n_split;  // CTAs that share the keys of a block
};
inline AttnPlan attn_plan(int N, int Tq, int Tk, int Hk, int g) {
  const long long seqs = std::max(1, std::min(N, Tq));
  AttnPlan p;
  // Sequences whose rows fit one block would leave a second one empty; those
  // whose rows fit a quarter of one (decoding) leave room for a third tile of
  // keys in flight.
  p.tiles = Tq <= seqs * (128 / g) ? 1 : 2;
  p.rows = g <= 32 && Tq <= seqs * (32 / g) ? 32 : 128;
  const long long step = static_cast<long long>(p.tiles) * (p.rows / g);
  const long long items = std::max(seqs, (Tq + step - 1) / step) * Hk;
  const long long key_tiles = (Tk / std::max(1, N) + 127) / 128;  // of an average sequence
  // Few items: as many shares as fill the GPU once.  With more, shares even out
  // what the sequences' lengths leave uneven (64 sequences of 2048 to 8192 keys,
  // 8 key heads: 287 us in one share, 258 in three, 251 in five, 254 in eight);
  // a share of fewer than four (eight) tiles costs more than it gains.
  const long long slots = p.tiles == 1 ? 304 : 152;
  long long n = 1;
  if (2 * items <= slots)
    n = std::min(slots / items, key_tiles / 4);
  else if (p.tiles == 1 && items < 8 * slots)
    n = std::min((8 * slots + items - 1) / items, key_tiles / 8);
  p.n_split = static_cast<int>(std::max<long long>(1, std::min<long long>(n, kMaxSplit)));
  return p;
}

// How the backward cuts the dk, dv work, and what its workspace holds: delta,
// for fp16 the norms of dout's rows and the sequences' largest, the order of the
// runs of keys, the shares' sums.
struct AttnBwdPlan {
  int n_split;   // shares of the rows that see a run of 128 keys
  bool ordered;  // more items than SMs: the longest first
  size_t off_norm2, off_range, off_order, off_part, total;
};
inline AttnBwdPlan attn_bwd_plan(int N, int Tq, int Tk, int Hq, int Hk, int D, bool fp16) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  AttnBwdPlan p;
  const long long runs = std::max<long long>((static_cast<long long>(Tk) + 127) / 128, std::min(N, Tk));
  const long long items = std::max<long long>(1, runs * Hk);
  // blocks of 128 rows that an average run of keys meets
  const long long blocks = static_cast<long long>(Tq / std::max(1, std::min(N, Tq))) * (Hq / Hk) / 128;
  p.n_split = 1;
  if (items < 2 * 152) p.n_split = static_cast<int>(std::max<long long>(1, std::min((3 * 152 + items - 1) / items, blocks / 16)));
  p.ordered = items * p.n_split > 152;
  const size_t per_row = up(static_cast<size_t>(Tq) * Hq * 4);
  p.off_norm2 = per_row;
  p.off_range = per_row * (fp16 ? 2 : 1);
  p.off_order = up(p.off_range + (fp16 ? static_cast<size_t>(N) * Hk * 8 : 0));
  p.off_part = up(p.off_order + (p.ordered ? (static_cast<size_t>((static_cast<long long>(Tk) + 127) / 128) + N + 1) * 4 : 0));
  p.total = p.off_part + (p.n_split > 1 ? static_cast<size_t>(p.n_split) * Tk * Hk * D * 8 : 0);
  return p;
}

// ----------------------------------------------------------------- packed sequences (device)
// Extents of one sequence, clamped to the tensors: query rows q0..q1-1, keys
// k0..k0+lk-1.  A row r (counted from q0) sees the keys j < see(r).
struct SeqExt {
  int q0, q1, k0, lk;
};

__device__ __forceinline__ SeqExt seq_extent(const AttnParams& p, int i) {
  const int a = p.cu_q[i], b = p.cu_q[i + 1], c = p.cu_k[i], d = p.cu_k[i + 1];
  SeqExt s;
  s.q0 = min(max(a, 0), p.Tq);
  s.q1 = min(max(b, s.q0), p.Tq);
  s.k0 = min(max(c, 0), p.Tk);
  const int k1 = min(max(d, s.k0), p.Tk);
  s.lk = k1 - s.k0;
  bool bad = a != s.q0 || b != s.q1 || c != s.k0 || d != k1;
  if (p.k_len != nullptr) {
    const int n = p.k_len[i], m = min(max(n, 0), s.lk);
    bad |= n != m;
    s.lk = m;
  }
  if (bad) record_error(kErrDevice);
  return s;
}

// Number of keys row r (0-based in its sequence) sees.
__device__ __forceinline__ int keys_seen(const AttnParams& p, const SeqExt& s, int r) {
  if (!p.causal) return s.lk;
  return max(0, min(s.lk, r + 1 + s.lk - (s.q1 - s.q0)));
}

}  // namespace csa
