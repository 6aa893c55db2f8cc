// csa_sparse_api.cu -- the C ABI declared in include/csa_sparse.h: argument
// checks and launches.  Nothing here computes any part of the operators.
#include <cmath>
#include <cstring>
#include <initializer_list>
#include <numeric>

#include "csa_sparse_internal.h"

namespace csa {
namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t size_of(int dtype) { return dtype == CSA_F32 ? 4 : 2; }
bool type_ok(int t) { return t == CSA_BF16 || t == CSA_F32 || t == CSA_F16; }
// Strides feed 16-byte accesses and TMA maps: multiples of 16 bytes below 2^40 bytes.
bool stride_ok(long long s, size_t esize) {
  return s >= 0 && s < (1ll << 38) && (s * static_cast<long long>(esize)) % 16 == 0;
}
// Pointers of a tensor with `n` rows (may be NULL when it has none).
bool tensor_ok(const void* x, long long n, size_t align) { return (x != nullptr || n == 0) && aligned(x, align); }

// ----------------------------------------------------------------- attention over listed blocks
csa_status check_sparse(const csa_sparse_problem* p) {
  if (p == nullptr) return CSA_ERR_INVALID_ARG;
  if (p->N < 0 || p->Tq < 0 || p->Tk < 0 || p->Hq < 1 || p->Hk < 1 || p->D < 1) return CSA_ERR_INVALID_ARG;
  if (p->top_k < 0 || p->block < 1 || p->window < 0 || p->page < 0 || p->table_width < 0) return CSA_ERR_INVALID_ARG;
  if (!type_ok(p->dtype) || (p->causal != 0 && p->causal != 1)) return CSA_ERR_INVALID_ARG;
  if (!(p->scale > 0.f) || !std::isfinite(p->scale)) return CSA_ERR_INVALID_ARG;
  if (p->Hq % p->Hk != 0 || (p->window > 0 && p->causal == 0)) return CSA_ERR_INVALID_ARG;
  if (p->page > 0 ? p->Tk % p->page != 0 : p->table_width != 0) return CSA_ERR_INVALID_ARG;
  if (p->idx_stride < 0 || (p->idx_stride > 0 && p->idx_stride < p->top_k)) return CSA_ERR_INVALID_ARG;
  if (p->table_stride < 0 || (p->table_stride > 0 && p->table_stride < p->table_width)) return CSA_ERR_INVALID_ARG;
  for (long long s : {p->idx_stride, p->table_stride})
    if (s >= (1ll << 38)) return CSA_ERR_INVALID_ARG;
  for (long long s : {p->q_stride_t, p->q_stride_h, p->k_stride_p, p->k_stride_t, p->k_stride_h, p->v_stride_p,
                      p->v_stride_t, p->v_stride_h})
    if (!stride_ok(s, 2)) return CSA_ERR_INVALID_ARG;
  return CSA_OK;
}

// Rows to gather; false where their numbers pass 32 bits.
bool gather_rows(const csa_sparse_problem* p, const void* base, long long sp, long long st, long long sh,
                 GatherRows* r) {
  const long long page = p->page > 0 ? p->page : p->Tk, pages = p->page > 0 ? p->Tk / p->page : 1;
  if (sh == 0) sh = p->D;
  if (st == 0) st = static_cast<long long>(p->Hk) * p->D;
  if (sp == 0) sp = page * p->Hk * p->D;
  // a dimension of one entry has no stride
  if (p->Hk == 1) sh = 0;
  if (page <= 1) st = 0;
  if (pages <= 1) sp = 0;
  long long unit = std::gcd(std::gcd(sh, st), sp);
  if (unit == 0) unit = p->D;
  if (unit >= (1ll << 30)) unit = std::gcd(unit, 1ll << 29);
  const double rows = p->Tk == 0 ? 0.0
                                 : (static_cast<double>(sp) * (pages - 1) + static_cast<double>(st) * (page - 1) +
                                    static_cast<double>(sh) * (p->Hk - 1)) / static_cast<double>(unit) + 1.0;
  if (rows > 2147483000.0) return false;
  r->base = base;
  r->unit_bytes = static_cast<uint32_t>(unit * 2);
  r->rp = static_cast<int>(sp / unit);
  r->rt = static_cast<int>(st / unit);
  r->rh = static_cast<int>(sh / unit);
  return true;
}

bool sparse_supported(const csa_sparse_problem* p) {
  if (p->D != 64 && p->D != 128) return false;
  if (p->dtype != CSA_BF16 && p->dtype != CSA_F16) return false;
  if (p->Hq / p->Hk > 128 || p->Hq > 65535 || p->block > 128 || (p->block & (p->block - 1)) != 0) return false;
  if (p->window + static_cast<long long>(p->top_k) * p->block > (1 << 20)) return false;
  if (p->scale > 0x1p127f) return false;  // scale * log2(e) is finite
  GatherRows r;
  if (!gather_rows(p, nullptr, p->k_stride_p, p->k_stride_t, p->k_stride_h, &r)) return false;
  if (!gather_rows(p, nullptr, p->v_stride_p, p->v_stride_t, p->v_stride_h, &r)) return false;
  const double rows = std::max(static_cast<double>(p->Tq) * p->Hq, static_cast<double>(p->Tk) * p->Hk);
  return rows < 8.0e9 && p->N < (1 << 30) && static_cast<long long>(p->Tk) / p->block + p->N < 0x7FFFFFF0ll;
}

SparseParams sparse_params(const csa_sparse_problem* p, const void* q, const void* k, const void* v,
                           const int32_t* idx, const int32_t* cu_q, const int32_t* cu_k, const int32_t* k_len,
                           const int32_t* table) {
  SparseParams a;
  std::memset(&a, 0, sizeof(a));
  a.N = p->N;
  a.Tq = p->Tq;
  a.Tk = p->Tk;
  a.Hq = p->Hq;
  a.Hk = p->Hk;
  a.g = p->Hq / p->Hk;
  a.D = p->D;
  a.top_k = p->top_k;
  while ((1 << a.block_shift) < p->block) ++a.block_shift;
  a.window = p->window;
  a.causal = p->causal;
  a.page = p->page;
  a.pages = p->page > 0 ? p->Tk / p->page : 0;
  a.table_width = p->table_width;
  a.page_shift = 31;
  while (p->page > (1ll << (a.page_shift - 31))) ++a.page_shift;
  a.page_mul = p->page > 0 ? static_cast<uint32_t>(((1ull << a.page_shift) + p->page - 1) / p->page) : 0;
  a.scale = p->scale;
  a.q = q;
  a.q_sh = p->q_stride_h ? p->q_stride_h : p->D;
  a.q_st = p->q_stride_t ? p->q_stride_t : static_cast<long long>(p->Hq) * p->D;
  a.idx_st = p->idx_stride ? p->idx_stride : p->top_k;
  a.table_st = p->table_stride ? p->table_stride : p->table_width;
  gather_rows(p, k, p->k_stride_p, p->k_stride_t, p->k_stride_h, &a.k);
  gather_rows(p, v, p->v_stride_p, p->v_stride_t, p->v_stride_h, &a.v);
  a.idx = idx;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.k_len = k_len;
  a.table = table;
  return a;
}

csa_status check_sparse_inputs(const csa_sparse_problem* p, const void* q, const void* k, const void* v,
                               const int32_t* idx, const int32_t* cu_q, const int32_t* cu_k, const int32_t* k_len,
                               const int32_t* table) {
  if (!tensor_ok(q, p->Tq, 16) || !tensor_ok(k, p->Tk, 16) || !tensor_ok(v, p->Tk, 16)) return CSA_ERR_INVALID_ARG;
  if (!tensor_ok(cu_q, p->N, 4) || !aligned(cu_k, 4) || !aligned(k_len, 4) || !aligned(table, 4) || !aligned(idx, 4))
    return CSA_ERR_INVALID_ARG;
  if (p->top_k == 0 ? idx != nullptr : (idx == nullptr && p->Tq > 0)) return CSA_ERR_INVALID_ARG;
  if (p->page > 0) {
    if (cu_k != nullptr || (k_len == nullptr && p->N > 0)) return CSA_ERR_INVALID_ARG;
    if (table == nullptr && p->N > 0 && p->table_width > 0) return CSA_ERR_INVALID_ARG;
  } else if (table != nullptr || (cu_k == nullptr && p->N > 0)) {
    return CSA_ERR_INVALID_ARG;
  }
  return CSA_OK;
}

size_t sparse_workspace_bytes(const csa_sparse_problem* p, int which) {
  if (check_sparse(p) != CSA_OK || !sparse_supported(p)) return 0;
  const SparseParams a = sparse_params(p, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr);
  if (which == 1) return p->page > 0 ? 0 : sparse_backward_workspace(a, p->dtype);
  if (which != 0 || p->Tq == 0) return 0;
  const int n = sparse_splits(p->Tq, p->Hk, sparse_slots(a));
  return n > 1 ? static_cast<size_t>(n) * p->Tq * p->Hq * (p->D + 1) * 4 : 0;
}
bool workspace_ok(const void* ws, size_t bytes, size_t need) {
  return need == 0 || (ws != nullptr && bytes >= need && aligned(ws, 16));
}

}  // namespace
}  // namespace csa

using namespace csa;

extern "C" {

csa_status csa_sparse_attn_forward(const csa_sparse_problem* p, const void* q, const void* k, const void* v,
                                   const int32_t* idx, const int32_t* cu_q, const int32_t* cu_k,
                                   const int32_t* k_len, const int32_t* table, void* out, float* lse,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  csa_status st = check_sparse(p);
  if (st != CSA_OK) return st;
  if ((st = check_sparse_inputs(p, q, k, v, idx, cu_q, cu_k, k_len, table)) != CSA_OK) return st;
  if (!tensor_ok(out, p->Tq, 16) || !tensor_ok(lse, p->Tq, 16)) return CSA_ERR_INVALID_ARG;
  if (!sparse_supported(p)) return CSA_ERR_UNSUPPORTED;
  if (!workspace_ok(workspace, workspace_bytes, sparse_workspace_bytes(p, 0))) return CSA_ERR_INVALID_ARG;
  if (p->Tq == 0) return CSA_OK;
  SparseParams a = sparse_params(p, q, k, v, idx, cu_q, cu_k, k_len, table);
  a.out = out;
  a.lse = lse;
  if (launch_sparse_forward(a, p->dtype, workspace, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return CSA_ERR_CUDA;
  return CSA_OK;
}

csa_status csa_sparse_attn_backward(const csa_sparse_problem* p, const void* dout, const void* q, const void* k,
                                    const void* v, const void* out, const float* lse, const int32_t* idx,
                                    const int32_t* cu_q, const int32_t* cu_k, const int32_t* k_len, void* dq,
                                    void* dk, void* dv, void* workspace, size_t workspace_bytes, void* stream) {
  csa_status st = check_sparse(p);
  if (st != CSA_OK) return st;
  if (p->page > 0) return CSA_ERR_UNSUPPORTED;
  if ((st = check_sparse_inputs(p, q, k, v, idx, cu_q, cu_k, k_len, nullptr)) != CSA_OK) return st;
  for (const void* x : {dout, out, static_cast<const void*>(lse), static_cast<const void*>(dq)})
    if (!tensor_ok(x, p->Tq, 16)) return CSA_ERR_INVALID_ARG;
  if (!tensor_ok(dk, p->Tk, 16) || !tensor_ok(dv, p->Tk, 16)) return CSA_ERR_INVALID_ARG;
  if (!sparse_supported(p)) return CSA_ERR_UNSUPPORTED;
  if (!workspace_ok(workspace, workspace_bytes, sparse_workspace_bytes(p, 1))) return CSA_ERR_INVALID_ARG;
  if (p->Tq == 0 && p->Tk == 0) return CSA_OK;
  SparseParams a = sparse_params(p, q, k, v, idx, cu_q, cu_k, k_len, nullptr);
  a.dout = dout;
  a.out = const_cast<void*>(out);
  a.lse = const_cast<float*>(lse);
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  if (launch_sparse_backward(a, p->dtype, workspace, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return CSA_ERR_CUDA;
  return CSA_OK;
}

size_t csa_sparse_attn_workspace_size(const csa_sparse_problem* p, int32_t which) {
  return sparse_workspace_bytes(p, which);
}

csa_status csa_norm_rope_append(const csa_norm_rope_problem* p, const csa_append_problem* c, const void* q,
                                const void* k, const void* v, const void* q_weight, const void* k_weight,
                                const int64_t* positions, const uint64_t* freqs, const int32_t* cu_q,
                                const int32_t* k_len, const int32_t* table, void* q_out, void* k_pages,
                                void* v_pages, void* stream) {
  NormRopeParams n;
  csa_status st = norm_rope_call(p, q, k, q_weight, k_weight, positions, freqs, q_out, k_pages, &n);
  if (st != CSA_OK && st != CSA_ERR_UNSUPPORTED) return st;
  if (c == nullptr || p->Hk < 1) return CSA_ERR_INVALID_ARG;
  if (c->N < 0 || c->pages < 0 || c->page < 1 || c->table_width < 0) return CSA_ERR_INVALID_ARG;
  if (c->table_stride < 0 || c->table_stride >= (1ll << 38) ||
      (c->table_stride > 0 && c->table_stride < c->table_width))
    return CSA_ERR_INVALID_ARG;
  for (long long s : {c->v_stride_t, c->v_stride_h, c->kc_stride_p, c->kc_stride_t, c->kc_stride_h, c->vc_stride_p,
                      c->vc_stride_t, c->vc_stride_h})
    if (!stride_ok(s, size_of(p->dtype))) return CSA_ERR_INVALID_ARG;
  if (st != CSA_OK) return st;
  if (p->T == 0) return CSA_OK;
  if (v == nullptr || !aligned(v, 16) || v_pages == nullptr || !aligned(v_pages, 16)) return CSA_ERR_INVALID_ARG;
  if (!tensor_ok(cu_q, c->N, 4) || !tensor_ok(k_len, c->N, 4) ||
      !tensor_ok(table, c->table_width > 0 ? c->N : 0, 4))
    return CSA_ERR_INVALID_ARG;
  AppendParams a;
  std::memset(&a, 0, sizeof(a));
  const long long head = p->D, token = static_cast<long long>(p->Hk) * p->D, page = token * c->page;
  a.N = c->N;
  a.pages = c->pages;
  a.page = c->page;
  a.table_width = c->table_width;
  a.table_st = c->table_stride ? c->table_stride : c->table_width;
  a.v = v;
  a.v_st = c->v_stride_t ? c->v_stride_t : token;
  a.v_sh = c->v_stride_h ? c->v_stride_h : head;
  a.kc = k_pages;
  a.vc = v_pages;
  a.kc_sp = c->kc_stride_p ? c->kc_stride_p : page;
  a.kc_st = c->kc_stride_t ? c->kc_stride_t : token;
  a.kc_sh = c->kc_stride_h ? c->kc_stride_h : head;
  a.vc_sp = c->vc_stride_p ? c->vc_stride_p : page;
  a.vc_st = c->vc_stride_t ? c->vc_stride_t : token;
  a.vc_sh = c->vc_stride_h ? c->vc_stride_h : head;
  a.cu_q = cu_q;
  a.k_len = k_len;
  a.table = table;
  n.yq = q_out;
  if (launch_norm_rope_append(n, a, p->dtype, p->interleaved != 0, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return CSA_ERR_CUDA;
  return CSA_OK;
}

int32_t csa_sparse_abi_version(void) { return 100; }

}  // extern "C"
