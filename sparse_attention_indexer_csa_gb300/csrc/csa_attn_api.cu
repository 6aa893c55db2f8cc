// csa_attn_api.cu -- the C ABI declared in include/csa_attn.h: argument checks
// and launches.  Nothing here computes any part of the operators.
#include <cmath>
#include <cstring>

#include "csa_attn_internal.h"

namespace csa {
namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t size_of(int dtype) { return dtype == CSA_F32 ? 4 : 2; }
bool type_ok(int t) { return t == CSA_BF16 || t == CSA_F32 || t == CSA_F16; }
// Strides feed 16-byte accesses and TMA maps: multiples of 16 bytes below 2^40 bytes.
bool stride_ok(long long s, size_t esize) {
  return s >= 0 && (s * static_cast<long long>(esize)) % 16 == 0 && s < (1ll << 38);
}

// ----------------------------------------------------------------- norm + rotation
csa_status check_norm_rope(const csa_norm_rope_problem* p) {
  if (p == nullptr) return CSA_ERR_INVALID_ARG;
  if (p->T < 0 || p->Hq < 1 || p->Hk < 0 || p->D < 1 || p->rot < 1 || p->rot_offset < 0) return CSA_ERR_INVALID_ARG;
  if (!type_ok(p->dtype) || !type_ok(p->w_dtype) || (p->interleaved != 0 && p->interleaved != 1))
    return CSA_ERR_INVALID_ARG;
  if (!(p->eps >= 0.f) || !std::isfinite(p->eps)) return CSA_ERR_INVALID_ARG;
  if (static_cast<long long>(p->rot_offset) + p->rot > p->D || p->rot % 2 != 0) return CSA_ERR_INVALID_ARG;
  if (static_cast<long long>(p->Hq) + p->Hk > (1 << 24)) return CSA_ERR_INVALID_ARG;
  for (long long s : {p->q_stride_t, p->q_stride_h, p->k_stride_t, p->k_stride_h})
    if (!stride_ok(s, size_of(p->dtype))) return CSA_ERR_INVALID_ARG;
  return CSA_OK;
}
bool norm_rope_supported(const csa_norm_rope_problem* p) {
  return p->D % 8 == 0 && p->D <= 256 && p->rot_offset % 8 == 0 && p->rot % (p->interleaved ? 8 : 16) == 0;
}
NormRopeParams norm_rope_params(const csa_norm_rope_problem* p, const void* q, const void* k, const void* qw,
                                const void* kw, const int64_t* pos, const uint64_t* freqs) {
  NormRopeParams n;
  std::memset(&n, 0, sizeof(n));
  n.T = p->T;
  n.Hq = p->Hq;
  n.Hk = p->Hk;
  n.D = p->D;
  n.rot = p->rot;
  n.off = p->rot_offset;
  n.w_dtype = p->w_dtype;
  n.eps = p->eps;
  n.inv_d = 1.0f / static_cast<float>(p->D);
  n.q = q;
  n.k = k;
  n.qw = qw;
  n.kw = kw;
  n.q_sh = p->q_stride_h ? p->q_stride_h : p->D;
  n.q_st = p->q_stride_t ? p->q_stride_t : static_cast<long long>(p->Hq) * p->D;
  n.k_sh = p->k_stride_h ? p->k_stride_h : p->D;
  n.k_st = p->k_stride_t ? p->k_stride_t : static_cast<long long>(p->Hk) * p->D;
  n.pos = pos;
  n.freqs = freqs;
  return n;
}
csa_status check_norm_rope_inputs(const csa_norm_rope_problem* p, const void* q, const void* k, const void* qw,
                                  const void* kw, const int64_t* pos, const uint64_t* freqs, const void* a,
                                  const void* b) {
  const size_t ws = size_of(p->w_dtype);
  for (const void* x : {q, a})
    if (x == nullptr || !aligned(x, 16)) return CSA_ERR_INVALID_ARG;
  if (qw == nullptr || pos == nullptr || freqs == nullptr) return CSA_ERR_INVALID_ARG;
  if (!aligned(qw, ws) || !aligned(pos, 8) || !aligned(freqs, 8)) return CSA_ERR_INVALID_ARG;
  if (p->Hk > 0) {
    for (const void* x : {k, b})
      if (x == nullptr || !aligned(x, 16)) return CSA_ERR_INVALID_ARG;
    if (kw == nullptr || !aligned(kw, ws)) return CSA_ERR_INVALID_ARG;
  } else if (k != nullptr || kw != nullptr || b != nullptr) {
    return CSA_ERR_INVALID_ARG;
  }
  return CSA_OK;
}

// ----------------------------------------------------------------- attention
csa_status check_attn(const csa_attn_problem* p) {
  if (p == nullptr) return CSA_ERR_INVALID_ARG;
  if (p->N < 0 || p->Tq < 0 || p->Tk < 0 || p->Hq < 1 || p->Hk < 1 || p->D < 1) return CSA_ERR_INVALID_ARG;
  if (!type_ok(p->dtype) || (p->causal != 0 && p->causal != 1)) return CSA_ERR_INVALID_ARG;
  if (!(p->scale > 0.f) || !std::isfinite(p->scale)) return CSA_ERR_INVALID_ARG;
  if (p->Hq % p->Hk != 0) return CSA_ERR_INVALID_ARG;
  for (long long s : {p->q_stride_t, p->q_stride_h, p->k_stride_t, p->k_stride_h, p->v_stride_t, p->v_stride_h})
    if (!stride_ok(s, 2)) return CSA_ERR_INVALID_ARG;
  return CSA_OK;
}
bool attn_supported(const csa_attn_problem* p) {
  if (p->D != 64 && p->D != 128) return false;
  if (p->dtype != CSA_BF16 && p->dtype != CSA_F16) return false;
  if (p->Hq / p->Hk > 128 || p->Hq > 65535) return false;
  if (static_cast<double>(p->q_stride_h) * (p->Hq / p->Hk) > static_cast<double>(1ll << 38)) return false;
  const double rows = std::max(static_cast<double>(p->Tq) * p->Hq, static_cast<double>(p->Tk) * p->Hk);
  return rows < 8.0e9 && p->N < (1 << 30);
}
AttnParams attn_params(const csa_attn_problem* p, const void* q, const void* k, const void* v, const int32_t* cu_q,
                       const int32_t* cu_k, const int32_t* k_len) {
  AttnParams a;
  std::memset(&a, 0, sizeof(a));
  a.N = p->N;
  a.Tq = p->Tq;
  a.Tk = p->Tk;
  a.Hq = p->Hq;
  a.Hk = p->Hk;
  a.g = p->Hq / p->Hk;
  a.D = p->D;
  a.causal = p->causal;
  a.scale = p->scale;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_sh = p->q_stride_h ? p->q_stride_h : p->D;
  a.q_st = p->q_stride_t ? p->q_stride_t : static_cast<long long>(p->Hq) * p->D;
  a.k_sh = p->k_stride_h ? p->k_stride_h : p->D;
  a.k_st = p->k_stride_t ? p->k_stride_t : static_cast<long long>(p->Hk) * p->D;
  a.v_sh = p->v_stride_h ? p->v_stride_h : p->D;
  a.v_st = p->v_stride_t ? p->v_stride_t : static_cast<long long>(p->Hk) * p->D;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.k_len = k_len;
  return a;
}
// Pointers of a tensor with `n` rows (may be NULL when it has none).
bool tensor_ok(const void* x, long long n, size_t align) { return (x != nullptr || n == 0) && aligned(x, align); }
csa_status check_attn_inputs(const csa_attn_problem* p, const void* q, const void* k, const void* v,
                             const int32_t* cu_q, const int32_t* cu_k, const int32_t* k_len) {
  if (!tensor_ok(q, p->Tq, 16) || !tensor_ok(k, p->Tk, 16) || !tensor_ok(v, p->Tk, 16)) return CSA_ERR_INVALID_ARG;
  if (!tensor_ok(cu_q, p->N, 4) || !tensor_ok(cu_k, p->N, 4) || !aligned(k_len, 4)) return CSA_ERR_INVALID_ARG;
  return CSA_OK;
}
size_t attn_workspace_bytes(const csa_attn_problem* p, int which) {
  if (check_attn(p) != CSA_OK) return 0;
  if (which == 1) return attn_bwd_plan(p->N, p->Tq, p->Tk, p->Hq, p->Hk, p->D, p->dtype == CSA_F16).total;
  if (which != 0 || p->Tq == 0 || !attn_supported(p)) return 0;
  // split keys: fp32 outputs and lse of each share
  const AttnPlan plan = attn_plan(p->N, p->Tq, p->Tk, p->Hk, p->Hq / p->Hk);
  return plan.n_split > 1 ? static_cast<size_t>(plan.n_split) * p->Tq * p->Hq * (p->D + 1) * 4 : 0;
}

// ----------------------------------------------------------------- frequencies
// A number as the sum of two doubles, some 100 bits: a table entry is multiplied by the position, so that the 53 bits
// of one would be off by 6e-5 of a radian at position 1e12.
struct Dd {
  double hi, lo;
};
Dd dd_sum(double a, double b) {  // exact
  const double s = a + b, t = s - a;
  return Dd{s, (a - (s - t)) + (b - t)};
}
Dd dd_add(Dd a, Dd b) {
  const Dd s = dd_sum(a.hi, b.hi);
  return dd_sum(s.hi, s.lo + (a.lo + b.lo));
}
Dd dd_mul(Dd a, Dd b) {
  const double p = a.hi * b.hi;
  return dd_sum(p, std::fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi));
}
Dd dd_div(Dd a, double n) {
  const double q = a.hi / n;
  return dd_sum(q, (std::fma(-q, n, a.hi) + a.lo) / n);
}
// e^x, |x| < 64: the series at x / 1024 (below 1/16; the 18th power over 18! is below 2^-120), squared ten times.
Dd dd_exp(Dd x) {
  const Dd r{std::ldexp(x.hi, -10), std::ldexp(x.lo, -10)}, one{1.0, 0.0};
  Dd e = one;
  for (int n = 17; n > 0; --n) e = dd_add(one, dd_div(dd_mul(r, e), n));
  for (int i = 0; i < 10; ++i) e = dd_mul(e, e);
  return e;
}
// ln x by one step from the double's: y + (x e^-y - 1), whose error is the square of the first.
Dd dd_log(double x) {
  const double y = std::log(x);
  const Dd d = dd_add(dd_mul(Dd{x, 0.0}, dd_exp(Dd{-y, 0.0})), Dd{-1.0, 0.0});
  return dd_add(Dd{y, 0.0}, d);
}

}  // namespace

csa_status norm_rope_call(const csa_norm_rope_problem* p, const void* q, const void* k, const void* q_weight,
                          const void* k_weight, const int64_t* positions, const uint64_t* freqs, const void* q_out,
                          const void* k_out, NormRopeParams* n) {
  const csa_status st = check_norm_rope(p);
  if (st != CSA_OK) return st;
  if (!norm_rope_supported(p)) return CSA_ERR_UNSUPPORTED;
  std::memset(n, 0, sizeof(*n));
  if (p->T == 0) return CSA_OK;
  *n = norm_rope_params(p, q, k, q_weight, k_weight, positions, freqs);
  return check_norm_rope_inputs(p, q, k, q_weight, k_weight, positions, freqs, q_out, k_out);
}

}  // namespace csa

using namespace csa;

extern "C" {

csa_status csa_rope_freqs(double theta, int32_t rot, uint64_t* freqs) {
  if (freqs == nullptr || rot < 2 || rot % 2 != 0 || !(theta > 1.0) || !(theta <= 1e18)) return CSA_ERR_INVALID_ARG;
  const Dd log_theta = dd_log(theta);
  const Dd inv_two_pi{0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};
  for (int i = 0; i < rot / 2; ++i) {
    const Dd turns = dd_mul(dd_exp(dd_div(dd_mul(log_theta, Dd{-2.0 * i, 0.0}), rot)), inv_two_pi);  // below 0.16
    const double whole = std::floor(std::ldexp(turns.hi, 64));
    const double rest = (std::ldexp(turns.hi, 64) - whole) + std::ldexp(turns.lo, 64);
    freqs[i] = static_cast<uint64_t>(whole) + static_cast<uint64_t>(static_cast<int64_t>(std::nearbyint(rest)));
  }
  return CSA_OK;
}

csa_status csa_norm_rope(const csa_norm_rope_problem* p, const void* q, const void* k, const void* q_weight,
                         const void* k_weight, const int64_t* positions, const uint64_t* freqs, void* q_out,
                         void* k_out, void* stream) {
  csa_status st = check_norm_rope(p);
  if (st != CSA_OK) return st;
  if (!norm_rope_supported(p)) return CSA_ERR_UNSUPPORTED;
  if (p->T == 0) return CSA_OK;
  if ((st = check_norm_rope_inputs(p, q, k, q_weight, k_weight, positions, freqs, q_out, k_out)) != CSA_OK) return st;
  NormRopeParams n = norm_rope_params(p, q, k, q_weight, k_weight, positions, freqs);
  n.yq = q_out;
  n.yk = k_out;
  if (launch_norm_rope(n, p->dtype, p->interleaved != 0, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return CSA_ERR_CUDA;
  return CSA_OK;
}

size_t csa_norm_rope_workspace_size(const csa_norm_rope_problem* p) {
  if (check_norm_rope(p) != CSA_OK) return 0;
  return static_cast<size_t>(kNormRopeBlocks) * 2 * p->D * sizeof(float);
}

csa_status csa_norm_rope_backward(const csa_norm_rope_problem* p, const void* dq_out, const void* dk_out,
                                  const void* q, const void* k, const void* q_weight, const void* k_weight,
                                  const int64_t* positions, const uint64_t* freqs, void* dq, void* dk,
                                  float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  csa_status st = check_norm_rope(p);
  if (st != CSA_OK) return st;
  if (!norm_rope_supported(p)) return CSA_ERR_UNSUPPORTED;
  if (dq_weight == nullptr || !aligned(dq_weight, 4) || !aligned(dk_weight, 4)) return CSA_ERR_INVALID_ARG;
  if ((p->Hk > 0) != (dk_weight != nullptr)) return CSA_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p->T == 0) {  // empty sums
    if (cudaMemsetAsync(dq_weight, 0, sizeof(float) * p->D, s) != cudaSuccess) return CSA_ERR_CUDA;
    if (dk_weight != nullptr && cudaMemsetAsync(dk_weight, 0, sizeof(float) * p->D, s) != cudaSuccess)
      return CSA_ERR_CUDA;
    return CSA_OK;
  }
  if ((st = check_norm_rope_inputs(p, q, k, q_weight, k_weight, positions, freqs, dq_out, dk_out)) != CSA_OK)
    return st;
  if (dq == nullptr || !aligned(dq, 16) || (p->Hk > 0) != (dk != nullptr) || !aligned(dk, 16))
    return CSA_ERR_INVALID_ARG;
  if (workspace == nullptr || workspace_bytes < csa_norm_rope_workspace_size(p) || !aligned(workspace, 16))
    return CSA_ERR_INVALID_ARG;
  NormRopeParams n = norm_rope_params(p, q, k, q_weight, k_weight, positions, freqs);
  n.gq = dq_out;
  n.gk = dk_out;
  n.yq = dq;
  n.yk = dk;
  n.dqw = dq_weight;
  n.dkw = dk_weight;
  n.part = static_cast<float*>(workspace);
  if (launch_norm_rope_backward(n, p->dtype, p->interleaved != 0, s) != cudaSuccess) return CSA_ERR_CUDA;
  return CSA_OK;
}

csa_status csa_attn_forward(const csa_attn_problem* p, const void* q, const void* k, const void* v,
                            const int32_t* cu_q, const int32_t* cu_k, const int32_t* k_len, void* out, float* lse,
                            void* workspace, size_t workspace_bytes, void* stream) {
  csa_status st = check_attn(p);
  if (st != CSA_OK) return st;
  if ((st = check_attn_inputs(p, q, k, v, cu_q, cu_k, k_len)) != CSA_OK) return st;
  if (!tensor_ok(out, p->Tq, 16) || !tensor_ok(lse, p->Tq, 16)) return CSA_ERR_INVALID_ARG;
  if (!attn_supported(p)) return CSA_ERR_UNSUPPORTED;
  const size_t need = attn_workspace_bytes(p, 0);
  if (need != 0 && (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 16)))
    return CSA_ERR_INVALID_ARG;
  if (p->Tq == 0) return CSA_OK;
  AttnParams a = attn_params(p, q, k, v, cu_q, cu_k, k_len);
  a.out = out;
  a.lse = lse;
  if (launch_attn_forward(a, p->dtype, workspace, static_cast<cudaStream_t>(stream)) != cudaSuccess) return CSA_ERR_CUDA;
  return CSA_OK;
}

csa_status csa_attn_backward(const csa_attn_problem* p, const void* dout, const void* q, const void* k,
                             const void* v, const void* out, const float* lse, const int32_t* cu_q,
                             const int32_t* cu_k, const int32_t* k_len, void* dq, void* dk, void* dv,
                             void* workspace, size_t workspace_bytes, void* stream) {
  csa_status st = check_attn(p);
  if (st != CSA_OK) return st;
  if ((st = check_attn_inputs(p, q, k, v, cu_q, cu_k, k_len)) != CSA_OK) return st;
  for (const void* x : {dout, out, static_cast<const void*>(lse), static_cast<const void*>(dq)})
    if (!tensor_ok(x, p->Tq, 16)) return CSA_ERR_INVALID_ARG;
  if (!tensor_ok(dk, p->Tk, 16) || !tensor_ok(dv, p->Tk, 16)) return CSA_ERR_INVALID_ARG;
  if (!attn_supported(p)) return CSA_ERR_UNSUPPORTED;
  const size_t need = attn_workspace_bytes(p, 1);
  if (need != 0 && (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 16)))
    return CSA_ERR_INVALID_ARG;
  if (p->Tq == 0 && p->Tk == 0) return CSA_OK;
  AttnParams a = attn_params(p, q, k, v, cu_q, cu_k, k_len);
  a.dout = dout;
  a.out = const_cast<void*>(out);
  a.lse = const_cast<float*>(lse);
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  if (launch_attn_backward(a, p->dtype, workspace, static_cast<cudaStream_t>(stream)) != cudaSuccess) return CSA_ERR_CUDA;
  return CSA_OK;
}

size_t csa_attn_workspace_size(const csa_attn_problem* p, int32_t which) { return attn_workspace_bytes(p, which); }

int32_t csa_attn_abi_version(void) { return 100; }

}  // extern "C"
