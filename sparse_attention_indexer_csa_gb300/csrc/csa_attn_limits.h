// csa_attn_limits.h -- how long the attention kernels wait before they give up.
// Host code without CUDA headers.
#pragma once

namespace csa {

// A wait inside a CTA lasts microseconds, but for the two that span an item: the
// warp that prepares items waits from an item's start until its last copy is under
// way, and the one that mends tiles until the last tiles arrive.  An item walks up to `steps`
// pairs of 128 rows and 128 keys, one after the other, some 1.4 us each; a
// lower clock or a GPU that is shared may take several times as long.  With
// 128 heads over one key head a run of keys in a sequence of 1.5 million tokens
// takes 2 s in this way.
constexpr unsigned long long kAttnWaitNs = 2000000000ull, kAttnStepNs = 20000ull;

inline unsigned long long attn_wait_ns(long long steps) {
  return kAttnWaitNs + (steps > 0 ? static_cast<unsigned long long>(steps) * kAttnStepNs : 0ull);
}
// Steps of the longest item: a run of rows walks the keys, a run of keys the rows (tq tokens a block).
inline long long attn_steps_keys(long long Tk) { return (Tk + 127) / 128; }
inline long long attn_steps_rows(long long Tq, long long tq) { return (Tq + tq - 1) / tq; }

}  // namespace csa
