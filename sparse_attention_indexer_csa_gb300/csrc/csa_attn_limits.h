// csa_attn_limits.h -- how long the attention kernels wait before they give up,
// and what they still have to wait for then.  Compiles without CUDA headers.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define CSA_HD __host__ __device__ __forceinline__
#else
#define CSA_HD inline
#endif

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

// The copies into a ring of stages (32 at most) that a producer has started: a CTA
// may not end before they have landed, also when a wait gave up and nobody else
// waits for them.  A copy completes a phase of its stage's ring barrier, or, when
// its tile is mended before its products, one of the stage's other barrier; who
// mends it completes the ring's, unless it gave up.
struct Copies {
  uint32_t started = 0, mended = 0;       // stages with a copy; those whose last copy is to be mended
  uint32_t ring_phase = 0, mend_phase = 0;  // parity of the phase that the last copy completes
  uint32_t mend_next = 0;                 // parity of the other barrier's next phase

  CSA_HD void start(int stage, bool mend, uint32_t phase) {
    const uint32_t bit = 1u << stage;
    started |= bit;
    if (mend) {
      mended |= bit;
      mend_phase = (mend_phase & ~bit) | (mend_next & bit);
      mend_next ^= bit;
    } else {
      mended &= ~bit;
      ring_phase = (ring_phase & ~bit) | (phase != 0u ? bit : 0u);
    }
  }
  // wait(stage, mended, parity) for the last copy of each stage; the others landed before it was started.
  template <typename F>
  CSA_HD void drain(F wait) const {
    for (int s = 0; s < 32 && (started >> s) != 0u; ++s)
      if ((started >> s) & 1u) {
        const bool m = ((mended >> s) & 1u) != 0u;
        wait(s, m, ((m ? mend_phase : ring_phase) >> s) & 1u);
      }
  }
};

}  // namespace csa
