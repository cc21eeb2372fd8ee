// Order of the copies of a ring of shared-memory stages with a barrier each, as the staged row kernels
// use it: a block takes `steps` steps; the copies of the first `stages` of them are issued before it
// starts, and each step that found its copy issues the one `stages` steps ahead.  Plain arithmetic, also
// for the host.
#pragma once

#if defined(__CUDACC__)
#define MOE_HD __host__ __device__ __forceinline__
#else
#define MOE_HD inline
#endif

namespace moe {

// Copies that the block has issued when it stops waiting for them in step `lost`: that step and the
// later ones issue none.
MOE_HD int ring_issued(int lost, int stages, int steps) {
  return steps - stages < lost ? steps : lost + stages;
}
// The oldest of `issued` copies that may still be on its way once the block has stopped.
MOE_HD int ring_oldest(int issued, int stages) { return issued < stages ? 0 : issued - stages; }
// Stage of copy j, and the parity of the phase that it completes on the stage's barrier.
MOE_HD int ring_slot(int j, int stages) { return j % stages; }
MOE_HD unsigned ring_parity(int j, int stages) { return (unsigned)(j / stages) & 1u; }

}  // namespace moe
