// A ring of shared-memory stages: fill i goes to stage i % stages, and the
// stage's barrier for "landed" completes its phase number i / stages, of
// parity (i / stages) & 1.  Plain C++, for device code and host tests.
#pragma once

#ifdef __CUDACC__
#define PAGEDKV_HD __host__ __device__ __forceinline__
#else
#define PAGEDKV_HD inline
#endif

namespace pagedkv {

// What a producer that leaves early has to wait for: calls wait(stage,
// parity) for each of the last `stages` of `armed` fills, oldest first.
// Earlier fills have landed, because a stage is armed again only after what
// it held was read; so every barrier waited for has completed all phases
// but, perhaps, the one that is asked for, and a parity is never one phase
// off.
template <typename Wait>
PAGEDKV_HD void fills_in_flight(int armed, int stages, Wait wait) {
  for (int i = armed > stages ? armed - stages : 0; i < armed; ++i) wait(i % stages, (i / stages) & 1);
}

}  // namespace pagedkv
