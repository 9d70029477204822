// loads.cuh — loads of what another kernel of the stream may have written.
#pragma once

namespace qg {

// A kernel that starts before the one ahead of it has ended (programmatic
// dependent launch) shares the SM's L1 with it for a while.  The wait makes
// that kernel's writes visible to ordinary loads; read-only loads (__ldg)
// promise that nobody writes for as long as the kernel lives, which a cache
// slot, a length or a page table cannot.  So this is an ordinary load: the
// name says, where a read-only one would suggest itself, that it is meant.
template <class T>
__device__ __forceinline__ T fresh(const T* p) {
  return *p;
}

}  // namespace qg
