// pdl.cuh - programmatic dependent launch.
#pragma once

namespace fa {

// A kernel launched with that attribute may begin before the one ahead of it
// on the stream ends: pdl_wait() returns once everything ahead has completed
// and its writes are visible.  pdl_launch() lets the kernel behind begin in
// the same way; after pdl_wait() what is ahead of this kernel is then complete
// for that one before it waits itself.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace fa
