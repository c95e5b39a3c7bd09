// h3q_roles.cuh -- how the attention kernels' roles (warps with work of their own in a CTA) tell each other to
// give up.
#pragma once

#include <cuda_runtime.h>

namespace h3q {

// Whether a role has raised *abort: as this lane sees it now (another may see it a moment later), and as one
// answer for a converged warp, whose next steps are the whole warp's (votes, elections, TMEM).
__device__ __forceinline__ bool raised_here(const volatile int* abort) { return *abort != 0; }
__device__ __forceinline__ bool raised(const volatile int* abort) {
  return __any_sync(0xffffffffu, raised_here(abort));
}

}  // namespace h3q
