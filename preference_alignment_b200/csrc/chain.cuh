// Two kernels in a row where the second continues the first (launch_after): the first lets the
// second take its place early, the second waits until the first has finished and its writes are
// visible.
#pragma once

namespace dpo {

__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace dpo
