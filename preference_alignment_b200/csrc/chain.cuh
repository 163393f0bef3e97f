// A kernel that continues the one before it on the stream (launch_after): it may be set up while
// that one still runs, and waits here until that one has finished and its writes are visible.
// What it reads of them goes past L1 (__ldcg). (Letting it start at the first kernel's beginning
// instead of its end was measured too and cost up to 10 us.)
#pragma once

namespace dpo {

__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace dpo
