// host_common.hpp -- what the entry points of all sources share on the host.
#pragma once

namespace lpgemm {

// Kernel forced by lpgemm_set_kernel_override on the calling thread.
int forced_kernel();
// Compute units of the current device.
int compute_units();

}  // namespace lpgemm
