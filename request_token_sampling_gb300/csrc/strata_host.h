// strata_host.h -- what the library's host files share: the per-thread error message, and what the
// calls without a context know of the current device.
#pragma once

#include <stdint.h>

namespace strata {

// Stores a one-line message for strata_last_error() and returns `code`.
__attribute__((visibility("hidden"), format(printf, 2, 3))) int host_fail(int code, const char* fmt, ...);

// The current device's word of STRATA_DEVERR_* bits and its number of SMs.
__attribute__((visibility("hidden"))) int tail_device(uint32_t** errors, int* sms);

}  // namespace strata
