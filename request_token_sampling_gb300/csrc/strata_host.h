// strata_host.h -- what the library's host files share: the per-thread error message.
#pragma once

namespace strata {

// Stores a one-line message for strata_last_error() and returns `code`.
__attribute__((visibility("hidden"), format(printf, 2, 3))) int host_fail(int code, const char* fmt, ...);

}  // namespace strata
