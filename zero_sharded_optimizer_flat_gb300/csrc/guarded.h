// What the training operators' entry points run their bodies in.
#pragma once

#include "internal.h"

namespace zopt {

// Runs an entry point's body; a C++ exception (an allocation that fails while a message is built)
// becomes a status, since none may leave a C function.
template <typename F>
zopt_status guarded(F body) noexcept {
  try {
    return body();
  } catch (...) {
    return ZOPT_ECUDA;
  }
}

}  // namespace zopt
