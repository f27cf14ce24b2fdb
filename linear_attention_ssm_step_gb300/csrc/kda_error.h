// kda_error.h - the status and message convention of the C ABI (kda_last_error), internal.
#pragma once

#include "kda.h"

namespace kda {

// Sets this host thread's message and returns `s`.
kda_status fail(kda_status s, const char* fmt, ...);
// Clears it and returns KDA_OK.
kda_status ok();

}  // namespace kda
