// kdn_errors.h -- the calling thread's error message (kdn_last_error_message),
// shared by the files of the host API.  Not part of the public ABI.
#pragma once

#include "kdn.h"

namespace kdn {

// sets the message and returns the status
kdn_status fail(kdn_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// clears it and returns KDN_OK
kdn_status ok();

}  // namespace kdn
