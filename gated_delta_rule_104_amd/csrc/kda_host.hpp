// Host-side services of the C-ABI layer that its translation units share: the
// calling thread's error text, the device's size and the process-wide options.
// Defined in kda_api.hip.
#pragma once

#include "../../include/libkda.h"

namespace kda {

// Sets kda_last_error() of this thread and returns st.
kda_status api_fail(kda_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears it and returns KDA_OK.
kda_status api_ok();
// Compute units of the current device.
int api_cu_count();
// Options "check" and "log".
bool api_check_on();
bool api_log_on();
// Option "glr_polls".
int api_glr_polls();

}  // namespace kda
