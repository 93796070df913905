// Host-side services of api.cu for the other translation units with entry
// points: the calling thread's error message and the current device.
#pragma once

#include <stdint.h>

namespace dec {

// Records a printf-style message as the calling thread's last error; returns `code`.
int host_fail(int code, const char* fmt, ...);
// SM count and error word of the current device, set up on first use.
int host_device(int* sms, uint32_t** err);

}  // namespace dec
