// host.h -- what the host side of every entry point shares.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <mutex>

#include "nucleus.h"

namespace nucleus {

// The library is built for gfx950 only; refuse other devices up front rather
// than fail inside a launch.
inline int check_device()
{
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return NUCLEUS_EDEVICE;
    static std::mutex mu;
    static int known[64] = {0};  // 0 unknown, 1 ok, -1 unsupported
    if (dev < 0 || dev >= 64) return NUCLEUS_EDEVICE;
    std::lock_guard<std::mutex> lock(mu);
    if (known[dev] == 0) {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return NUCLEUS_EDEVICE;
        known[dev] = (strncmp(prop.gcnArchName, "gfx950", 6) == 0) ? 1 : -1;
    }
    return known[dev] == 1 ? NUCLEUS_OK : NUCLEUS_EDEVICE;
}

template <class T>
bool aligned(const T* p)
{
    return ((uintptr_t)p % alignof(T)) == 0;
}

}  // namespace nucleus
