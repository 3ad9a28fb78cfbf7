// context.hpp -- what the entry points outside proj.cpp use of a context.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/proj.h"

namespace proj {

struct ContextView {
    int device;
    int cus;          // compute units of the device
    float *ws;        // the context's workspace, ws_bytes long
    size_t ws_bytes;
    uint32_t *counters;  // ncounters of them, zero between calls: a kernel that counts sets its own back
    int ncounters;
};

// PROJ_OK and the view of a live context, or the status of a call with `c`.
proj_status context_view(proj_ctx *c, ContextView *v);

// Keep a message in the (live) context and return `s`.
proj_status context_error(proj_ctx *c, proj_status s, const char *fmt, ...) __attribute__((format(printf, 3, 4)));

class DeviceGuard {
   public:
    explicit DeviceGuard(int dev) {
        if (hipGetDevice(&prev_) != hipSuccess) prev_ = -1;
        if (prev_ != dev) hipSetDevice(dev);
    }
    ~DeviceGuard() {
        int cur = -1;
        if (prev_ >= 0 && hipGetDevice(&cur) == hipSuccess && cur != prev_) hipSetDevice(prev_);
    }

   private:
    int prev_ = -1;
};

// Whether byte ranges [a, a + na) and [b, b + nb) share a byte.
inline bool overlap(const void *a, uint64_t na, const void *b, uint64_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    return pa < pb + nb && pb < pa + na;
}

}  // namespace proj
