// What the C ABI's translation units share: checks of arguments on the host, before any HIP call.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>

#include "../../include/kda.h"

namespace {

constexpr int64_t kMaxElems = (int64_t)1 << 60;

bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
bool valid_io(kda_dtype_t t) { return t == KDA_DTYPE_FP32 || t == KDA_DTYPE_BF16; }
bool valid_decay(kda_decay_t d) { return d == KDA_DECAY_PER_TOKEN || d == KDA_DECAY_PER_HEAD; }
bool supported_dim(int32_t d) { return d == 32 || d == 64 || d == 128; }
size_t elem(kda_dtype_t t) { return t == KDA_DTYPE_BF16 ? 2 : 4; }

// A range of device memory a call reads or writes; p null: absent.
struct Range {
    const void *p;
    int64_t bytes;
};
bool meet(const Range &a, const Range &b) {
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}
// Whether any written range meets a read one or another written one.
template <int NO, int NI>
bool clash(const Range (&out)[NO], const Range (&in)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < NI; ++j)
            if (meet(out[i], in[j])) return true;
        for (int j = i + 1; j < NO; ++j)
            if (meet(out[i], out[j])) return true;
    }
    return false;
}

kda_status_t check_device() {
    static std::atomic<bool> found{false};  // a device that was visible stays so
    if (found.load(std::memory_order_relaxed)) return KDA_SUCCESS;
    int n = 0;
    if (hipGetDeviceCount(&n) != hipSuccess || n < 1) {
        (void)hipGetLastError();
        return KDA_ERROR_NO_DEVICE;
    }
    found.store(true, std::memory_order_relaxed);
    return KDA_SUCCESS;
}
kda_status_t launched(hipError_t e) {
    if (e == hipSuccess) return KDA_SUCCESS;
    (void)hipGetLastError();
    return KDA_ERROR_HIP;
}

}  // namespace
