// host.hpp -- what the host sides of the entry points share: environment
// switches, size and device checks, stream-ordered scratch memory.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <initializer_list>
#include <mutex>
#include <string>

#include "kernels.hpp"
#include "selscan.h"

namespace selscan {
namespace host {

inline int64_t env_int(const char* name, int64_t dflt) {
    const char* v = std::getenv(name);
    if (!v || !*v) return dflt;
    return std::strtoll(v, nullptr, 10);
}

inline bool log_plans() { return env_int("SELSCAN_LOG", 0) != 0; }

// Compute units of the current device (256 on MI355X); cached per device.
inline int device_cus() {
    static std::mutex mu;
    static int cache[64] = {0};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    std::lock_guard<std::mutex> lk(mu);
    if (!cache[dev]) {
        int cus = 0;
        if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0)
            cus = 256;
        cache[dev] = cus;
    }
    return cache[dev];
}

// Overflow-checked product of non-negative sizes; -1 on overflow.
inline int64_t mul_checked(std::initializer_list<int64_t> xs) {
    int64_t r = 1;
    for (int64_t x : xs) {
        if (x < 0) return -1;
        if (x != 0 && r > INT64_MAX / x) return -1;
        r *= x;
    }
    return r;
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The current device must be a gfx950.  The architecture check runs once per
// device (cached like device_cus()); later calls only read the current device.
inline selscan_status_t device_check() {
    static std::mutex mu;
    static signed char arch_state[64] = {0};   // 0 unknown, 1 gfx950, -1 other
    static std::string other[64];
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) return set_error(SELSCAN_ERR_NO_DEVICE, "no HIP device available");
    if (dev < 64) {
        std::lock_guard<std::mutex> lk(mu);
        if (arch_state[dev] == 1) return SELSCAN_OK;
        if (arch_state[dev] == -1)
            return set_error(SELSCAN_ERR_NO_DEVICE, "libselscan is built for gfx950, device is " + other[dev]);
    }
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess)
        return set_error(SELSCAN_ERR_NO_DEVICE, "cannot query the HIP device");
    const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    if (dev < 64) {
        std::lock_guard<std::mutex> lk(mu);
        arch_state[dev] = ok ? 1 : -1;
        if (!ok) other[dev] = prop.gcnArchName;
    }
    if (!ok)
        return set_error(SELSCAN_ERR_NO_DEVICE, std::string("libselscan is built for gfx950, device is ") +
                                               prop.gcnArchName);
    return SELSCAN_OK;
}

// Stream-ordered scratch: the caller's workspace when given, else an
// allocation freed on the same stream after the launches.
struct Scratch {
    void* ptr = nullptr;
    bool owned = false;
    hipStream_t stream = nullptr;
    selscan_status_t get(void* user, size_t user_bytes, size_t need, hipStream_t st) {
        stream = st;
        if (need == 0) return SELSCAN_OK;
        if (user) {
            if (user_bytes < need)
                return set_error(SELSCAN_ERR_WORKSPACE, "workspace is smaller than the required " + std::to_string(need) +
                                                       " bytes");
            if ((reinterpret_cast<uintptr_t>(user) & 255) != 0)
                return set_error(SELSCAN_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
            ptr = user;
            return SELSCAN_OK;
        }
        if (hipMallocAsync(&ptr, need, st) != hipSuccess) {
            (void)hipGetLastError();
            return set_error(SELSCAN_ERR_LAUNCH, "hipMallocAsync of " + std::to_string(need) + " workspace bytes failed");
        }
        owned = true;
        return SELSCAN_OK;
    }
    void release() {
        if (owned && ptr) (void)hipFreeAsync(ptr, stream);
        ptr = nullptr;
        owned = false;
    }
};

}  // namespace host
}  // namespace selscan
