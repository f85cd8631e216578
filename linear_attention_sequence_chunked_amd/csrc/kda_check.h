// kda_check.h -- host-side argument checks and error text shared by the C ABI sources.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <string>

#include "../../include/kda.h"

namespace kda {

// detail of the calling thread's last failed call (kda_last_error)
inline std::string& last_error() {
    static thread_local std::string text;
    return text;
}

inline kda_status fail(kda_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    last_error() = buf;
    return s;
}

inline kda_status ok() {
    last_error().clear();
    return KDA_OK;
}

struct Range {
    const char* name;
    uintptr_t lo, hi;  // [lo, hi)
};

inline bool overlaps(const Range& a, const Range& b) {
    return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi;
}

inline Range range(const char* name, const void* p, uint64_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{name, lo, p ? lo + bytes : lo};
}

inline kda_status check_ptr(const char* name, const void* ptr, size_t align) {
    if (!ptr) return fail(KDA_ERR_INVALID_ARGUMENT, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(ptr) % align)
        return fail(KDA_ERR_INVALID_ARGUMENT, "%s is not %zu-byte aligned", name, align);
    return KDA_OK;
}

inline int device_cu_count() {
    static std::atomic<int> cached{0};  // calls may come from several threads
    if (const int known = cached.load(std::memory_order_relaxed)) return known;
    int dev = 0, cus = 0;
    if (hipGetDevice(&dev) == hipSuccess &&
        hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess &&
        cus > 0)
        cached.store(cus, std::memory_order_relaxed);
    else
        cached.store(cus = 256, std::memory_order_relaxed);
    return cus;
}

}  // namespace kda
