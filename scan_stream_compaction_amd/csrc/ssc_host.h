// Host-side helpers shared by the sources of the library: status handling,
// device checks and argument checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include "ssc.h"

namespace ssc {

inline thread_local int g_last_hip_error = 0;

inline int hip_fail(hipError_t e) {
    g_last_hip_error = static_cast<int>(e);
    return SSC_ERR_HIP;
}

#define SSC_TRY(expr)                  \
    do {                               \
        const int rc_ = (expr);        \
        if (rc_ != SSC_OK) return rc_; \
    } while (0)

// Compute units of the current device: the persistent compaction kernel
// runs one workgroup on each.
inline int compute_units(uint32_t *out) {
    static int cus[64];
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_fail(e);
    if (dev >= 0 && dev < 64 && cus[dev] > 0) {
        *out = static_cast<uint32_t>(cus[dev]);
        return SSC_OK;
    }
    int c = 0;
    e = hipDeviceGetAttribute(&c, hipDeviceAttributeMultiprocessorCount, dev);
    if (e != hipSuccess) return hip_fail(e);
    if (c <= 0) return SSC_ERR_DEVICE;
    if (dev >= 0 && dev < 64) cus[dev] = c;
    *out = static_cast<uint32_t>(c);
    return SSC_OK;
}

// Per-device check that the current device is gfx950 with 64-lane waves.
inline int check_device() {
    static int state[64];  // 0 unknown, 1 ok, 2 wrong device
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_fail(e);
    if (dev >= 0 && dev < 64 && state[dev] == 1) return SSC_OK;
    hipDeviceProp_t prop;
    e = hipGetDeviceProperties(&prop, dev);
    if (e != hipSuccess) return hip_fail(e);
    const bool ok = strncmp(prop.gcnArchName, "gfx950", 6) == 0 && prop.warpSize == 64;
    if (dev >= 0 && dev < 64) state[dev] = ok ? 1 : 2;
    return ok ? SSC_OK : SSC_ERR_DEVICE;
}

inline bool overlap(const void *a, size_t abytes, const void *b, size_t bbytes) {
    if (a == nullptr || b == nullptr || abytes == 0 || bbytes == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + bbytes && b0 < a0 + abytes;
}

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int launched() {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? SSC_OK : hip_fail(e);
}

// Arrays of one call with their byte extents: any two that overlap, or a
// pointer below the required alignment, make the call fail.
struct Span {
    const void *p;
    size_t bytes;
};

template <size_t N>
bool spans_overlap(const Span (&a)[N]) {
    for (size_t i = 0; i < N; ++i)
        for (size_t j = i + 1; j < N; ++j)
            if (overlap(a[i].p, a[i].bytes, a[j].p, a[j].bytes)) return true;
    return false;
}

inline size_t elem_bytes(int dtype) { return dtype == SSC_F32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype == SSC_F32 || dtype == SSC_BF16 || dtype == SSC_F16; }

// Calls f with a value of the element type of dtype (an ssc_dtype).
template <class F>
int with_dtype(int dtype, F f) {
    switch (dtype) {
    case SSC_F32: return f(float{});
    case SSC_BF16: return f(__bf16{});
    default: return f(_Float16{});
    }
}

// A view of `dims` nested sizes with strides in elements, the innermost
// contiguous: the elements from its first to past its last (0 for an empty
// one), and whether no two of its indexes share an element.
template <int DIMS>
struct View {
    int64_t size[DIMS], stride[DIMS];

    bool strides_ok() const {  // products of sizes and strides fit into 62 bits
        for (int i = 0; i < DIMS; ++i)
            if (stride[i] < 0 || stride[i] > (int64_t{1} << 46) || size[i] > INT32_MAX) return false;
        for (int i = 0; i < DIMS; ++i)
            if (size[i] > 1 && static_cast<__int128>(size[i]) * stride[i] > (int64_t{1} << 60)) return false;
        return true;
    }
    int64_t extent() const {
        int64_t n = 1;
        for (int i = 0; i < DIMS; ++i) {
            if (size[i] == 0) return 0;
            n += (size[i] - 1) * stride[i];
        }
        return n;
    }
    bool distinct() const {
        int64_t covered = 1;  // elements spanned by the dimensions of smaller strides
        bool used[DIMS] = {};
        for (int i = 0; i < DIMS; ++i) {
            int next = -1;
            for (int j = 0; j < DIMS; ++j)
                if (!used[j] && (next < 0 || stride[j] < stride[next] ||
                                 (stride[j] == stride[next] && size[j] < size[next])))
                    next = j;
            used[next] = true;
            if (size[next] <= 1) continue;
            if (stride[next] < covered) return false;
            covered += (size[next] - 1) * stride[next];
        }
        return true;
    }
};

}  // namespace ssc
