// Helpers of the C ABI's entry points: error messages and argument checks.
#pragma once
#include <cstdarg>
#include <cstdio>

#include "moe_internal.cuh"

#define MOE_EXPORT extern "C" __attribute__((visibility("default")))

namespace moe {
namespace {

__attribute__((format(printf, 2, 3))) moe_status fail(moe_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    try {
        set_last_error(buf);
    } catch (...) {          // no memory for the message: the status still says what happened
    }
    return s;
}

// The runtime keeps a failed call's error until somebody asks; left there, the next checked launch would report it.
__attribute__((unused)) moe_status cuda_fail(cudaError_t e, const char* what) {
    cudaGetLastError();
    return fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr uint32_t kDefaultWaitLimitUs = 2000000u;

// Synchronise, read and clear a device status word.
__attribute__((unused)) moe_status read_status(uint32_t* word, void* stream, uint32_t* flags) {
    uint32_t v = 0;
    cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    if (e == cudaSuccess) e = cudaMemcpy(&v, word, 4, cudaMemcpyDeviceToHost);
    if (e == cudaSuccess && v) e = cudaMemset(word, 0, 4);
    if (e != cudaSuccess) return cuda_fail(e, "reading the status word");
    if (flags) *flags = v;
    if (v & MOE_DEV_WAIT_TIMEOUT) return fail(MOE_ERR_TIMEOUT, "a kernel wait gave up (status 0x%x)", v);
    if (v) return fail(MOE_ERR_DEVICE_CHECK, "a kernel flagged bad data (status 0x%x)", v);
    return MOE_OK;
}

}  // namespace
}  // namespace moe
