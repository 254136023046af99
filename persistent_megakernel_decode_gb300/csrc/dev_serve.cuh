// Shared by the serving operators (cache.cu, attend.cu, sample.cu): host
// status helpers, e4m3 conversions and the record of failed device checks.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "dev_common.cuh"
#include "planner.h"

namespace mk {

inline int serve_cuda_fail(cudaError_t e, const char *what) {
    return set_error(MK_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

// Function attributes are set once per device and kernel: `ready` has a bit
// per kernel for each device (setting them twice at once does no harm).
constexpr int SERVE_MAX_DEVICES = 64, SERVE_SMEM = 227 * 1024;
inline int serve_prepare(const void *f, std::atomic<uint32_t> (&ready)[SERVE_MAX_DEVICES], int bit, bool large_clusters) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return serve_cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= SERVE_MAX_DEVICES) return set_error(MK_ERR_INVALID, "device ordinal out of range");
    if (ready[dev].load(std::memory_order_acquire) >> bit & 1u) return MK_OK;
    e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, SERVE_SMEM);
    if (e == cudaSuccess && large_clusters) e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return serve_cuda_fail(e, "cudaFuncSetAttribute");
    ready[dev].fetch_or(1u << bit, std::memory_order_release);
    return MK_OK;
}

// The cache's arrays with typed pointers, by value in kernel parameters.
struct CacheView {
    uint8_t *k, *v;
    float *ks, *vs;
    int *status;
    int layers, pages, hkv;
    // byte / element offset of (layer, page, head) in units of P * D codes
    DEV size_t at(int layer, int page, int head) const { return ((size_t)layer * pages + page) * hkv + head; }
};

int cache_check(const mk_cache_desc *c, CacheView &v);  // cache.cu

// Keeps the first failed check (code, sequence, position, page).
static __device__ __noinline__ void note_failure(int *status, int code, int seq, int pos, int page) {
    if (status && atomicCAS(&status[0], 0, code) == 0) {
        status[1] = seq;
        status[2] = pos;
        status[3] = page;
    }
}

// e4m3 codes of (lo, hi), lo in the low byte: nearest even, +-448 beyond,
// infinities too; NaN becomes the NaN code.
DEV uint32_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
DEV uint32_t half2_to_e4m3x2(uint32_t h) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
    return r;
}
// Two codes (low 16 bits) as an f16 pair: exact, every e4m3 value is one of f16.
DEV uint32_t e4m3x2_to_half2(uint32_t v) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)(v & 0xffffu)));
    return h;
}
// Four codes as two f16 pairs.
DEV void e4m3x4_to_half2(uint32_t v, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(v));
}
DEV uint32_t half2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
DEV void half2_floats(uint32_t h, float &lo, float &hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(lo), "=f"(hi) : "r"(h));
}
DEV uint32_t bf16_pair(float lo, float hi) {
    return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(lo)) |
           ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(hi)) << 16);
}

}  // namespace mk
