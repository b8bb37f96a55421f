// layers.cuh — what the entry points of uno_layers.h share: argument checks, e4m3 conversion,
// register pairs and clusters.
#pragma once

#include <cuda_bf16.h>

#include "../../include/uno_layers.h"
#include "common.cuh"

namespace uno {

constexpr int kBlockCols = 128;      // columns of a scale block
constexpr float kE4m3Max = 448.0f;   // largest e4m3 value
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126

// the devices an entry point keeps per-device facts for
constexpr int kDevices = 64;

inline bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

inline bool bad_dtype(uno_dtype t) { return t != UNO_BF16 && t != UNO_F32; }

// SMs of the current device (0 on failure)
int device_sms();

// two floats to two e4m3 bytes, the first in the low byte
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
}

// two float32 values in a register pair
__device__ __forceinline__ uint64_t pair_of(float x, float y) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
    return v;
}
__device__ __forceinline__ float2 two(uint64_t v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}

// the calling CTA's place in its cluster, the cluster's CTAs, and a barrier of all their threads
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

}  // namespace uno
