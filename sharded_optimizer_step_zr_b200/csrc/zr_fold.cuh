// The replica fold and the streaming loads and stores that the elementwise
// passes share (zr_kernels.cu: the AdamW step; zr_muon.cu: the momentum pass).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "zr_internal.hpp"

namespace zr {
namespace {

template <int CAP>
struct GradPtrs {
    const uint16_t* p[CAP];
};

// ---------------------------------------------------------------------------
// memory helpers
// ---------------------------------------------------------------------------

// Read-only streaming 16-byte load (gradients are never written by the step).
__device__ __forceinline__ uint4 ld_grad16(const uint16_t* p) {
    uint4 r;
    asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
        : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
        : "l"(p));
    return r;
}

__device__ __forceinline__ uint16_t ld_grad2(const uint16_t* p) {
    unsigned short r;
    asm("ld.global.nc.L1::no_allocate.u16 %0, [%1];" : "=h"(r) : "l"(p));
    return r;
}

__device__ __forceinline__ float4 ld_state16(const float* p) { return __ldcs(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ void st_state16(float* p, float4 x) { __stcs(reinterpret_cast<float4*>(p), x); }

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float bf16_1(uint16_t h) { return __uint_as_float(static_cast<uint32_t>(h) << 16); }

__device__ __forceinline__ void unpack8(const uint4 q, float s[8]) {
    s[0] = bf16_lo(q.x); s[1] = bf16_hi(q.x);
    s[2] = bf16_lo(q.y); s[3] = bf16_hi(q.y);
    s[4] = bf16_lo(q.z); s[5] = bf16_hi(q.z);
    s[6] = bf16_lo(q.w); s[7] = bf16_hi(q.w);
}

__device__ __forceinline__ void add8(const uint4 q, float s[8]) {
    s[0] = __fadd_rn(s[0], bf16_lo(q.x)); s[1] = __fadd_rn(s[1], bf16_hi(q.x));
    s[2] = __fadd_rn(s[2], bf16_lo(q.y)); s[3] = __fadd_rn(s[3], bf16_hi(q.y));
    s[4] = __fadd_rn(s[4], bf16_lo(q.z)); s[5] = __fadd_rn(s[5], bf16_hi(q.z));
    s[6] = __fadd_rn(s[6], bf16_lo(q.w)); s[7] = __fadd_rn(s[7], bf16_hi(q.w));
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);   // RNE on both halves
    uint32_t u;
    memcpy(&u, &h, 4);
    return u;
}

// Args: any launch arguments with world_size, w_is_pow2 and inv_w
// (set_world_size).
template <typename Args>
__device__ __forceinline__ float average(float s, const Args& a) {
    // Division by a power of two is exact scaling: multiplying by 1/W gives
    // the same correctly rounded value as the division (zr_debug_average_check
    // compares the two on every fp32 input).
    return a.w_is_pow2 ? __fmul_rn(s, a.inv_w) : __fdiv_rn(s, static_cast<float>(a.world_size));
}

// Left fold of W replicas for 8 consecutive owned elements at `off`.  The
// loads of one group of G replicas are all issued before the first add.
template <int CAP, int G>
__device__ __forceinline__ void fold8(const GradPtrs<CAP>& gp, int W, int64_t off, float s[8]) {
    uint4 q[G];
#pragma unroll
    for (int j = 0; j < G; ++j)
        if (j < W) q[j] = ld_grad16(gp.p[j] + off);
    unpack8(q[0], s);
#pragma unroll
    for (int j = 1; j < G; ++j)
        if (j < W) add8(q[j], s);
    if constexpr (CAP > G && CAP <= 2 * G) {
        // At most one more group (W = 9 .. 16): its replica indices are
        // compile-time constants, so the pointer array stays in the
        // parameter bank (a runtime index made the compiler copy it to
        // local memory, 128 bytes per thread) and the loads of both groups
        // can be issued together.
        if (W > G) {
#pragma unroll
            for (int j = 0; j < G; ++j)
                if (G + j < W) q[j] = ld_grad16(gp.p[G + j] + off);
#pragma unroll
            for (int j = 0; j < G; ++j)
                if (G + j < W) add8(q[j], s);
        }
    } else if constexpr (CAP > G) {
        for (int w0 = G; w0 < W; w0 += G) {
#pragma unroll
            for (int j = 0; j < G; ++j)
                if (w0 + j < W) q[j] = ld_grad16(gp.p[w0 + j] + off);
#pragma unroll
            for (int j = 0; j < G; ++j)
                if (w0 + j < W) add8(q[j], s);
        }
    }
}

template <int CAP>
__device__ __forceinline__ float fold1(const GradPtrs<CAP>& gp, int W, int64_t off) {
    float s = bf16_1(ld_grad2(gp.p[0] + off));
    if constexpr (CAP <= 16) {
#pragma unroll
        for (int w = 1; w < CAP; ++w)
            if (w < W) s = __fadd_rn(s, bf16_1(ld_grad2(gp.p[w] + off)));
    } else {
        for (int w = 1; w < W; ++w) s = __fadd_rn(s, bf16_1(ld_grad2(gp.p[w] + off)));
    }
    return s;
}

// Deterministic block sum of one double per thread (fixed shuffle tree, then
// warp partials in order).
__device__ double block_sum(double x) {
    __shared__ double warp_part[kThreads / 32];
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) x += __shfl_down_sync(0xFFFFFFFFu, x, d);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) warp_part[warp] = x;
    __syncthreads();
    double total = 0.0;
    if (threadIdx.x == 0) {
        for (int w = 0; w < kThreads / 32; ++w) total += warp_part[w];
    }
    return total;   // valid in thread 0
}

}  // namespace
}  // namespace zr
