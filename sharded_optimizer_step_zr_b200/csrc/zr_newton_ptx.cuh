// Device pieces that the Newton-Schulz kernels share: the scratch's number
// formats, waits that give up, and the instructions of sm_100a that have no
// C++ form.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

namespace zr {
namespace {

// Operands are fp16 values times a fixed power of two, which keeps small
// elements out of fp16's subnormals with a factor of 32 to spare above.
constexpr float kNsScaleX = 1024.0f;    // stored X = X * kNsScaleX
constexpr float kNsScaleA = 2048.0f;
constexpr float kNsScaleB = 1024.0f;
constexpr float kNsScaleLo = 2048.0f;   // stored error = (X * kNsScaleX - stored X) * kNsScaleLo

// Factors of the accumulator, the elementwise term and the diagonals: of A,
// B, an update of X and the last one, whose result is not scaled.
struct Affine { float alpha, beta, gamma; };
inline void ns_factors(Affine (&k)[4], const float coeffs[3]) {
    const float a = coeffs[0], b = coeffs[1], c = coeffs[2];
    k[0] = {kNsScaleA / (kNsScaleX * kNsScaleX), 0.0f, 0.0f};
    k[1] = {c * (kNsScaleB / (kNsScaleA * kNsScaleA)), b * (kNsScaleB / kNsScaleA), c * kNsScaleB};
    k[2] = {1.0f / kNsScaleB, a, 1.0f};
    k[3] = {1.0f / (kNsScaleB * kNsScaleX), a / kNsScaleX, 1.0f / kNsScaleX};
}

// kNsScaleX / (norm + eps) from the sum of squares, as two fp32 factors, a
// power of two and the rest, so that neither leaves fp32's normal range for
// any norm of fp32 data (a product with the power of two is exact).
__device__ __forceinline__ float2 ns_scale_of(double sum, double eps) {
    const double d = sqrt(sum) + eps;
    int e = 0;
    if (isfinite(d) && d > 0.0) e = -ilogb(d);
    e = e < -100 ? -100 : e > 100 ? 100 : e;
    return make_float2(static_cast<float>(scalbn(1.0, e)), static_cast<float>(static_cast<double>(kNsScaleX) / scalbn(d, e)));
}

// ---------------------------------------------------------------------------
// PTX
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// One lane of a whole warp.  The compiler knows that a branch on it has one
// thread, and issues copies and products in it from uniform registers; in a
// branch on the lane's number each costs some 300 and 75 cycles.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint32_t leader_address(uint32_t addr) {     // the same address in the pair's first CTA
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}
// Orders no memory: what the arrival announces is that tensor memory has been
// read (tcgen05.wait::ld and the fence before it).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ uint64_t now_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
// A word of this block's shared memory that announces what its writer has seen or done.
__device__ __forceinline__ void st_shared_release(uint32_t addr, uint32_t v) {
    asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_shared_acquire(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ void red_release(uint32_t* p, uint32_t v) {
    asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// Waits are bounded: a wait that lasts kWaitNs gives up -- it sets the
// launch's abort word and the caller's status word, every role of every CTA
// leaves its loop, and the kernel returns with its results unfinished.  The
// longest wait of a sound launch is one product of the whole batch (a second
// for 100000 x 100000).
constexpr uint64_t kWaitNs = 20ull * 1000 * 1000 * 1000;
constexpr uint32_t kWaitTries = 1u << 30;
constexpr uint32_t kDrainTries = 1u << 14;

struct Bail {
    volatile uint32_t* local;     // shared: this CTA's flag
    uint32_t* word;               // global: the launch's
    uint32_t* gave_up;            // global: the caller's
};

template <typename Ready>
__device__ __noinline__ bool wait_slow(Ready ready, const Bail& b) {
    const uint64_t start = now_ns();
    for (uint32_t i = 0; i < kWaitTries; ++i) {
        if (ready()) return true;
        if ((i & 63) != 63) continue;
        if (*b.local) return false;
        if (*reinterpret_cast<volatile uint32_t*>(b.word)) break;
        if (now_ns() - start > kWaitNs) {
            atomicExch(b.gave_up, 1u);
            break;
        }
    }
    *b.local = 1u;
    atomicExch(b.word, 1u);
    return false;
}
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, const Bail& b) {
    if (mbar_try(bar, parity)) return true;
    return wait_slow([=] { return mbar_try(bar, parity); }, b);
}
__device__ __forceinline__ bool count_wait(const uint32_t* p, uint32_t need, const Bail& b) {
    if (ld_acquire(p) >= need) return true;
    return wait_slow([=] { return ld_acquire(p) >= need; }, b);
}

// An operand box; its bytes count on the leader's barrier.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, int x, int y, int z, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
                 ::"l"(map), "r"(x), "r"(y), "r"(z), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, int x, int y, int z, int w, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];"
                 ::"l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void store_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void fence_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }
// Before a block's first use of a tensor map that a copy from the host wrote
// to global memory (hence the system's scope).
__device__ __forceinline__ void fence_tensor_map(const CUtensorMap* map) {
    asm volatile("fence.proxy.tensormap::generic.acquire.sys [%0], 128;" ::"l"(map) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

// Shared-memory matrix descriptor, 128-byte swizzle.  K-major: rows of 128
// bytes (64 contraction elements), groups of 8 rows 1024 bytes apart.
// MN-major: rows of 64 row-or-column elements, one per contraction index;
// groups of 8 contraction indices 1024 bytes apart, chunks of 64 elements
// `chunk` bytes apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, bool mn_major, uint32_t chunk) {
    const uint64_t lead = mn_major ? (chunk >> 4) : 1;
    return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (lead << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives on the barrier at this address in both CTAs of the pair.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// Two fp32 values as one operand of the packed instructions.
using f32x2 = uint64_t;
__device__ __forceinline__ f32x2 pack2(float x, float y) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpack2(f32x2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 32 columns of an accumulator's row.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, f32x2 (&v)[16]) {
    float r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
          "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
          "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
          "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(addr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = pack2(r[2 * i], r[2 * i + 1]);
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
    uint4 q;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(addr) : "memory");
    return q;
}
__device__ __forceinline__ void st_shared16(uint32_t addr, uint4 q) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(q.x), "r"(q.y), "r"(q.z), "r"(q.w) : "memory");
}
__device__ __forceinline__ void st_shared2(uint32_t addr, uint16_t v) {
    asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void ld_shared_f32x4(uint32_t addr, f32x2 (&v)[2]) {
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v[0]), "=l"(v[1]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint16_t ld_shared2(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
    return v;
}

// ---------------------------------------------------------------------------
// number formats
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint16_t half_bits(float x) {
    const __half h = __float2half_rn(x);
    uint16_t u;
    memcpy(&u, &h, 2);
    return u;
}
__device__ __forceinline__ float half_value(uint16_t u) {
    __half h;
    memcpy(&h, &u, 2);
    return __half2float(h);
}
__device__ __forceinline__ uint16_t bf16_bits(float x) {
    const __nv_bfloat16 h = __float2bfloat16_rn(x);
    uint16_t u;
    memcpy(&u, &h, 2);
    return u;
}
__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    uint32_t u;
    memcpy(&u, &h, 4);
    return u;
}
__device__ __forceinline__ float2 half2_values(uint32_t u) {
    __half2 h;
    memcpy(&h, &u, 4);
    return __half22float2(h);
}

// Half a staged row: 32 fp16 values of row `r` from 16-byte piece `first` on,
// in the order that the 128-byte swizzle gives the pieces.
__device__ __forceinline__ uint32_t staged(uint32_t part, int r, int piece) {
    return part + r * 128 + ((piece ^ (r & 7)) << 4);
}
__device__ __forceinline__ void ld_staged32(uint32_t part, int r, int first, f32x2 (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 q = ld_shared16(staged(part, r, first + i));
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = half2_values(w[j]);
            v[4 * i + j] = pack2(f.x, f.y);
        }
    }
}

}  // namespace
}  // namespace zr
