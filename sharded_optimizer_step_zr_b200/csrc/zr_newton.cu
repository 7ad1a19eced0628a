// Newton-Schulz orthogonalisation for B200 (sm_100a): tcgen05 products of
// TMA-fed fp16 tiles.
//
//   X_0 = U / (||U||_F + eps);   A = X X^T,  B = b A + c A A,  X <- a X + B X
//
// (m <= n; for m > n the same polynomial acts from the right, on X^T X, so no
// operand is ever transposed in memory).  A pass over the m x n matrix costs
// g^2 l multiply-adds for A, g^3 for A A (g = min, l = max) and g^2 l for
// B X; A and A A are symmetric and only the tiles that touch the lower
// triangle are computed, each stored twice.  This is bound by the tensor
// cores for every matrix of a model; the small ones are bound by launches.
//
// Number formats.  Operands are fp16, not bf16: the same tensor-core rate,
// and three more bits -- the rounding of X, A and B is what the result's
// error consists of.  The values are bounded -- singular values of X stay
// below about 1.3 -- so fixed powers of two (kNsScale*) keep small elements
// out of fp16's subnormals with a factor of 32 to spare above.  Accumulators
// are fp32 in tensor memory.  What fp16 would lose most is kept beside it:
//   * the diagonals of A and B, which are of order 1 while everything else in
//     them is of order 1 / sqrt(g), stay in fp32 and enter the next product's
//     epilogue, (D + R)^2 = R R + D R + R D + D D for A A, (a + D) X + R X for
//     the update;
//   * X's rounding error is a second fp16 matrix that enters the elementwise
//     term (a + D) X.  Without it a matrix with a few strong directions loses
//     its weak ones to the rounding of the strong.
// After five steps the result is within 4e-4 to 7e-4 of its norm of the exact
// iteration (1e-2 with bf16 operands; 1.2e-3 with fp16 ones alone, and 2e-2
// when 16 directions are 400 times stronger than the rest).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "zr.h"
#include "zr_newton.hpp"

namespace zr {
namespace {

constexpr float kNsScaleX = 1024.0f;    // stored X = X * kNsScaleX
constexpr float kNsScaleA = 2048.0f;
constexpr float kNsScaleB = 1024.0f;
constexpr float kNsScaleLo = 2048.0f;   // stored error = (X * kNsScaleX - stored X) * kNsScaleLo

// ---------------------------------------------------------------------------
// product kernel: shapes
// ---------------------------------------------------------------------------

constexpr int kBM = 128, kBN = 256, kBK = 64;
constexpr int kStages = 4;
constexpr int kBoxBytes = 64 * 64 * 2;                     // one TMA box: 64 rows of 128 bytes
constexpr int kOp1Bytes = kBM / 64 * kBoxBytes;            // 16 KB
constexpr int kOp2Bytes = kBN / 64 * kBoxBytes;            // 32 KB
constexpr int kStageBytes = kOp1Bytes + kOp2Bytes;
constexpr int kGemmThreads = 192;                          // producer, issuer, four epilogue warps
constexpr int kGemmSmem = kStages * kStageBytes + 1024;    // + alignment to a swizzle atom
constexpr int kMaxGroups = 16;

enum class Ns : int { kGram = 0, kPoly = 1, kUpdate = 2, kOut = 3, kApply = 4 };

// One group's share of a launch: D = op1 op2^T, D rows x cols, K = k.
struct GemmGroup {
    CUtensorMap op1, op2;
    int32_t rows, cols, k;
    int32_t op1_mn, op2_mn;           // operand stored with its contraction extent as rows
    int32_t tiles_n, tiles_per_matrix, first_tile;
    int64_t ld, slot;                 // row pitch and matrix pitch of in and out
    const uint16_t *in_hi, *in_lo;    // A (kPoly) or X (kUpdate, kOut, kApply)
    uint16_t *out_hi, *out_lo;
    const float* diag_in;             // A's (kPoly) or B's (kUpdate, kOut, kApply)
    float* diag_out;                  // A's (kGram) or B's (kPoly)
    int32_t diag_rows;                // B acts on X's rows (wide), not its columns
    int64_t out_row, out_batch;       // kOut
    const int64_t *master_offsets, *param_offsets;   // kApply
    float step_size;
};

struct GemmLaunch {
    int32_t n_groups, total_tiles;
    float alpha, beta, gamma, decay;   // of the accumulator, the elementwise term, the diagonals; kApply
    uint32_t* gave_up;
    float* master;
    uint16_t* param_out;
    uint16_t* const* targets;
    int32_t n_targets;
    GemmGroup g[kMaxGroups];
};

// ---------------------------------------------------------------------------
// PTX
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
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

// Waits are bounded: after kWaitTries failed tries (each blocks for up to a
// hardware time slice) the block gives up -- the error word is set, every
// role leaves its loop, and the kernel returns with its results unfinished.
constexpr int kWaitTries = 1 << 20;
constexpr int kDrainTries = 1 << 14;

__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag,
                                          uint32_t* gave_up) {
    if (mbar_try(bar, parity)) return true;
    for (int i = 0; i < kWaitTries; ++i) {
        if (mbar_try(bar, parity)) return true;
        if ((i & 63) == 63 && *abort_flag) return false;
    }
    *abort_flag = 1u;
    atomicExch(gave_up, 1u);
    return false;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle.  K-major: rows of 128
// bytes (64 contraction elements), groups of 8 rows 1024 bytes apart.
// MN-major: rows of 64 row-or-column elements, one per contraction index;
// groups of 8 contraction indices 1024 bytes apart, chunks of 64 elements
// one TMA box apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, bool mn_major) {
    const uint64_t lead = mn_major ? (kBoxBytes >> 4) : 1;
    return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (lead << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t addr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// ---------------------------------------------------------------------------
// epilogue pieces
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

// 32 consecutive fp16 values at a 16-byte aligned address.
__device__ __forceinline__ void ld_half32(const uint16_t* p, float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 q = *reinterpret_cast<const uint4*>(p + 8 * i);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[8 * i + 2 * j] = half_value(static_cast<uint16_t>(w[j]));
            v[8 * i + 2 * j + 1] = half_value(static_cast<uint16_t>(w[j] >> 16));
        }
    }
}
__device__ __forceinline__ void st_half32(uint16_t* p, const uint16_t (&h)[32]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint4 q;
        q.x = h[8 * i] | (static_cast<uint32_t>(h[8 * i + 1]) << 16);
        q.y = h[8 * i + 2] | (static_cast<uint32_t>(h[8 * i + 3]) << 16);
        q.z = h[8 * i + 4] | (static_cast<uint32_t>(h[8 * i + 5]) << 16);
        q.w = h[8 * i + 6] | (static_cast<uint32_t>(h[8 * i + 7]) << 16);
        *reinterpret_cast<uint4*>(p + 8 * i) = q;
    }
}

// Which tile: its group, matrix and position.  Symmetric results (A, B) list
// only tiles that touch the lower triangle: of row blocks 2p and 2p + 1 (128
// rows each), the first p + 1 column blocks (256 columns each).
struct TileAt {
    int32_t group, slot, row0, col0;
};

template <bool SYM>
__device__ __forceinline__ TileAt find_tile(const GemmLaunch& L, int32_t tile) {
    int32_t gi = 0;
    while (gi + 1 < L.n_groups && tile >= L.g[gi + 1].first_tile) ++gi;
    const GemmGroup& g = L.g[gi];
    const int32_t t = tile - g.first_tile;
    TileAt at;
    at.group = gi;
    at.slot = t / g.tiles_per_matrix;
    const int32_t r = t - at.slot * g.tiles_per_matrix;
    if constexpr (SYM) {
        int32_t p = static_cast<int32_t>((sqrtf(4.0f * static_cast<float>(r) + 1.0f) - 1.0f) * 0.5f);
        while (static_cast<int64_t>(p + 1) * (p + 2) <= r) ++p;
        while (static_cast<int64_t>(p) * (p + 1) > r) --p;
        const int32_t rem = r - p * (p + 1);
        const int32_t second = rem >= p + 1 ? 1 : 0;
        at.row0 = (2 * p + second) * kBM;
        at.col0 = (rem - second * (p + 1)) * kBN;
    } else {
        at.row0 = (r / g.tiles_n) * kBM;
        at.col0 = (r % g.tiles_n) * kBN;
    }
    return at;
}

// ---------------------------------------------------------------------------
// the product kernel
// ---------------------------------------------------------------------------

// One CTA per SM walks the tiles of all groups.  Warp 0 feeds a ring of four
// 48 KB stages by TMA, warp 1 issues the tensor-core instructions into one of
// two accumulators, warps 2 to 5 empty the other one, so a tile's epilogue
// runs under the next tile's products.
template <Ns MODE>
__global__ void __launch_bounds__(kGemmThreads, 1) zr_ns_product_kernel(const __grid_constant__ GemmLaunch L) {
    constexpr bool kSym = MODE == Ns::kGram || MODE == Ns::kPoly;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * kStages + 4];
    __shared__ uint32_t s_tmem;
    __shared__ volatile uint32_t s_abort;
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t full = smem_u32(bars), empty = full + 8 * kStages;
    const uint32_t acc_full = empty + 8 * kStages, acc_empty = acc_full + 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        s_abort = 0u;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(acc_empty + 8 * i, 4);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = s_tmem;
    // The previous kernel wrote the operands; nothing above read memory.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == 0) {
        if (lane == 0) {
            // ordinary stores wrote what the copies below read
            asm volatile("fence.proxy.async.global;" ::: "memory");
            uint32_t it = 0;
            bool ok = true;
            for (int32_t tile = blockIdx.x; ok && tile < L.total_tiles; tile += gridDim.x) {
                const TileAt at = find_tile<kSym>(L, tile);
                const GemmGroup& g = L.g[at.group];
                const int32_t nk = (g.k + kBK - 1) / kBK;
                for (int32_t kb = 0; kb < nk; ++kb, ++it) {
                    const uint32_t s = it % kStages, phase = (it / kStages) & 1;
                    if (!mbar_wait(empty + 8 * s, phase ^ 1, &s_abort, L.gave_up)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = full + 8 * s, dst = smem + s * kStageBytes;
                    mbar_expect(bar, kStageBytes);
                    const int k0 = kb * kBK;
#pragma unroll
                    for (int b = 0; b < kBM / 64; ++b) {
                        const int r = at.row0 + 64 * b;
                        tma_load_3d(dst + b * kBoxBytes, &g.op1, g.op1_mn ? r : k0, g.op1_mn ? k0 : r, at.slot, bar);
                    }
#pragma unroll
                    for (int b = 0; b < kBN / 64; ++b) {
                        const int c = at.col0 + 64 * b;
                        tma_load_3d(dst + kOp1Bytes + b * kBoxBytes, &g.op2, g.op2_mn ? c : k0, g.op2_mn ? k0 : c,
                                    at.slot, bar);
                    }
                }
            }
            // A block that gave up may still have copies in flight into its
            // shared memory: see them land (each ring slot's last fill).
            if (s_abort)
                for (uint32_t back = 1; back <= kStages && back <= it; ++back) {
                    const uint32_t last = it - back;
                    for (int i = 0; i < kDrainTries && !mbar_try(full + 8 * (last % kStages), (last / kStages) & 1); ++i) {}
                }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            uint32_t it = 0, acc = 0;
            bool ok = true;
            for (int32_t tile = blockIdx.x; ok && tile < L.total_tiles; tile += gridDim.x, ++acc) {
                const TileAt at = find_tile<kSym>(L, tile);
                const GemmGroup& g = L.g[at.group];
                const int32_t nk = (g.k + kBK - 1) / kBK;
                const uint32_t buf = acc & 1;
                if (!mbar_wait(acc_empty + 8 * buf, ((acc >> 1) & 1) ^ 1, &s_abort, L.gave_up)) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t d = tmem + buf * kBN;
                // fp32 accumulators, fp16 operands, their majors, N / 8, M / 16
                const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(g.op1_mn) << 15) |
                                       (static_cast<uint32_t>(g.op2_mn) << 16) | ((kBN >> 3) << 17) | ((kBM >> 4) << 24);
                const uint32_t step1 = (g.op1_mn ? 16 * 128 : 32) >> 4, step2 = (g.op2_mn ? 16 * 128 : 32) >> 4;
                for (int32_t kb = 0; kb < nk; ++kb, ++it) {
                    const uint32_t s = it % kStages, phase = (it / kStages) & 1;
                    if (!mbar_wait(full + 8 * s, phase, &s_abort, L.gave_up)) {
                        ok = false;
                        break;
                    }
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint32_t base = smem + s * kStageBytes;
                    const uint64_t d1 = smem_desc(base, g.op1_mn), d2 = smem_desc(base + kOp1Bytes, g.op2_mn);
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk)
                        mma_f16(d, d1 + kk * step1, d2 + kk * step2, idesc, (kb | kk) != 0);
                    mma_commit(empty + 8 * s);
                }
                if (ok) mma_commit(acc_full + 8 * buf);
            }
        }
    } else {
        const int quad = warp & 3;                 // the TMEM lanes this warp may read
        uint32_t acc = 0;
        for (int32_t tile = blockIdx.x; tile < L.total_tiles; tile += gridDim.x, ++acc) {
            const TileAt at = find_tile<kSym>(L, tile);
            const GemmGroup& g = L.g[at.group];
            const uint32_t buf = acc & 1;
            if (!mbar_wait(acc_full + 8 * buf, (acc >> 1) & 1, &s_abort, L.gave_up)) break;
            __syncwarp();
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const int32_t row = at.row0 + quad * 32 + lane;
            const bool live = row < g.rows;
            const int64_t at_row = at.slot * g.slot + static_cast<int64_t>(row) * g.ld;
#pragma unroll 1
            for (int ch = 0; ch < kBN / 32; ++ch) {
                const int32_t c0 = at.col0 + ch * 32;
                if (c0 >= g.cols) break;
                if (kSym && c0 > at.row0 + quad * 32 + 31) break;      // above the diagonal for the whole warp
                float v[32];
                tmem_ld32(tmem + (static_cast<uint32_t>(quad * 32) << 16) + buf * kBN + ch * 32, v);
                if constexpr (MODE == Ns::kGram) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] *= L.alpha;
                } else if (live) {
                    float x[32];
                    ld_half32(g.in_hi + at_row + c0, x);
                    if constexpr (MODE == Ns::kPoly) {
                        // c A A + b A, A = D + R: acc = R R, x = R
                        const float* diag = g.diag_in + static_cast<int64_t>(at.slot) * g.rows;
                        const float dr = diag[row];
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float dc = c0 + i < g.cols ? diag[c0 + i] : 0.0f;
                            v[i] = c0 + i == row ? fmaf(fmaf(dr, L.gamma, L.beta * kNsScaleA), dr, v[i] * L.alpha)
                                                 : fmaf(fmaf(dr + dc, L.gamma * (1.0f / kNsScaleA), L.beta), x[i], v[i] * L.alpha);
                        }
                    } else {
                        float lo[32];
                        ld_half32(g.in_lo + at_row + c0, lo);
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = fmaf(lo[i], 1.0f / kNsScaleLo, x[i]);
                        const float* diag = g.diag_in + static_cast<int64_t>(at.slot) * (g.diag_rows ? g.rows : g.cols);
                        if (g.diag_rows) {
                            const float d = diag[row] * L.gamma + L.beta;
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = fmaf(x[i], d, v[i] * L.alpha);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const float d = c0 + i < g.cols ? diag[c0 + i] * L.gamma + L.beta : 0.0f;
                                v[i] = fmaf(x[i], d, v[i] * L.alpha);
                            }
                        }
                    }
                }
                if constexpr (kSym) {
                    uint16_t h[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) h[i] = half_bits(v[i]);
                    uint16_t* out = g.out_hi + at.slot * g.slot;
                    if (live) {
                        uint16_t* p = out + static_cast<int64_t>(row) * g.ld + c0;
                        if (c0 + 31 < row) {
                            st_half32(p, h);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                if (c0 + i < row) p[i] = h[i];
                                if (c0 + i == row) {
                                    p[i] = 0;
                                    g.diag_out[static_cast<int64_t>(at.slot) * g.rows + row] =
                                        v[i] * (MODE == Ns::kGram ? 1.0f / kNsScaleA : 1.0f / kNsScaleB);
                                }
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 32; ++i)      // the mirror image: a warp's 32 rows are contiguous there
                            if (c0 + i < row) out[static_cast<int64_t>(c0 + i) * g.ld + row] = h[i];
                    }
                } else if constexpr (MODE == Ns::kUpdate) {
                    if (live) {
                        uint16_t h[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) h[i] = half_bits(v[i]);
                        st_half32(g.out_hi + at_row + c0, h);
#pragma unroll
                        for (int i = 0; i < 32; ++i) h[i] = half_bits((v[i] - half_value(h[i])) * kNsScaleLo);
                        st_half32(g.out_lo + at_row + c0, h);
                    }
                } else if constexpr (MODE == Ns::kOut) {
                    if (live) {
                        uint16_t* p = g.out_hi + at.slot * g.out_batch + static_cast<int64_t>(row) * g.out_row + c0;
                        if (c0 + 32 <= g.cols && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
                            uint16_t h[32];
#pragma unroll
                            for (int i = 0; i < 32; ++i) h[i] = bf16_bits(v[i]);
                            st_half32(p, h);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (c0 + i < g.cols) p[i] = bf16_bits(v[i]);
                        }
                    }
                } else {
                    if (live) {
                        const int64_t e = static_cast<int64_t>(row) * g.cols + c0;
                        float* pm = L.master + g.master_offsets[at.slot] + e;
                        const int64_t po = g.param_offsets[at.slot] + e;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            if (c0 + i >= g.cols) continue;
                            const float p = __fsub_rn(__fmul_rn(pm[i], L.decay), __fmul_rn(v[i], g.step_size));
                            pm[i] = p;
                            const uint16_t u = bf16_bits(p);
                            if (L.n_targets == 0) L.param_out[po + i] = u;
                            else
                                for (int t = 0; t < L.n_targets; ++t) L.targets[t][po + i] = u;
                        }
                    }
                }
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty + 8 * buf);
        }
    }
    // Every role is done (or gave up).  Products issued by a block that gave
    // up drain through a commit to the first accumulator's barrier.
    __syncthreads();
    if (s_abort && threadIdx.x == 32) {
        mma_commit(acc_full);
        for (int i = 0; i < kDrainTries; ++i) (void)mbar_try(acc_full, 0);
    }
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    __syncthreads();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ---------------------------------------------------------------------------
// norm and X_0
// ---------------------------------------------------------------------------

constexpr int kPrepThreads = 256;
constexpr int kPrepRows = 8, kPrepCols = kPrepThreads * 4;     // a CTA's piece of one matrix

struct PrepGroup {
    const void* src;
    int32_t dtype, vec;                   // vec: four elements load as one 8- or 16-byte word
    int64_t rows, cols, src_row, src_batch;
    int32_t pieces_n, pieces_per_matrix, batch;
    int64_t first_piece;
    double* partials;
    const int32_t* first_partial;
    int32_t n_partials;
    float2* scale;
    uint16_t *xh, *xl;
    int64_t ld;
};
struct PrepLaunch {
    int32_t n_groups;
    int32_t total_matrices;
    double eps;
    PrepGroup g[kMaxGroups];
};

__device__ __forceinline__ float load_one(const void* p, int32_t dtype, int64_t i) {
    if (dtype == ZR_DTYPE_F32) return static_cast<const float*>(p)[i];
    const uint16_t u = static_cast<const uint16_t*>(p)[i];
    return dtype == ZR_DTYPE_BF16 ? __uint_as_float(static_cast<uint32_t>(u) << 16) : half_value(u);
}

// Four consecutive elements at `i`, of which `count` exist.
__device__ __forceinline__ void load_four(const PrepGroup& g, int64_t i, int64_t count, float (&v)[4]) {
    if (g.vec && count >= 4) {
        if (g.dtype == ZR_DTYPE_F32) {
            const float4 q = *reinterpret_cast<const float4*>(static_cast<const float*>(g.src) + i);
            v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
        } else {
            const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(g.src) + i);
            const uint32_t w[2] = {q.x, q.y};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint16_t u = static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1)));
                v[k] = g.dtype == ZR_DTYPE_BF16 ? __uint_as_float(static_cast<uint32_t>(u) << 16) : half_value(u);
            }
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = k < count ? load_one(g.src, g.dtype, i + k) : 0.0f;
}

struct PieceAt {
    int32_t group, slot, piece;
    int64_t row0, col, src;      // this thread's first column, its element's index in row 0
};

__device__ __forceinline__ PieceAt find_piece(const PrepLaunch& L) {
    PieceAt at;
    const int64_t b = blockIdx.x;
    int32_t gi = 0;
    while (gi + 1 < L.n_groups && b >= L.g[gi + 1].first_piece) ++gi;
    const PrepGroup& g = L.g[gi];
    const int64_t t = b - g.first_piece;
    at.group = gi;
    at.slot = static_cast<int32_t>(t / g.pieces_per_matrix);
    at.piece = static_cast<int32_t>(t - static_cast<int64_t>(at.slot) * g.pieces_per_matrix);
    at.row0 = static_cast<int64_t>(at.piece / g.pieces_n) * kPrepRows;
    at.col = static_cast<int64_t>(at.piece % g.pieces_n) * kPrepCols + threadIdx.x * 4;
    at.src = at.slot * g.src_batch + at.row0 * g.src_row + at.col;
    return at;
}

__device__ double prep_block_sum(double x) {
    __shared__ double part[kPrepThreads / 32];
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) x += __shfl_down_sync(0xFFFFFFFFu, x, d);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    double total = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < kPrepThreads / 32; ++w) total += part[w];
    return total;   // valid in thread 0
}

// Squares are exact in fp64, and so are their sums to 2^-53: one partial per
// piece of 8 x 1024 elements.
__global__ void __launch_bounds__(kPrepThreads) zr_ns_sumsq_kernel(const __grid_constant__ PrepLaunch L) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const PieceAt at = find_piece(L);
    const PrepGroup& g = L.g[at.group];
    double sum = 0.0;
    if (at.col < g.cols) {
#pragma unroll
        for (int r = 0; r < kPrepRows; ++r) {
            if (at.row0 + r >= g.rows) break;
            float v[4];
            load_four(g, at.src + r * g.src_row, g.cols - at.col, v);
#pragma unroll
            for (int k = 0; k < 4; ++k) sum += static_cast<double>(v[k]) * static_cast<double>(v[k]);
        }
    }
    sum = prep_block_sum(sum);
    if (threadIdx.x == 0) g.partials[static_cast<int64_t>(at.slot) * g.n_partials + at.piece] = sum;
}

// One CTA per matrix: the norm, and 1 / (norm + eps) as two fp32 factors, a
// power of two and the rest, so that neither leaves fp32's normal range for
// any norm of fp32 data (a product with the power of two is exact).
__global__ void __launch_bounds__(kPrepThreads) zr_ns_scale_kernel(const __grid_constant__ PrepLaunch L) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    int32_t slot = blockIdx.x, gi = 0;
    while (slot >= L.g[gi].batch) slot -= L.g[gi++].batch;
    const PrepGroup& g = L.g[gi];
    const int64_t first = g.first_partial ? g.first_partial[slot] : static_cast<int64_t>(slot) * g.n_partials;
    const int64_t last = g.first_partial ? g.first_partial[slot + 1] : first + g.n_partials;
    double sum = 0.0;
    for (int64_t i = first + threadIdx.x; i < last; i += kPrepThreads) sum += __ldcg(g.partials + i);
    sum = prep_block_sum(sum);
    if (threadIdx.x == 0) {
        const double d = sqrt(sum) + L.eps;
        int e = 0;
        if (isfinite(d) && d > 0.0) e = -ilogb(d);
        e = e < -100 ? -100 : e > 100 ? 100 : e;
        g.scale[slot] = make_float2(static_cast<float>(scalbn(1.0, e)),
                                    static_cast<float>(static_cast<double>(kNsScaleX) / scalbn(d, e)));
    }
}

__global__ void __launch_bounds__(kPrepThreads) zr_ns_start_kernel(const __grid_constant__ PrepLaunch L) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const PieceAt at = find_piece(L);
    const PrepGroup& g = L.g[at.group];
    if (at.col >= g.cols) return;
    const float2 s = g.scale[at.slot];
    const int64_t out = (static_cast<int64_t>(at.slot) * g.rows + at.row0) * g.ld + at.col;
#pragma unroll
    for (int r = 0; r < kPrepRows; ++r) {
        if (at.row0 + r >= g.rows) break;
        float v[4];
        load_four(g, at.src + r * g.src_row, g.cols - at.col, v);
        uint16_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float x = (v[k] * s.x) * s.y;
            hi[k] = half_bits(x);
            lo[k] = half_bits((x - half_value(hi[k])) * kNsScaleLo);
        }
        // rows of ld elements, a multiple of 64: the last word may reach past
        // the last column, never past the row
        *reinterpret_cast<uint2*>(g.xh + out + r * g.ld) =
            make_uint2(hi[0] | (static_cast<uint32_t>(hi[1]) << 16), hi[2] | (static_cast<uint32_t>(hi[3]) << 16));
        *reinterpret_cast<uint2*>(g.xl + out + r * g.ld) =
            make_uint2(lo[0] | (static_cast<uint32_t>(lo[1]) << 16), lo[2] | (static_cast<uint32_t>(lo[3]) << 16));
    }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// A batch of rows x cols fp16 matrices with rows of ld elements, read in
// boxes of 64 x 64; what lies outside a matrix reads as zero.
int encode_map(CUtensorMap* map, void* base, int64_t cols, int64_t rows, int64_t batch, int64_t ld) {
    const EncodeTiled fn = encode_tiled();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(batch)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(ld) * rows * 2};
    const cuuint32_t box[3] = {64, 64, 1}, unit[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, base, dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

uint64_t align256(uint64_t x) { return (x + 255) & ~uint64_t(255); }

int32_t symmetric_tiles(int64_t g) {
    const int64_t r = (g + kBM - 1) / kBM, p = r / 2;
    return static_cast<int32_t>(p * (p + 1) + (r % 2 ? p + 1 : 0));
}
int64_t full_tiles(int64_t rows, int64_t cols) { return ((rows + kBM - 1) / kBM) * ((cols + kBN - 1) / kBN); }

template <typename Launch>
struct Dependent {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    Dependent(unsigned grid, unsigned block, size_t smem, void* stream) {
        cfg.gridDim = dim3(grid);
        cfg.blockDim = dim3(block);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = static_cast<cudaStream_t>(stream);
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    cudaError_t run(void (*kernel)(Launch), const Launch& l) { return cudaLaunchKernelEx(&cfg, kernel, l); }
};

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 148;
    return n;
}

template <Ns MODE>
int launch_product(GemmLaunch& L, const NsGroup* groups, int32_t n, int32_t from, void* stream) {
    int64_t tiles = 0;
    L.n_groups = n;
    for (int32_t i = 0; i < n; ++i) {
        const NsGroup& s = groups[i];
        GemmGroup& g = L.g[i];
        const bool wide = s.m <= s.n;
        const int64_t dim = s.gram_dim();
        g.first_tile = static_cast<int32_t>(tiles);
        if (MODE == Ns::kGram || MODE == Ns::kPoly) {
            g.rows = g.cols = static_cast<int32_t>(dim);
            g.op1 = g.op2 = MODE == Ns::kGram ? s.map_x[from] : s.map_gram;
            g.k = static_cast<int32_t>(MODE == Ns::kGram ? std::max(s.m, s.n) : dim);
            g.op1_mn = g.op2_mn = MODE == Ns::kGram && !wide;
            g.tiles_per_matrix = symmetric_tiles(dim);
            g.tiles_n = 0;
            g.ld = s.ldg();
            g.slot = dim * s.ldg();
            g.in_hi = s.gram;
            g.out_hi = MODE == Ns::kGram ? s.gram : s.poly;
            g.diag_in = s.gram_diag;
            g.diag_out = MODE == Ns::kGram ? s.gram_diag : s.poly_diag;
        } else {
            // wide: B X, X's rows are the contraction; tall: X B, B symmetric
            g.rows = static_cast<int32_t>(s.m);
            g.cols = static_cast<int32_t>(s.n);
            g.k = static_cast<int32_t>(dim);
            g.op1 = wide ? s.map_poly : s.map_x[from];
            g.op2 = wide ? s.map_x[from] : s.map_poly;
            g.op1_mn = 0;
            g.op2_mn = wide ? 1 : 0;
            g.tiles_n = static_cast<int32_t>((s.n + kBN - 1) / kBN);
            g.tiles_per_matrix = static_cast<int32_t>(full_tiles(s.m, s.n));
            g.ld = s.ld();
            g.slot = s.m * s.ld();
            g.in_hi = s.xh[from];
            g.in_lo = s.xl[from];
            g.diag_in = s.poly_diag;
            g.diag_rows = wide ? 1 : 0;
            if (MODE == Ns::kUpdate) {
                g.out_hi = s.xh[from ^ 1];
                g.out_lo = s.xl[from ^ 1];
            } else {
                g.out_hi = s.out;
                g.out_row = s.out_row;
                g.out_batch = s.out_batch;
                g.master_offsets = s.master_offsets;
                g.param_offsets = s.param_offsets;
                g.step_size = s.step_size;
            }
        }
        tiles += s.batch * g.tiles_per_matrix;
        if (tiles > 0x7FFFFFFF) return cudaErrorInvalidValue;
    }
    L.total_tiles = static_cast<int32_t>(tiles);
    cudaError_t e = cudaFuncSetAttribute(zr_ns_product_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kGemmSmem);
    if (e != cudaSuccess) return e;
    const int sms = sm_count();
    Dependent<GemmLaunch> d(static_cast<unsigned>(std::min<int64_t>(tiles, sms)), kGemmThreads, kGemmSmem, stream);
    return d.run(zr_ns_product_kernel<MODE>, L);
}

int64_t fill_prep(PrepLaunch& L, const NsGroup* groups, int32_t n) {
    int64_t pieces = 0, matrices = 0;
    L.n_groups = n;
    for (int32_t i = 0; i < n; ++i) {
        const NsGroup& s = groups[i];
        PrepGroup& g = L.g[i];
        g.src = s.src;
        g.dtype = s.src_dtype;
        const int64_t bytes = s.src_dtype == ZR_DTYPE_F32 ? 16 : 8;
        g.vec = reinterpret_cast<uintptr_t>(s.src) % bytes == 0 && s.src_row % 4 == 0 && s.src_batch % 4 == 0;
        g.rows = s.m;
        g.cols = s.n;
        g.src_row = s.src_row;
        g.src_batch = s.src_batch;
        g.pieces_n = static_cast<int32_t>((s.n + kPrepCols - 1) / kPrepCols);
        g.pieces_per_matrix = static_cast<int32_t>(ns_partials_per_matrix(s.m, s.n));
        g.batch = static_cast<int32_t>(s.batch);
        g.first_piece = pieces;
        g.partials = s.partials;
        g.first_partial = s.first_partial;
        g.n_partials = s.n_partials;
        g.scale = s.scale;
        g.xh = s.xh[0];
        g.xl = s.xl[0];
        g.ld = s.ld();
        pieces += s.batch * g.pieces_per_matrix;
        matrices += s.batch;
    }
    L.total_matrices = static_cast<int32_t>(matrices);
    return pieces;
}

}  // namespace

int64_t ns_partials_per_matrix(int64_t m, int64_t n) {
    return ((m + kPrepRows - 1) / kPrepRows) * ((n + kPrepCols - 1) / kPrepCols);
}

bool ns_shape_fits(int64_t batch, int64_t m, int64_t n) {
    // Extents small enough that no count below overflows; then tile and
    // piece counts within 32 bits and scratch within 2^47 bytes.
    if (m > (1 << 24) || n > (1 << 24) || batch > (1 << 24)) return false;
    const double total = static_cast<double>(batch) * static_cast<double>(m) * static_cast<double>(n);
    if (total > 2.0e12) return false;
    const int64_t g = std::min(m, n);
    if (g > (1 << 17)) return false;
    return batch * full_tiles(m, n) < (1ll << 31) && batch * ns_partials_per_matrix(m, n) < (1ll << 31) &&
           batch * symmetric_tiles(g) < (1ll << 31);
}

uint64_t ns_scratch_bytes(int64_t batch, int64_t m, int64_t n) {
    NsGroup g;
    g.batch = batch;
    g.m = m;
    g.n = n;
    const uint64_t x = align256(static_cast<uint64_t>(batch) * m * g.ld() * 2);
    const uint64_t a = align256(static_cast<uint64_t>(batch) * g.gram_dim() * g.ldg() * 2);
    return 4 * x + 2 * a + 2 * align256(static_cast<uint64_t>(batch) * g.gram_dim() * sizeof(float));
}

uint64_t ns_source_offset(int64_t batch, int64_t m, int64_t n) {
    NsGroup g;
    g.n = n;
    return 2 * align256(static_cast<uint64_t>(batch) * m * g.ld() * 2);
}

int ns_bind_scratch(NsGroup& g, void* base) {
    const uint64_t x = align256(static_cast<uint64_t>(g.batch) * g.m * g.ld() * 2);
    const uint64_t a = align256(static_cast<uint64_t>(g.batch) * g.gram_dim() * g.ldg() * 2);
    char* p = static_cast<char*>(base);
    for (int i = 0; i < 2; ++i) {
        g.xh[i] = reinterpret_cast<uint16_t*>(p + 2 * i * x);
        g.xl[i] = reinterpret_cast<uint16_t*>(p + (2 * i + 1) * x);
    }
    g.gram = reinterpret_cast<uint16_t*>(p + 4 * x);
    g.poly = reinterpret_cast<uint16_t*>(p + 4 * x + a);
    g.gram_diag = reinterpret_cast<float*>(p + 4 * x + 2 * a);
    g.poly_diag = reinterpret_cast<float*>(
        p + 4 * x + 2 * a + align256(static_cast<uint64_t>(g.batch) * g.gram_dim() * sizeof(float)));
    int e = cudaSuccess;
    for (int i = 0; i < 2 && e == cudaSuccess; ++i) e = encode_map(&g.map_x[i], g.xh[i], g.n, g.m, g.batch, g.ld());
    if (e == cudaSuccess) e = encode_map(&g.map_gram, g.gram, g.gram_dim(), g.gram_dim(), g.batch, g.ldg());
    if (e == cudaSuccess) e = encode_map(&g.map_poly, g.poly, g.gram_dim(), g.gram_dim(), g.batch, g.ldg());
    return e;
}

int launch_ns_sumsq(const NsGroup* groups, int32_t n_groups, void* stream) {
    for (int32_t at = 0; at < n_groups; at += kMaxGroups) {
        PrepLaunch L{};
        const int64_t pieces = fill_prep(L, groups + at, std::min(kMaxGroups, n_groups - at));
        if (pieces > 0x7FFFFFFF) return cudaErrorInvalidValue;
        Dependent<PrepLaunch> d(static_cast<unsigned>(pieces), kPrepThreads, 0, stream);
        const cudaError_t e = d.run(zr_ns_sumsq_kernel, L);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

int launch_ns_scales(const NsGroup* groups, int32_t n_groups, double eps, void* stream) {
    for (int32_t at = 0; at < n_groups; at += kMaxGroups) {
        PrepLaunch L{};
        fill_prep(L, groups + at, std::min(kMaxGroups, n_groups - at));
        L.eps = eps;
        Dependent<PrepLaunch> d(static_cast<unsigned>(L.total_matrices), kPrepThreads, 0, stream);
        const cudaError_t e = d.run(zr_ns_scale_kernel, L);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

int launch_ns_iterations(const NsGroup* groups, int32_t n_groups, int32_t steps, const float coeffs[3],
                         const NsApply& apply, uint32_t* gave_up, void* stream) {
    const float a = coeffs[0], b = coeffs[1], c = coeffs[2];
    for (int32_t at = 0; at < n_groups; at += kMaxGroups) {
        const NsGroup* gs = groups + at;
        const int32_t n = std::min(kMaxGroups, n_groups - at);
        {
            PrepLaunch P{};
            const int64_t pieces = fill_prep(P, gs, n);
            if (pieces > 0x7FFFFFFF) return cudaErrorInvalidValue;
            Dependent<PrepLaunch> d(static_cast<unsigned>(pieces), kPrepThreads, 0, stream);
            const cudaError_t e = d.run(zr_ns_start_kernel, P);
            if (e != cudaSuccess) return e;
        }
        GemmLaunch L{};
        L.gave_up = gave_up;
        L.master = apply.master;
        L.param_out = apply.param_out;
        L.targets = apply.targets;
        L.n_targets = apply.n_targets;
        L.decay = apply.decay;
        for (int32_t i = 0; i < steps; ++i) {
            const int32_t from = i & 1;
            const bool last = i + 1 == steps;
            L.alpha = kNsScaleA / (kNsScaleX * kNsScaleX);
            int e = launch_product<Ns::kGram>(L, gs, n, from, stream);
            if (e != cudaSuccess) return e;
            L.alpha = c * (kNsScaleB / (kNsScaleA * kNsScaleA));
            L.beta = b * (kNsScaleB / kNsScaleA);
            L.gamma = c * kNsScaleB;
            e = launch_product<Ns::kPoly>(L, gs, n, from, stream);
            if (e != cudaSuccess) return e;
            if (!last) {
                L.alpha = 1.0f / kNsScaleB;
                L.beta = a;
                L.gamma = 1.0f;
                e = launch_product<Ns::kUpdate>(L, gs, n, from, stream);
            } else {
                L.alpha = 1.0f / (kNsScaleB * kNsScaleX);
                L.beta = a / kNsScaleX;
                L.gamma = 1.0f / kNsScaleX;
                e = apply.master ? launch_product<Ns::kApply>(L, gs, n, from, stream)
                                 : launch_product<Ns::kOut>(L, gs, n, from, stream);
            }
            if (e != cudaSuccess) return e;
        }
    }
    return cudaSuccess;
}

bool ns_coefficients_fit(const float coeffs[3], int32_t steps) {
    const double a = coeffs[0], b = coeffs[1], c = coeffs[2];
    if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return false;
    double top = 1.0 + 1e-2;                     // the largest singular value, with rounding
    for (int32_t i = 0; i < steps; ++i) {
        // |p| and |b s + c s^2| over x in [0, top], s = x^2: at the ends and
        // where their derivatives vanish
        const double s_top = top * top;
        auto poly = [&](double s) { return std::fabs(std::sqrt(s) * (a + s * (b + s * c))); };
        auto inner = [&](double s) { return std::fabs(s * (b + s * c)); };
        double p = poly(s_top), q = inner(s_top);
        if (c != 0.0) {
            const double v = -b / (2.0 * c);
            if (v > 0.0 && v < s_top) q = std::max(q, inner(v));
            const double disc = 9.0 * b * b - 20.0 * a * c;
            if (disc >= 0.0)
                for (double sign : {-1.0, 1.0}) {
                    const double r = (-3.0 * b + sign * std::sqrt(disc)) / (10.0 * c);
                    if (r > 0.0 && r < s_top) p = std::max(p, poly(r));
                }
        } else if (b != 0.0) {
            const double r = -a / (3.0 * b);
            if (r > 0.0 && r < s_top) p = std::max(p, poly(r));
        }
        // A, B and X in fp16's range (65504 over their scales), halved for rounding
        if (s_top * kNsScaleA > 32000.0 || q * kNsScaleB > 32000.0 || p * kNsScaleX > 32000.0) return false;
        top = p * (1.0 + 1e-2);
    }
    return true;
}

}  // namespace zr
