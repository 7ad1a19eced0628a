// Newton-Schulz orthogonalisation of small matrices: a whole iteration per
// cluster, nothing in global memory between the source and the result.
//
// For a smaller extent of at most 128, A and B are one 128 x 128 tile, and
// what a product costs in the persistent kernel is the way from one product
// to the next through global memory (5 us), not its arithmetic (0.5 us).  Here
// a cluster of C CTAs holds one matrix: Z = X for wide ones, X^T for tall
// ones, each CTA up to 256 of Z's columns, X in fp32 registers and as the fp16
// operand in shared memory.  A step is
//   A    = sum over the cluster of Z_c Z_c^T  (tcgen05; fp32 partial sums are
//          exchanged through distributed shared memory, each CTA adding up
//          128 / C rows in the order of the CTAs),
//   B    = b A + c A A                        (each CTA for itself),
//   Z_c <- (a + D) Z_c + R Z_c                (local).
// Five steps (graph replays) of 128 x 128: 81 us in the persistent kernel, 27
// here; 100 x 2000: 104 and 51; 24 of 128 x 4096: 392 and 244; 150 of 128 x
// 128: 153 and 51.  So it is taken wherever it fits.  It ends where the layout
// does (one tile of A, 16 CTAs of 256 columns), not where the persistent
// kernel catches up, which takes two to five times as long just past it: 129 x
// 129 77 us, 128 x 4097 133 (128 x 4096 here: 64), 24 of 128 x 4097 405 (244),
// 150 of 129 x 129 249 (51).  A step of 128 x 256 is 7.4 k cycles:
// 3.5 k of products with the way into and out of tensor memory, the rest is
// the epilogues' arithmetic; with C > 1 the exchange adds 5 to 8 k, bound by
// the distributed shared memory.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>

#include "zr.h"
#include "zr_newton.hpp"
#include "zr_newton_ptx.cuh"

namespace zr {
namespace {

constexpr int kDim = 128;                       // A, B: 128 x 128
constexpr int kWide = 256;                      // columns of Z on a CTA
constexpr int kMostCtas = 16;
constexpr int kSmallThreads = 256;              // warp w: rows 32 (w % 4) on, the left or right half of the columns
constexpr int kChunkBytes = kDim * 128;         // 64 columns of 128 rows
constexpr int kOffA = kWide / 64 * kChunkBytes, kOffB = kOffA + 2 * kChunkBytes, kOffEx = kOffB + 2 * kChunkBytes;
constexpr int kExBytes = kDim * kDim * 4;       // partial sums of A; 128 columns of Z in fp32
constexpr int kOffDiagA = kOffEx + kExBytes, kOffDiagB = kOffDiagA + kDim * 4;
constexpr int kOffSums = kOffDiagB + kDim * 4, kOffWords = kOffSums + 8 * 8 + 8;
constexpr int kSmallSmem = kOffWords + 32;
constexpr int kSmallGroups = 16;

struct SmallGroup {
    const void* src;
    int32_t dtype, tall, g, l, width;           // width: columns of Z on a CTA, a multiple of 64
    int32_t vec_in, vec_out;                    // four elements of a row move as one word
    int64_t src_row, src_batch;
    int32_t first, n;                           // the group's first cluster; columns of X
    uint16_t* out;
    int64_t out_row, out_batch;
    const int64_t *master_offsets, *param_offsets;
    float step_size;
};

struct SmallLaunch {
    int32_t n_groups, steps, ctas;
    Affine k[4];                                // A, B, update, last update
    double eps;
    float decay;
    uint32_t* gave_up;
    int32_t clear;                              // *gave_up first
    float* master;
    uint16_t* param_out;
    uint16_t* const* targets;
    int32_t n_targets;
    SmallGroup g[kSmallGroups];
};

__device__ __forceinline__ void mma_one(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_commit_one(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ uint32_t cluster_address(uint32_t addr, uint32_t cta) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(cta));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 ld_cluster16(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ double ld_cluster_f64(uint32_t addr) {
    double v;
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_cluster8(uint32_t addr, uint32_t x, uint32_t y) {
    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float x) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(x) : "memory");
}
// N elements, number k at src[at(k)] if ok(k), else zero.  All loads are issued before the first is used.
template <int N, typename At, typename Ok>
__device__ __forceinline__ void load_source(const void* src, int32_t dtype, float (&v)[N], At at, Ok ok) {
    if (dtype == ZR_DTYPE_F32) {
        const float* p = static_cast<const float*>(src);
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = ok(k) ? p[at(k)] : 0.0f;
        return;
    }
    const uint16_t* p = static_cast<const uint16_t*>(src);
    uint16_t u[N];
#pragma unroll
    for (int k = 0; k < N; ++k) u[k] = ok(k) ? p[at(k)] : static_cast<uint16_t>(0);
#pragma unroll
    for (int k = 0; k < N; ++k)
        v[k] = dtype == ZR_DTYPE_BF16 ? __uint_as_float(static_cast<uint32_t>(u[k]) << 16) : half_value(u[k]);
}
// 16-byte piece j of row r of the fp32 exchange buffer (512 bytes a row).
__device__ __forceinline__ uint32_t ex_piece(uint32_t ex, int r, int j) { return ex + r * 512 + ((j ^ (r & 7)) << 4); }

// fp32 accumulators, fp16 operands, op2's major, N / 8, M / 16
__device__ __forceinline__ uint32_t small_idesc(uint32_t mn2, int n) {
    return (1u << 4) | (mn2 << 16) | (static_cast<uint32_t>(n >> 3) << 17) | ((kDim >> 4) << 24);
}

// Every C-th row of A from the cluster's partial sums, added in the order of
// the CTAs, into every CTA's operand and diagonal.  A thread has 16 / C
// pieces of four columns, so 16 loads in flight for any C.  Bound by the
// distributed shared memory (some 18 bytes per clock): rows and columns past
// `dim` stay as they are, zero.
template <int C>
__device__ __forceinline__ void exchange(uint32_t smem, int rank, int tid, int dim, float alpha) {
    constexpr int kPieces = 16 / C;
    uint32_t at[C];
#pragma unroll
    for (int c = 0; c < C; ++c) at[c] = cluster_address(smem, c);
    const int j = tid & 31;
    auto row_of = [&](int e) { return ((tid >> 5) + 8 * e) * C + rank; };
    if (4 * j >= dim) return;
    float4 p[kPieces][C];
#pragma unroll
    for (int e = 0; e < kPieces; ++e)
#pragma unroll
        for (int c = 0; c < C; ++c) p[e][c] = ld_cluster16(at[c] + ex_piece(kOffEx, min(row_of(e), dim - 1), j));
#pragma unroll
    for (int e = 0; e < kPieces; ++e) {
        const int r = row_of(e);
        if (r >= dim) continue;
        float4 s = p[e][0];
#pragma unroll
        for (int c = 1; c < C; ++c) {
            s.x += p[e][c].x; s.y += p[e][c].y; s.z += p[e][c].z; s.w += p[e][c].w;
        }
        float v[4] = {s.x * alpha, s.y * alpha, s.z * alpha, s.w * alpha};
        float on = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (4 * j + i == r) {
                on = v[i] * (1.0f / kNsScaleA);
                v[i] = 0.0f;
            }
        const uint32_t to = staged(kOffA + (j >> 4) * kChunkBytes, r, (j & 15) >> 1) + 8 * (j & 1);
        const uint32_t w0 = half2_bits(v[0], v[1]), w1 = half2_bits(v[2], v[3]);
#pragma unroll
        for (int c = 0; c < C; ++c) st_cluster8(at[c] + to, w0, w1);
        if ((r >> 2) == j) {
#pragma unroll
            for (int c = 0; c < C; ++c) st_cluster_f32(at[c] + kOffDiagA + 4 * r, on);
        }
    }
}

template <bool APPLY>
__global__ void __launch_bounds__(kSmallThreads, 1) zr_ns_small_kernel(const __grid_constant__ SmallLaunch L) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];       // the swizzle's period
    volatile double* s_sums = reinterpret_cast<volatile double*>(smem_raw + kOffSums);      // 8 warps', then the CTA's
    uint32_t* words = reinterpret_cast<uint32_t*>(smem_raw + kOffWords + 8);
    uint32_t& s_tmem = words[0];
    const uint32_t smem = smem_u32(smem_raw);
    const uint32_t xs = smem, as = smem + kOffA, bs = smem + kOffB, ex = smem + kOffEx;
    const uint32_t diag_a = smem + kOffDiagA, diag_b = smem + kOffDiagB, bar = smem + kOffWords;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int quad = warp & 3, half = warp >> 2, row = quad * 32 + lane;
    const int32_t C = L.ctas, rank = static_cast<int32_t>(blockIdx.x) % C, matrix = static_cast<int32_t>(blockIdx.x) / C;
    const Bail bail{words + 1, words + 2, L.gave_up};

    if (tid == 0) {
        words[1] = words[2] = 0u;
        mbar_init(bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = s_tmem;
    const uint32_t tm_z = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * 128, tm_a = tm_z + kWide - half * 64;

    int32_t gi = 0;
    while (gi + 1 < L.n_groups && matrix >= L.g[gi + 1].first) ++gi;
    const SmallGroup& g = L.g[gi];
    const int64_t slot = matrix - g.first;
    const int32_t width = g.width, col0 = rank * width;         // this CTA's columns of Z
    const int32_t mine = min(max(width - half * 128, 0), 128);  // of them, in this warp's half (a multiple of 64)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // (a wait gives up 20 s after its block began: never before block 0 is here)
    if (blockIdx.x == 0 && tid == 0 && L.clear) *L.gave_up = 0u;

    // Z, a row's 128 columns per thread: x[i] holds columns 2 i and 2 i + 1.
    f32x2 x[64];
    const int64_t src0 = slot * g.src_batch;
    if (g.tall) {
        // Z's rows run along the source's rows: lanes read side by side
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float v[64];
            const int32_t c0 = col0 + half * 128 + 64 * q;
            const int64_t e0 = src0 + static_cast<int64_t>(c0) * g.src_row + row;
            const int32_t count = 64 * q < mine && row < g.g ? g.l - c0 : 0;
            load_source(g.src, g.dtype, v, [&](int k) { return e0 + k * g.src_row; }, [&](int k) { return k < count; });
#pragma unroll
            for (int i = 0; i < 32; ++i) x[32 * q + i] = pack2(v[2 * i], v[2 * i + 1]);
        }
    } else {
#pragma unroll 1
        for (int pass = 0; pass * 128 < width; ++pass) {
            // warp w reads rows w, w + 8, ..: 32 lanes along a row
            if (g.vec_in) {
                const int32_t c0 = col0 + pass * 128 + 4 * lane;
                const int64_t e0 = src0 + warp * g.src_row + c0;
                uint4 q[16];
                if (g.dtype == ZR_DTYPE_F32) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        q[i] = warp + 8 * i < g.g && c0 < g.l
                                   ? *reinterpret_cast<const uint4*>(static_cast<const float*>(g.src) + e0 + 8 * i * g.src_row)
                                   : make_uint4(0, 0, 0, 0);
                } else {
                    uint2 u[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        u[i] = warp + 8 * i < g.g && c0 < g.l
                                   ? *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(g.src) + e0 + 8 * i * g.src_row)
                                   : make_uint2(0, 0);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        if (g.dtype == ZR_DTYPE_BF16) {
                            q[i] = make_uint4(u[i].x << 16, u[i].x & 0xFFFF0000u, u[i].y << 16, u[i].y & 0xFFFF0000u);
                        } else {
                            const float2 f = half2_values(u[i].x), h = half2_values(u[i].y);
                            q[i] = make_uint4(__float_as_uint(f.x), __float_as_uint(f.y), __float_as_uint(h.x), __float_as_uint(h.y));
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) st_shared16(ex_piece(ex, warp + 8 * i, lane), q[i]);
            } else {
                const int32_t c0 = col0 + pass * 128 + lane;
                const int64_t e0 = src0 + warp * g.src_row + c0;
                float v[64];
                load_source(
                    g.src, g.dtype, v, [&](int k) { return e0 + 8 * (k >> 2) * g.src_row + 32 * (k & 3); },
                    [&](int k) { return warp + 8 * (k >> 2) < g.g && c0 + 32 * (k & 3) < g.l; });
#pragma unroll
                for (int k = 0; k < 64; ++k) {
                    const int cl = 32 * (k & 3) + lane;
                    st_shared_f32(ex_piece(ex, warp + 8 * (k >> 2), cl >> 2) + 4 * (cl & 3), v[k]);
                }
            }
            __syncthreads();
            if (half == pass) {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const uint4 q = ld_shared16(ex_piece(ex, row, i));
                    x[2 * i] = pack2(__uint_as_float(q.x), __uint_as_float(q.y));
                    x[2 * i + 1] = pack2(__uint_as_float(q.z), __uint_as_float(q.w));
                }
            }
            __syncthreads();
        }
        if (mine == 0) {
#pragma unroll
            for (int i = 0; i < 64; ++i) x[i] = 0;
        }
        // (columns of a pass past the width belong to the next CTA)
        if (mine == 64) {
#pragma unroll
            for (int i = 32; i < 64; ++i) x[i] = 0;
        }
    }

    // The norm: squares are exact in fp64, the order of the sum is fixed.
    double part[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int i = 0; i < 64; ++i) {
        const float2 f = unpack2(x[i]);
        part[2 * (i & 1)] = fma(static_cast<double>(f.x), static_cast<double>(f.x), part[2 * (i & 1)]);
        part[2 * (i & 1) + 1] = fma(static_cast<double>(f.y), static_cast<double>(f.y), part[2 * (i & 1) + 1]);
    }
    double sum = (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) sum += __shfl_down_sync(0xFFFFFFFFu, sum, d);
    if (lane == 0) s_sums[warp] = sum;
    __syncthreads();
    sum = 0.0;
    for (int w = 0; w < kSmallThreads / 32; ++w) sum += s_sums[w];
    if (C > 1) {
        if (tid == 0) s_sums[8] = sum;
        cluster_sync();
        sum = 0.0;
        for (int32_t c = 0; c < C; ++c) sum += ld_cluster_f64(cluster_address(smem + kOffSums + 64, c));
    }
    const float2 scale = ns_scale_of(sum, L.eps);
#pragma unroll
    for (int i = 0; i < 64; ++i) x[i] = mul2(mul2(x[i], pack2(scale.x, scale.x)), pack2(scale.y, scale.y));

    auto write_operand = [&] {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (8 * i >= mine) break;
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = unpack2(x[4 * i + j]);
                w[j] = half2_bits(f.x, f.y);
            }
            st_shared16(staged(xs + (2 * half + (i >> 3)) * kChunkBytes, row, i & 7), make_uint4(w[0], w[1], w[2], w[3]));
        }
    };
    // What every thread wrote, before the products that one of them issues;
    // and the products, before what every thread reads.  A block whose wait
    // runs out goes on without its products (the cluster's barriers still
    // match), and the caller's word says so.
    uint32_t phase = 0;
    auto products = [&](auto issue) {
        fence_async_shared();
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncthreads();
        if (warp == 0 && elect_one()) {
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            issue();
            mma_commit_one(bar);
        }
        __syncwarp();
        (void)mbar_wait(bar, phase & 1, bail);
        ++phase;
        __syncwarp();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    };
    // 64 columns of a row of A or B: fp16 without the diagonal into `part`
    auto keep_half = [&](f32x2(&v)[16], int first, uint32_t part, float& on) {
        if (half * 64 + first == quad * 32) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float2 f = unpack2(v[i]);
                on = 2 * i == lane ? f.x : 2 * i + 1 == lane ? f.y : on;
                v[i] = pack2(2 * i == lane ? 0.0f : f.x, 2 * i + 1 == lane ? 0.0f : f.y);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = unpack2(v[4 * i + j]);
                w[j] = half2_bits(f.x, f.y);
            }
            st_shared16(staged(part, row, (first >> 3) + i), make_uint4(w[0], w[1], w[2], w[3]));
        }
    };
    const bool on_diagonal = half == (quad >> 1);    // this warp's 64 columns of A hold its rows' diagonal

    if (C > 1) {
        for (int i = tid; i < 2 * kChunkBytes / 16; i += kSmallThreads) st_shared16(as + 16 * i, make_uint4(0, 0, 0, 0));
        if (tid < kDim) st_shared_f32(diag_a + 4 * tid, 0.0f);
    }
    write_operand();
#pragma unroll 1
    for (int32_t step = 0; step < L.steps; ++step) {
        products([&] {
            for (int kk = 0; kk < width / 16; ++kk) {
                const uint64_t d = smem_desc(xs + (kk >> 2) * kChunkBytes + (kk & 3) * 32, false, 0);
                mma_one(tmem + kWide, d, d, small_idesc(0, kDim), kk != 0);
            }
        });
        {
            const Affine k = L.k[0];
            const f32x2 alpha = pack2(k.alpha, k.alpha);
            if (C == 1) {
                float on = 0.0f;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    f32x2 v[16];
                    tmem_ld32(tm_a + 32 * h, v);
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = mul2(v[i], alpha);
                    keep_half(v, 32 * h, as + half * kChunkBytes, on);
                }
                if (on_diagonal) st_shared_f32(diag_a + 4 * row, on * (1.0f / kNsScaleA));
                __syncthreads();
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    f32x2 v[16];
                    tmem_ld32(tm_a + 32 * h, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 p = unpack2(v[2 * i]), q = unpack2(v[2 * i + 1]);
                        st_shared16(ex_piece(ex, row, half * 16 + h * 8 + i),
                                    make_uint4(__float_as_uint(p.x), __float_as_uint(p.y), __float_as_uint(q.x), __float_as_uint(q.y)));
                    }
                }
                cluster_sync();
                if (C == 2) exchange<2>(smem, rank, tid, g.g, k.alpha);
                else if (C == 4) exchange<4>(smem, rank, tid, g.g, k.alpha);
                else if (C == 8) exchange<8>(smem, rank, tid, g.g, k.alpha);
                else exchange<16>(smem, rank, tid, g.g, k.alpha);
                cluster_sync();
            }
        }
        products([&] {
#pragma unroll
            for (int kk = 0; kk < kDim / 16; ++kk) {
                const uint64_t d = smem_desc(as + (kk >> 2) * kChunkBytes + (kk & 3) * 32, false, 0);
                mma_one(tmem + kWide, d, d, small_idesc(0, kDim), kk != 0);
            }
        });
        {
            // c A A + b A, A = D + R: acc = R R
            const Affine k = L.k[1];
            const float s = k.gamma * (1.0f / kNsScaleA);
            const float dr = ld_shared_f32(diag_a + 4 * row), base = fmaf(dr, s, k.beta);
            float on = 0.0f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f32x2 v[16], y[16];
                ld_staged32(as + half * kChunkBytes, row, 4 * h, y);
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    f32x2 d[2];
                    ld_shared_f32x4(diag_a + 256 * half + 128 * h + 8 * i, d);
#pragma unroll
                    for (int j = 0; j < 2; ++j) y[i + j] = mul2(y[i + j], fma2(d[j], pack2(s, s), pack2(base, base)));
                }
                if (half * 64 + 32 * h == quad * 32) {
                    const float o = fmaf(dr, k.gamma, k.beta * kNsScaleA) * dr;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 f = unpack2(y[i]);
                        y[i] = pack2(2 * i == lane ? o : f.x, 2 * i + 1 == lane ? o : f.y);
                    }
                }
                tmem_ld32(tm_a + 32 * h, v);
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = fma2(v[i], pack2(k.alpha, k.alpha), y[i]);
                keep_half(v, 32 * h, bs + half * kChunkBytes, on);
            }
            if (on_diagonal) st_shared_f32(diag_b + 4 * row, on * (1.0f / kNsScaleB));
        }
        products([&] {
#pragma unroll
            for (int kk = 0; kk < kDim / 16; ++kk)
                mma_one(tmem, smem_desc(bs + (kk >> 2) * kChunkBytes + (kk & 3) * 32, false, 0),
                        smem_desc(xs + kk * 16 * 128, true, kChunkBytes), small_idesc(1, width), kk != 0);
        });
        {
            const bool last = step + 1 == L.steps;
            const Affine k = L.k[last ? 3 : 2];
            const float d = fmaf(ld_shared_f32(diag_b + 4 * row), k.gamma, k.beta);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (32 * q >= mine) break;
                f32x2 v[16];
                tmem_ld32(tm_z + 32 * q, v);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    x[16 * q + i] = fma2(v[i], pack2(k.alpha, k.alpha), mul2(x[16 * q + i], pack2(d, d)));
            }
            if (!last) write_operand();
        }
    }

    // The result: element (r, c) of Z is (r, c) of X, or (c, r) for tall ones.
    // N values for the elements first + at(k) of the destination.
    const int64_t pitch = APPLY ? g.n : g.out_row;
    auto store = [&](auto& v, int64_t first, auto at, auto ok) {
        constexpr int N = sizeof(v) / sizeof(float);
        if constexpr (APPLY) {
            float* pm = L.master + g.master_offsets[slot] + first;
            const int64_t po = g.param_offsets[slot] + first;
            float p[N];
#pragma unroll
            for (int k = 0; k < N; ++k)
                if (ok(k)) p[k] = pm[at(k)];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                if (!ok(k)) continue;
                const float q = __fsub_rn(__fmul_rn(p[k], L.decay), __fmul_rn(v[k], g.step_size));
                pm[at(k)] = q;
                const uint16_t u = bf16_bits(q);
                if (L.n_targets == 0) L.param_out[po + at(k)] = u;
                else
                    for (int t = 0; t < L.n_targets; ++t) L.targets[t][po + at(k)] = u;
            }
        } else {
            uint16_t* out = g.out + slot * g.out_batch + first;
#pragma unroll
            for (int k = 0; k < N; ++k)
                if (ok(k)) out[at(k)] = bf16_bits(v[k]);
        }
    };
    if (g.tall) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int32_t c0 = col0 + half * 128 + 32 * q;
            const int32_t count = 32 * q < mine && row < g.g ? g.l - c0 : 0;
            float v[32];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float2 f = unpack2(x[16 * q + i]);
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
            store(v, c0 * pitch + row, [&](int k) { return k * pitch; }, [&](int k) { return k < count; });
        }
    } else {
#pragma unroll 1
        for (int pass = 0; pass * 128 < width; ++pass) {
            __syncthreads();
            if (half == pass) {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float2 p = unpack2(x[2 * i]), q = unpack2(x[2 * i + 1]);
                    st_shared16(ex_piece(ex, row, i),
                                make_uint4(__float_as_uint(p.x), __float_as_uint(p.y), __float_as_uint(q.x), __float_as_uint(q.y)));
                }
            }
            __syncthreads();
            // 32 lanes along a row; columns past the width are the next CTA's
            const int32_t cols = min(min(width - pass * 128, 128), g.l - (col0 + pass * 128));
            if (!APPLY && g.vec_out) {
                uint16_t* out = g.out + slot * g.out_batch + warp * g.out_row + col0 + pass * 128 + 4 * lane;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    if (warp + 8 * i >= g.g || 4 * lane >= cols) continue;
                    const uint4 q = ld_shared16(ex_piece(ex, warp + 8 * i, lane));
                    const uint32_t w0 = bf16_bits(__uint_as_float(q.x)) | (static_cast<uint32_t>(bf16_bits(__uint_as_float(q.y))) << 16);
                    const uint32_t w1 = bf16_bits(__uint_as_float(q.z)) | (static_cast<uint32_t>(bf16_bits(__uint_as_float(q.w))) << 16);
                    *reinterpret_cast<uint2*>(out + 8 * i * g.out_row) = make_uint2(w0, w1);
                }
                continue;
            }
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
                const int r0 = warp + 64 * i;
                float v[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const int cl = 32 * (k & 3) + lane;
                    v[k] = ld_shared_f32(ex_piece(ex, r0 + 8 * (k >> 2), cl >> 2) + 4 * (cl & 3));
                }
                store(v, r0 * pitch + col0 + pass * 128 + lane, [&](int k) { return 8 * (k >> 2) * pitch + 32 * (k & 3); },
                      [&](int k) { return r0 + 8 * (k >> 2) < g.g && 32 * (k & 3) + lane < cols; });
            }
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncwarp();
    __syncthreads();
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// The cluster's size for a larger extent; 0 if none holds it.
int cluster_ctas(int64_t l) {
    for (int c = 1; c <= kMostCtas; c *= 2)
        if (l <= static_cast<int64_t>(c) * kWide) return c;
    return 0;
}

// Whether clusters of `ctas` can run on the current device (and the kernel's
// shared memory is allowed there).
template <bool APPLY>
bool clusters_run(int ctas) {
    static std::atomic<int> known[64][kMostCtas + 1];        // 1 yes, 2 no
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    const int k = known[dev][ctas].load(std::memory_order_acquire);
    if (k != 0) return k == 1;
    auto kernel = zr_ns_small_kernel<APPLY>;
    int n = 0;
    bool ok = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmallSmem) == cudaSuccess &&
              cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
    if (ok) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(ctas);
        cfg.blockDim = dim3(kSmallThreads);
        cfg.dynamicSmemBytes = kSmallSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {static_cast<unsigned>(ctas), 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        ok = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n >= 1;
        if (!ok) (void)cudaGetLastError();
    }
    known[dev][ctas].store(ok ? 1 : 2, std::memory_order_release);
    return ok;
}

template <bool APPLY>
int launch_small(const NsGroup* groups, int32_t n, int ctas, int32_t steps, const float coeffs[3], double eps,
                 const NsApply& apply, uint32_t* gave_up, bool clear, void* stream) {
    SmallLaunch L{};
    L.n_groups = n;
    L.steps = steps;
    L.ctas = ctas;
    ns_factors(L.k, coeffs);
    L.eps = eps;
    L.decay = apply.decay;
    L.gave_up = gave_up;
    L.clear = clear;
    L.master = apply.master;
    L.param_out = apply.param_out;
    L.targets = apply.targets;
    L.n_targets = apply.n_targets;
    int64_t matrices = 0;
    for (int32_t i = 0; i < n; ++i) {
        const NsGroup& s = groups[i];
        SmallGroup& g = L.g[i];
        g.src = s.src;
        g.dtype = s.src_dtype;
        g.tall = s.m > s.n;
        g.g = static_cast<int32_t>(s.gram_dim());
        g.l = static_cast<int32_t>(std::max(s.m, s.n));
        g.width = static_cast<int32_t>((g.l + 64 * ctas - 1) / (64 * ctas) * 64);
        g.src_row = s.src_row;
        g.src_batch = s.src_batch;
        auto aligned = [&](const void* p, uint64_t bytes, int64_t row, int64_t batch) {
            return s.n % 4 == 0 && reinterpret_cast<uintptr_t>(p) % bytes == 0 && row % 4 == 0 && batch % 4 == 0;
        };
        g.vec_in = aligned(s.src, s.src_dtype == ZR_DTYPE_F32 ? 16 : 8, s.src_row, s.src_batch);
        g.vec_out = s.out != nullptr && aligned(s.out, 8, s.out_row, s.out_batch);
        g.first = static_cast<int32_t>(matrices);
        g.n = static_cast<int32_t>(s.n);
        g.out = s.out;
        g.out_row = s.out_row;
        g.out_batch = s.out_batch;
        g.master_offsets = s.master_offsets;
        g.param_offsets = s.param_offsets;
        g.step_size = s.step_size;
        matrices += s.batch;
    }
    if (matrices * ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(matrices * ctas));
    cfg.blockDim = dim3(kSmallThreads);
    cfg.dynamicSmemBytes = kSmallSmem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {static_cast<unsigned>(ctas), 1, 1};
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, zr_ns_small_kernel<APPLY>, L);
}

}  // namespace

bool ns_small(const NsGroup* groups, int32_t n_groups, bool apply) {
    int most = 0;
    for (int32_t i = 0; i < n_groups; ++i) {
        const int c = cluster_ctas(std::max(groups[i].m, groups[i].n));
        if (groups[i].gram_dim() > kDim || c == 0) return false;
        most = std::max(most, c);
    }
    return most > 0 && (apply ? clusters_run<true>(most) : clusters_run<false>(most));
}

int launch_ns_small(const NsGroup* groups, int32_t n_groups, int32_t steps, const float coeffs[3], double eps,
                    const NsApply& apply, uint32_t* gave_up, bool clear, void* stream) {
    for (int32_t at = 0; at < n_groups; at += kSmallGroups) {
        const int32_t n = std::min(kSmallGroups, n_groups - at);
        int most = 1;
        for (int32_t i = 0; i < n; ++i) most = std::max(most, cluster_ctas(std::max(groups[at + i].m, groups[at + i].n)));
        const int e = apply.master ? launch_small<true>(groups + at, n, most, steps, coeffs, eps, apply, gave_up, clear, stream)
                                   : launch_small<false>(groups + at, n, most, steps, coeffs, eps, apply, gave_up, clear, stream);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace zr
