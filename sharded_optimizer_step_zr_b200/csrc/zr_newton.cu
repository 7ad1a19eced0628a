// Newton-Schulz orthogonalisation for B200 (sm_100a): tcgen05 products of
// TMA-fed fp16 tiles.
//
//   X_0 = U / (||U||_F + eps);   A = X X^T,  B = b A + c A A,  X <- a X + B X
//
// (m <= n; for m > n the same polynomial acts from the right, on X^T X, so no
// operand is ever transposed in memory).  A pass over the m x n matrix costs
// g^2 l multiply-adds for A, g^3 for A A (g = min, l = max) and g^2 l for
// B X; A and A A are symmetric and only the tiles that touch the lower
// triangle are computed, each stored twice.  Large matrices are bound by the
// tensor cores (and they by the power limit), small ones by the way from one
// product to the next: one persistent kernel runs all of them.  Matrices with
// a smaller extent of at most 128 have a kernel of their own
// (zr_newton_small.cu).
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
// After five steps the result of a random or gradient-like matrix is 1e-4 to
// 1.2e-3 of its norm off the exact iteration (7e-4 at 512 x 512, where bf16
// operands give 1e-2 and fp16 ones alone 1.2e-3); 3e-4 to 3e-3 when 16
// directions are 400 times stronger than the rest (fp16 alone: 2e-2).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "zr.h"
#include "zr_newton.hpp"
#include "zr_newton_ptx.cuh"

namespace zr {
namespace {

// ---------------------------------------------------------------------------
// the iteration kernel: shapes
// ---------------------------------------------------------------------------

constexpr int kBM = 256;                                   // rows of a tile: 128 on each CTA of a pair
constexpr int kBN = 256;                                   // columns, or half as many for launches of few tiles
constexpr int kBK = 64;
constexpr int kStages = 5;
constexpr int kBoxBytes = 64 * 64 * 2;                     // one operand box: 64 rows of 128 bytes
constexpr int kOpBytes = 2 * kBoxBytes;                    // a CTA's 128 rows of op1, or its half (128 or 64) of op2's
constexpr int kStageBytes = 2 * kOpBytes;
constexpr int kEpiWarps = 8;                               // two for each 32 rows, taking turns at 64 columns
constexpr int kPartBytes = 32 * 128;                       // a warp's 32 rows of 64 fp16 columns
constexpr int kBufBytes = 2 * kPartBytes;                  // X and its rounding error; or a result and its mirror image; or 32 x 64 fp32
constexpr int kDiagBytes = 64 * 4;                         // a warp's 64 columns of a diagonal
constexpr int kIterThreads = 64 + 32 * kEpiWarps;          // producer, issuer, epilogue warps
constexpr int kSmemStaging = kStages * kStageBytes, kSmemDiag = kSmemStaging + kEpiWarps * kBufBytes;
constexpr int kSmemBars = kSmemDiag + kEpiWarps * kDiagBytes;
constexpr int kBars = 2 * kStages + 4 + kEpiWarps;
constexpr int kIterSmem = kSmemBars + 8 * kBars + 16;
static_assert(kIterSmem <= 227 * 1024, "one CTA per SM");
constexpr int kMaxGroups = 16;                             // of a launch

enum : int { kGram = 0, kPoly = 1, kUpdate = 2 };          // products of a step, in order

// A group's tensor maps: the products' operands (pairs are for either X), and
// the epilogue's, as in NsMaps.
struct IterMaps {
    CUtensorMap gram1[2], gram2[2], poly1, poly2, update1[2], update2[2];
    CUtensorMap ex[2], egram, epoly, mgram, mpoly;
};
static_assert(sizeof(CUtensorMap) == 128 && sizeof(IterMaps) % sizeof(CUtensorMap) == 0, "maps and nothing else");

struct IterGroup {
    int32_t m, n, dim, tall;
    int32_t sym_tiles, out_tiles, out_tiles_n;             // tiles of a matrix: A and A A; the update
    int64_t first_sym, first_out;                          // the group's first tile of a product
    uint32_t* done;                                        // per matrix: finished warps' shares of tiles
    float *gram_diag, *poly_diag;
    uint16_t* out;                                         // the last update's result in bf16
    int64_t out_row, out_batch;
    int32_t out_vec;                                       // its rows and matrices start 16-byte aligned
    const int64_t *master_offsets, *param_offsets;
    float step_size;
};

// Parameters past 4 KB cost a launch 70 us on the host, so only a single
// group's maps are among them; those of several are in device memory, where
// another plan's maps may have stood before: each block fences all of them
// before its first copy.
struct InlineMaps {
    IterMaps one;
    __device__ __forceinline__ void fence(int32_t) const {}
    __device__ __forceinline__ const IterMaps& of(int32_t) const { return one; }
};
struct DeviceMaps {
    const IterMaps* all;
    __device__ __forceinline__ void fence(int32_t n_groups) const {
        constexpr int kMapsOfGroup = sizeof(IterMaps) / sizeof(CUtensorMap);
        const CUtensorMap* maps = reinterpret_cast<const CUtensorMap*>(all);
        for (int i = threadIdx.x; i < n_groups * kMapsOfGroup; i += kIterThreads) fence_tensor_map(maps + i);
    }
    __device__ __forceinline__ const IterMaps& of(int32_t group) const { return all[group]; }
};
template <int NG>
struct IterLaunch {
    std::conditional_t<NG == 1, InlineMaps, DeviceMaps> maps;
    IterGroup g[NG];
    int32_t n_groups, steps, pairs;
    int32_t sym_bn, out_bn;
    int64_t sym_total, out_total;                          // tiles of all matrices
    Affine k[4];                                           // A, B, update, last update
    float decay;
    uint32_t *abort_word, *gave_up;
    float* master;
    uint16_t* param_out;
    uint16_t* const* targets;
    int32_t n_targets;
};
static_assert(sizeof(IterLaunch<1>) <= 4096 && sizeof(IterLaunch<kMaxGroups>) <= 4096, "a launch's fast parameters");


// ---------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------

// One role's walk over the launch's tiles: product by product, in each the
// matrices in order, every `pairs`-th tile.
struct TileAt {
    int32_t step = 0, op = 0, group = 0, slot = 0, row0 = 0, col0 = 0, bn = 0;
};

template <int NG>
struct TileWalk {
    const IterLaunch<NG>& L;
    int64_t r;
    int32_t step = 0;
    __device__ __forceinline__ TileWalk(const IterLaunch<NG>& l, int32_t pair) : L(l), r(pair) { wrap(); }
    __device__ __forceinline__ void wrap() {
        const int64_t per_step = 2 * L.sym_total + L.out_total;
        while (r >= per_step) {
            r -= per_step;
            ++step;
        }
    }
    __device__ __forceinline__ bool live() const { return step < L.steps; }
    __device__ __forceinline__ void next() {
        r += L.pairs;
        wrap();
    }
    __device__ __forceinline__ TileAt at() const {
        TileAt a;
        a.step = step;
        a.op = r < L.sym_total ? kGram : r < 2 * L.sym_total ? kPoly : kUpdate;
        const int64_t t0 = r - a.op * L.sym_total;
        int32_t gi = 0;
        if (a.op == kUpdate) {
            while (gi + 1 < L.n_groups && t0 >= L.g[gi + 1].first_out) ++gi;
            const IterGroup& g = L.g[gi];
            const int64_t t = t0 - g.first_out;
            a.slot = static_cast<int32_t>(t / g.out_tiles);
            const int32_t q = static_cast<int32_t>(t - static_cast<int64_t>(a.slot) * g.out_tiles);
            a.bn = L.out_bn;
            a.row0 = (q / g.out_tiles_n) * kBM;
            a.col0 = (q % g.out_tiles_n) * a.bn;
        } else {
            // Row block i of 256 has the column tiles up to its diagonal
            // block: i + 1 of 256 columns, or 2 (i + 1) of 128.
            while (gi + 1 < L.n_groups && t0 >= L.g[gi + 1].first_sym) ++gi;
            const IterGroup& g = L.g[gi];
            const int64_t t = t0 - g.first_sym;
            a.slot = static_cast<int32_t>(t / g.sym_tiles);
            const int32_t q = static_cast<int32_t>(t - static_cast<int64_t>(a.slot) * g.sym_tiles);
            a.bn = L.sym_bn;
            const int32_t twice = a.bn == kBN ? 2 * q : q;      // i (i + 1) <= twice
            int32_t i = static_cast<int32_t>((sqrtf(4.0f * static_cast<float>(twice) + 1.0f) - 1.0f) * 0.5f);
            while (static_cast<int64_t>(i + 1) * (i + 2) <= twice) ++i;
            while (static_cast<int64_t>(i) * (i + 1) > twice) --i;
            a.row0 = i * kBM;
            a.col0 = (q - (a.bn == kBN ? i * (i + 1) / 2 : i * (i + 1))) * a.bn;
        }
        a.group = gi;
        return a;
    }
};

// What the matrix's counter shows once everything that a tile reads is written.
__device__ __forceinline__ uint32_t shares_before(const IterGroup& g, const TileAt& at) {
    const uint32_t tiles = static_cast<uint32_t>(at.step) * (2 * g.sym_tiles + g.out_tiles) + at.op * g.sym_tiles;
    return tiles * (2 * kEpiWarps);
}

// ---------------------------------------------------------------------------
// the iteration kernel
// ---------------------------------------------------------------------------

// All products of all steps in one launch: 15 for five steps.  A pair of CTAs
// (two SMs, tcgen05 cta_group::2) walks the tiles; tiles of a product wait
// for their own matrix's counter of finished tiles, never for the whole grid,
// so a batch's matrices fill each other's gaps and a small matrix pays a
// counter's round trip where it paid a launch.  The walk is in dependency
// order and the launch cooperative (every pair resident), so each wait ends.
//
// Per CTA: warp 0 feeds a ring of five 32 KB stages by TMA (128 rows of op1,
// half of op2's columns, one copy each), the leader's warp 1 issues the
// pair's tensor-core instructions into one of two accumulators, warps 2 to 9
// empty the other one, so a tile's epilogue runs under the next tile's
// products.  An SM takes in 64 bytes per clock at most.  256 x 256 tiles on a
// pair need just that at the tensor cores' full rate (measured: 512 cycles
// per 64 contraction indices, the ideal, in A; 500 in A A; 570 to 620 in the
// update, whose epilogue reads and writes twice as much); 256 x 128 tiles
// need 96 and take 400 cycles in place of 256, but spread few tiles over more
// SMs; 128 x 256 on one SM would need 96 too.
//
// Two epilogue warps share 32 rows.  A warp's elementwise operand comes by
// TMA into its staging buffer of 32 x 64 and the result leaves from there by
// TMA, both halves of a row in place; a symmetric result below the diagonal
// blocks is staged a second time transposed.
//
// Measured (five steps, calls back to back, two cards): 3 x 2048 x 8192 1.76
// to 1.85 ms = 905 to 953 TFLOP/s of useful work and 11008 x 4096 2.85 to 2.96
// ms = 1053 to 1092, at 1.2 to 1.3 GHz under the power limit (79 % of the
// tensor pipe's cycles; a library's fp16 product of the same operands sustains
// 1250 to 1310).  512 x 512 95 us as a graph's replay, 15 products of some 11 k
// cycles: 3 k of copies and products, 4 k to the result's visibility, 2 k to
// the next product's first load.  A long thin matrix has one or two tiles of
// A, and as many pairs contract its whole length: 128 x 4097 133 us, 128 x
// 11008 242, 256 x 8192 189.
template <int NG, bool APPLY>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kIterThreads, 1)
zr_ns_iterate_kernel(const __grid_constant__ IterLaunch<NG> L) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];       // the swizzle's period
    uint32_t* words = reinterpret_cast<uint32_t*>(smem_raw + kSmemBars + 8 * kBars);
    uint32_t& s_tmem = words[0];
    volatile uint32_t& s_abort = words[1];
    const uint32_t smem = smem_u32(smem_raw);
    const uint32_t ready = smem_u32(words + 2);     // tiles whose operands are written
    const uint32_t full = smem + kSmemBars, empty = full + 8 * kStages;
    const uint32_t acc_full = empty + 8 * kStages, acc_empty = acc_full + 16, staged_in = acc_empty + 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t rank = blockIdx.x & 1, pair = blockIdx.x >> 1;
    const Bail bail{&s_abort, L.abort_word, L.gave_up};

    if (threadIdx.x == 0) {
        s_abort = 0u;
        words[2] = 0u;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(acc_empty + 8 * i, 2 * kEpiWarps);
        }
        for (int i = 0; i < kEpiWarps; ++i) mbar_init(staged_in + 8 * i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_shared();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    L.maps.fence(L.n_groups);
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = s_tmem;

    if (warp == 0) {
        if (elect_one()) {
            const uint32_t pair_full = leader_address(full);
            fence_async_global();      // the kernel before this one wrote X_0 by ordinary stores
            uint32_t s = 0, phase = 1, seen = 0;
            bool ok = true;
            for (TileWalk<NG> walk(L, pair); ok && walk.live(); walk.next()) {
                const TileAt at = walk.at();
                const IterGroup& g = L.g[at.group];
                const IterMaps& maps = L.maps.of(at.group);
                const int from = at.step & 1;
                const CUtensorMap* op1 = at.op == kGram ? &maps.gram1[from] : at.op == kPoly ? &maps.poly1 : &maps.update1[from];
                const CUtensorMap* op2 = at.op == kGram ? &maps.gram2[from] : at.op == kPoly ? &maps.poly2 : &maps.update2[from];
                const uint32_t need = shares_before(g, at);
                if (need != 0) {
                    if (!count_wait(g.done + at.slot, need, bail)) break;
                    fence_async_global();
                }
                st_shared_release(ready, ++seen);
                const int32_t k = at.op == kGram ? max(g.m, g.n) : g.dim;
                const int32_t nk = (k + kBK - 1) / kBK;
                // A box of a K-major operand is 64 contraction indices x 64 or
                // 128 rows; of an MN-major one, one or two chunks of 64 columns
                // x 64 contraction indices (one chunk: columns as they are).
                const bool mn1 = at.op == kGram && g.tall, mn2 = at.op == kGram ? g.tall : at.op == kUpdate && !g.tall;
                const bool chunks2 = mn2 && at.bn == kBN;
                const int32_t r0 = at.row0 + rank * 128, c0 = at.col0 + rank * (at.bn / 2);
                const uint32_t bytes = 2 * (kOpBytes + at.bn / 128 * kBoxBytes);
                for (int32_t kb = 0; kb < nk; ++kb) {
                    if (!mbar_wait(empty + 8 * s, phase, bail)) {
                        ok = false;
                        break;
                    }
                    const int32_t k0 = kb * kBK;
                    const uint32_t dst = smem + s * kStageBytes, bar = pair_full + 8 * s;
                    if (rank == 0) mbar_expect(full + 8 * s, bytes);
                    tma_load_pair(dst, op1, mn1 ? 0 : k0, mn1 ? k0 : r0, mn1 ? r0 / 64 : 0, at.slot, bar);
                    tma_load_pair(dst + kOpBytes, op2, !mn2 ? k0 : chunks2 ? 0 : c0, mn2 ? k0 : c0, chunks2 ? c0 / 64 : 0, at.slot, bar);
                    if (++s == kStages) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            uint32_t it = 0, acc = 0;
            bool ok = true;
            for (TileWalk<NG> walk(L, pair); ok && walk.live(); walk.next(), ++acc) {
                const TileAt at = walk.at();
                const IterGroup& g = L.g[at.group];
                const uint32_t mn1 = at.op == kGram && g.tall, mn2 = at.op == kGram ? g.tall : at.op == kUpdate && !g.tall;
                const int32_t k = at.op == kGram ? max(g.m, g.n) : g.dim;
                const int32_t nk = (k + kBK - 1) / kBK;
                const uint32_t buf = acc & 1;
                if (!mbar_wait(acc_empty + 8 * buf, ((acc >> 1) & 1) ^ 1, bail)) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t d = tmem + buf * kBN;
                // fp32 accumulators, fp16 operands, their majors, N / 8, M / 16
                const uint32_t idesc = (1u << 4) | (mn1 << 15) | (mn2 << 16) | (static_cast<uint32_t>(at.bn >> 3) << 17) |
                                       ((kBM >> 4) << 24);
                const uint32_t step1 = (mn1 ? 16 * 128 : 32) >> 4, step2 = (mn2 ? 16 * 128 : 32) >> 4;
                for (int32_t kb = 0; kb < nk; ++kb, ++it) {
                    const uint32_t s = it % kStages, phase = (it / kStages) & 1;
                    if (!mbar_wait(full + 8 * s, phase, bail)) {
                        ok = false;
                        break;
                    }
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint32_t base = smem + s * kStageBytes;
                    const uint64_t d1 = smem_desc(base, mn1, kBoxBytes), d2 = smem_desc(base + kOpBytes, mn2, kBoxBytes);
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
        const int turn = (warp - 2) >> 2;          // its chunks of 64 columns: turn, turn + 2
        const uint32_t hi = smem + kSmemStaging + (warp - 2) * kBufBytes, lo = hi + kPartBytes;
        const uint32_t diag_cols = smem + kSmemDiag + (warp - 2) * kDiagBytes;
        const uint32_t in_bar = staged_in + 8 * (warp - 2);
        const uint32_t free_bar = leader_address(acc_empty);
        uint32_t in_phase = 0;                     // parity of the next load
        const bool one = elect_one();              // the lane that issues this warp's copies
        uint32_t acc = 0;
        // One tile; the product, whether it is the last and which way X lies
        // are compile-time choices (as branches they cost 2 to 6 %; graph
        // replays: 6 x 777 x 1025 201 us against 194, the step of 333 x 517, 1
        // x 2000 and 640 x 1 107 against 101).
        auto tile = [&](const TileAt& at, auto op_, auto last_, auto tall_) -> bool {
            constexpr int OP = decltype(op_)::value;
            constexpr bool sym = OP != kUpdate, last = decltype(last_)::value, tall = decltype(tall_)::value;
            const IterGroup& g = L.g[at.group];
            const int32_t rows = sym ? g.dim : g.m, cols = sym ? g.dim : g.n;
            const int32_t row_w = at.row0 + rank * 128 + quad * 32, row = row_w + lane;
            const int32_t chunks = row_w < rows ? (min(at.bn, cols - at.col0) + 63) / 64 : 0;
            const uint32_t buf = acc & 1;
            const IterMaps& maps = L.maps.of(at.group);
            auto load = [&](int ch) {              // lane 0: the elementwise operand of a chunk
                const int32_t x = at.col0 + ch * 64;
                mbar_expect(in_bar, sym ? kPartBytes : 2 * kPartBytes);
                if (sym) tma_load_3d(hi, &maps.egram, x, row_w, at.slot, in_bar);
                else tma_load_4d(hi, &maps.ex[at.step & 1], x, row_w, 0, at.slot, in_bar);
            };
            const Affine k = L.k[last ? 3 : OP];
            const float* diag = (OP == kPoly ? g.gram_diag : g.poly_diag) + static_cast<int64_t>(at.slot) * g.dim;
            constexpr bool by_row = OP == kPoly || !tall, by_col = OP == kPoly || tall;         // of the diagonal
            float dr = 0.0f;
            if (OP != kGram && turn < chunks) {
                bool ok = true;
                if (one) {
                    // what the producer has acquired from the matrix's
                    // counter, this lane acquires from its word, and the
                    // barrier below passes on to the warp (a vote would not)
                    auto written = [&] { return ld_shared_acquire(ready) > acc; };
                    ok = written() || wait_slow(written, bail);
                    if (ok) {
                        store_wait_read<0>();      // the buffer is free
                        fence_async();
                        load(turn);
                    }
                }
                if (!__all_sync(0xFFFFFFFFu, ok)) return false;
                __syncwarp();
                if (by_row && row < rows) dr = __ldcg(diag + row);
            }
            const uint32_t tm = tmem + (static_cast<uint32_t>(quad * 32) << 16) + buf * kBN;
            const bool mirror = sym && at.col0 + at.bn <= at.row0;      // diagonal blocks are whole as they are
            auto products = [&] {                  // the accumulator is complete
                const bool done = __all_sync(0xFFFFFFFFu, mbar_wait(acc_full + 8 * buf, (acc >> 1) & 1, bail));
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                return done;
            };
            bool ok = true;
#pragma unroll 1
            for (int ch = turn; ch < chunks; ch += 2) {
                const int32_t c = at.col0 + ch * 64;
                // y: the elementwise term of a row's 64 columns, formed while
                // the products still run
                f32x2 y[2][16];
                if constexpr (OP == kGram) {
                    if (one) store_wait_read<0>();
                } else {
                    if (by_col) {
                        float d[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j) d[j] = c + 32 * j + lane < cols ? __ldcg(diag + c + 32 * j + lane) : 0.0f;
                        st_shared_f32(diag_cols + 4 * lane, d[0]);
                        st_shared_f32(diag_cols + 128 + 4 * lane, d[1]);
                        __syncwarp();
                    }
                    if (!(ok = __all_sync(0xFFFFFFFFu, mbar_wait(in_bar, in_phase, bail)))) break;
                    in_phase ^= 1u;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        ld_staged32(hi, lane, 4 * half, y[half]);
                        if (OP == kPoly) {
                            // c A A + b A, A = D + R: acc = R R, y = b R + c (D R + R D) + (b D + c D D)
                            const float s = k.gamma * (1.0f / kNsScaleA), base = fmaf(dr, s, k.beta);
#pragma unroll
                            for (int i = 0; i < 16; i += 2) {
                                f32x2 d[2];
                                ld_shared_f32x4(diag_cols + 128 * half + 8 * i, d);
#pragma unroll
                                for (int j = 0; j < 2; ++j)
                                    y[half][i + j] = mul2(y[half][i + j], fma2(d[j], pack2(s, s), pack2(base, base)));
                            }
                            if (c + 32 * half == row_w) {
                                const float on = fmaf(dr, k.gamma, k.beta * kNsScaleA) * dr;
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    const float2 f = unpack2(y[half][i]);
                                    y[half][i] = pack2(2 * i == lane ? on : f.x, 2 * i + 1 == lane ? on : f.y);
                                }
                            }
                        } else {
                            f32x2 e[16];
                            ld_staged32(lo, lane, 4 * half, e);
                            constexpr float kLo = 1.0f / kNsScaleLo;
#pragma unroll
                            for (int i = 0; i < 16; ++i) y[half][i] = fma2(e[i], pack2(kLo, kLo), y[half][i]);
                            if (tall) {
#pragma unroll
                                for (int i = 0; i < 16; i += 2) {
                                    f32x2 d[2];
                                    ld_shared_f32x4(diag_cols + 128 * half + 8 * i, d);
#pragma unroll
                                    for (int j = 0; j < 2; ++j)
                                        y[half][i + j] = mul2(y[half][i + j], fma2(d[j], pack2(k.gamma, k.gamma), pack2(k.beta, k.beta)));
                                }
                            } else {
                                const float d = fmaf(dr, k.gamma, k.beta);
#pragma unroll
                                for (int i = 0; i < 16; ++i) y[half][i] = mul2(y[half][i], pack2(d, d));
                            }
                        }
                    }
                }
                if constexpr (last && APPLY) {      // the master weights, towards L2 while the products run
                    if (row < rows) {
                        const float* pm = L.master + g.master_offsets[at.slot] + static_cast<int64_t>(row) * cols + c;
                        prefetch_l2(pm);
                        if (c + 32 < cols) prefetch_l2(pm + 32);
                    }
                }
                if (ch == turn && !(ok = products())) break;
                __syncwarp();
                // v: 32 columns of the result from column c + 32 half on
                auto result = [&](int half, f32x2(&v)[16]) {
                    tmem_ld32(tm + ch * 64 + half * 32, v);
                    const f32x2 alpha = pack2(k.alpha, k.alpha);
                    if (OP == kGram) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = mul2(v[i], alpha);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = fma2(v[i], alpha, y[half][i]);
                    }
                };
                auto release = [&] {               // the accumulator is read
                    if (ch + 2 < chunks) return;
                    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                    __syncwarp();
                    if (one) mbar_arrive_cluster(free_bar + 8 * buf);
                };
                if constexpr (!last) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        f32x2 v[16];
                        result(half, v);
                        if (sym && c + 32 * half == row_w) {
                            float d = 0.0f;
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float2 f = unpack2(v[i]);
                                d = 2 * i == lane ? f.x : 2 * i + 1 == lane ? f.y : d;
                                v[i] = pack2(2 * i == lane ? 0.0f : f.x, 2 * i + 1 == lane ? 0.0f : f.y);
                            }
                            if (row < rows)
                                (OP == kGram ? g.gram_diag : g.poly_diag)[static_cast<int64_t>(at.slot) * g.dim + row] =
                                    d * (OP == kGram ? 1.0f / kNsScaleA : 1.0f / kNsScaleB);
                        }
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 f = unpack2(v[i]);
                            w[i] = half2_bits(f.x, f.y);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            st_shared16(staged(hi, lane, 4 * half + i), make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
                        if (!sym) {
                            const f32x2 up = pack2(kNsScaleLo, kNsScaleLo), down = pack2(-kNsScaleLo, -kNsScaleLo);
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float2 h = half2_values(w[i]);
                                const float2 f = unpack2(fma2(pack2(h.x, h.y), down, mul2(v[i], up)));
                                w[i] = half2_bits(f.x, f.y);
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                st_shared16(staged(lo, lane, 4 * half + i),
                                            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
                        } else if (mirror) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                st_shared2(lo + (32 * half + i) * 64 + lane * 2,
                                           static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1))));
                        }
                    }
                    fence_async_shared();
                    __syncwarp();
                    if (one) {
                        if (sym) {
                            tma_store_3d(OP == kGram ? &maps.egram : &maps.epoly, c, row_w, at.slot, hi);
                            if (mirror)
                                tma_store_3d(OP == kGram ? &maps.mgram : &maps.mpoly, row_w, c, at.slot, lo);
                        } else {
                            tma_store_4d(&maps.ex[(at.step & 1) ^ 1], c, row_w, 0, at.slot, hi);
                        }
                        store_commit();
                        if (OP != kGram && ch + 2 < chunks) {
                            store_wait_read<0>();
                            load(ch + 2);
                        }
                    }
                    release();
                } else if constexpr (!APPLY) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        f32x2 v[16];
                        result(half, v);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t w[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float2 f = unpack2(v[4 * i + j]);
                                w[j] = bf16_bits(f.x) | (static_cast<uint32_t>(bf16_bits(f.y)) << 16);
                            }
                            st_shared16(staged(hi, lane, 4 * half + i), make_uint4(w[0], w[1], w[2], w[3]));
                        }
                    }
                    release();
                    __syncwarp();
                    uint16_t* out = g.out + at.slot * g.out_batch;
                    if (g.out_vec) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int r = 4 * i + (lane >> 3), piece = lane & 7;
                            const int32_t cc = c + 8 * piece;
                            if (row_w + r >= rows || cc >= cols) continue;
                            uint16_t* p = out + static_cast<int64_t>(row_w + r) * g.out_row + cc;
                            const uint4 q = ld_shared16(staged(hi, r, piece));
                            if (cc + 8 <= cols) {
                                *reinterpret_cast<uint4*>(p) = q;
                            } else {
                                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                                for (int j = 0; j < 8; ++j)
                                    if (cc + j < cols) p[j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
                            }
                        }
                    } else {
#pragma unroll 8
                        for (int i = 0; i < 64; ++i) {
                            const int r = i >> 1, cl = 32 * (i & 1) + lane;
                            if (row_w + r < rows && c + cl < cols)
                                out[static_cast<int64_t>(row_w + r) * g.out_row + c + cl] =
                                    ld_shared2(staged(hi, r, cl >> 3) + 2 * (cl & 7));
                        }
                    }
                    __syncwarp();
                    if (one && ch + 2 < chunks) {
                        fence_async_shared();
                        load(ch + 2);
                    }
                } else {
                    // (every row's operand has been read) the result takes its place, 256 bytes a row
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        f32x2 v[16];
                        result(half, v);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 f = unpack2(v[2 * i]), h = unpack2(v[2 * i + 1]);
                            st_shared16(hi + lane * 256 + (((8 * half + i) ^ (lane & 7)) << 4),
                                        make_uint4(__float_as_uint(f.x), __float_as_uint(f.y), __float_as_uint(h.x), __float_as_uint(h.y)));
                        }
                    }
                    release();
                    __syncwarp();
                    const int64_t e0 = static_cast<int64_t>(row_w) * cols + c + lane;
                    float* pm = L.master + g.master_offsets[at.slot] + e0;
                    const int64_t po = g.param_offsets[at.slot] + e0;
                    // (two rows at a time: more spill, and the weights come from L2)
#pragma unroll 1
                    for (int r0 = 0; r0 < 32; r0 += 2) {
                        float p[2][2];
#pragma unroll
                        for (int r = 0; r < 2; ++r)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                if (row_w + r0 + r < rows && c + 32 * j + lane < cols)
                                    p[r][j] = pm[(r0 + r) * cols + 32 * j];
#pragma unroll
                        for (int r = 0; r < 2; ++r)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                if (row_w + r0 + r < rows && c + 32 * j + lane < cols) {
                                    const int cl = 32 * j + lane;
                                    const float o = ld_shared_f32(hi + (r0 + r) * 256 + (((cl >> 2) ^ ((r0 + r) & 7)) << 4) + 4 * (cl & 3));
                                    const float q = __fsub_rn(__fmul_rn(p[r][j], L.decay), __fmul_rn(o, g.step_size));
                                    const int32_t e = (r0 + r) * cols + 32 * j;      // at most 32 rows of 2^24
                                    pm[e] = q;
                                    const uint16_t u = bf16_bits(q);
                                    if (L.n_targets == 0) L.param_out[po + e] = u;
                                    else
                                        for (int t = 0; t < L.n_targets; ++t) L.targets[t][po + e] = u;
                                }
                    }
                    __syncwarp();
                    if (one && ch + 2 < chunks) {
                        fence_async_shared();
                        load(ch + 2);
                    }
                }
            }
            if (!ok) return false;
            if (turn >= chunks) {
                if (!products()) return false;
                __syncwarp();
                if (one) mbar_arrive_cluster(free_bar + 8 * buf);
            }
            if (!last) {
                __syncwarp();
                if (one) {
                    store_wait();
                    fence_async_global();
                    red_release(g.done + at.slot, 1u);
                }
            }
            return true;
        };
        for (TileWalk<NG> walk(L, pair); walk.live(); walk.next(), ++acc) {
            const TileAt at = walk.at();
            using Yes = std::true_type;
            using No = std::false_type;
            const bool last = at.step + 1 == L.steps, tall = L.g[at.group].tall;
            bool ok;
            if (at.op == kGram) ok = tile(at, std::integral_constant<int, kGram>{}, No{}, No{});
            else if (at.op == kPoly) ok = tile(at, std::integral_constant<int, kPoly>{}, No{}, No{});
            else if (!last && !tall) ok = tile(at, std::integral_constant<int, kUpdate>{}, No{}, No{});
            else if (!last) ok = tile(at, std::integral_constant<int, kUpdate>{}, No{}, Yes{});
            else if (!tall) ok = tile(at, std::integral_constant<int, kUpdate>{}, Yes{}, No{});
            else ok = tile(at, std::integral_constant<int, kUpdate>{}, Yes{}, Yes{});
            if (!ok) break;
        }
        if (one) store_wait();
    }
    // Every role is done (or gave up).  A pair that gave up may still have
    // copies and products in flight: the copies land within microseconds, and
    // a commit after the products arrives when they are done.
    __syncwarp();
    __syncthreads();
    if (s_abort) {
        if (threadIdx.x == 32 && rank == 0) {
            const uint32_t was = mbar_try(acc_full, 0) ? 1u : 0u;
            mma_commit(acc_full);
            for (uint32_t i = 0; i < kDrainTries && !mbar_try(acc_full, was); ++i) {}
        }
        for (int i = 0; i < 1000; ++i) __nanosleep(1000);
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncwarp();
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
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
    uint32_t* done;
};
struct PrepLaunch {
    int32_t n_groups;
    uint32_t *abort_word, *gave_up;
    int32_t total_matrices, own_scale;    // own_scale: every CTA of the start kernel adds up its matrix's partials
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
    if (threadIdx.x == 0 && blockIdx.x == 0 && L.gave_up) *L.gave_up = 0u;
    if (threadIdx.x == 0) g.partials[static_cast<int64_t>(at.slot) * g.n_partials + at.piece] = sum;
}

// A matrix's scale from its partials, in a fixed order; valid in thread 0.
__device__ __forceinline__ float2 matrix_scale(const PrepGroup& g, int32_t slot, double eps) {
    const int64_t first = g.first_partial ? g.first_partial[slot] : static_cast<int64_t>(slot) * g.n_partials;
    const int64_t last = g.first_partial ? g.first_partial[slot + 1] : first + g.n_partials;
    double sum = 0.0;
#pragma unroll 4
    for (int64_t i = first + threadIdx.x; i < last; i += kPrepThreads) sum += __ldcg(g.partials + i);
    return ns_scale_of(prep_block_sum(sum), eps);
}

// One CTA per matrix, for matrices of many partials.
__global__ void __launch_bounds__(kPrepThreads) zr_ns_scale_kernel(const __grid_constant__ PrepLaunch L) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    int32_t slot = blockIdx.x, gi = 0;
    while (slot >= L.g[gi].batch) slot -= L.g[gi++].batch;
    const PrepGroup& g = L.g[gi];
    const float2 scale = matrix_scale(g, slot, L.eps);
    if (threadIdx.x == 0) g.scale[slot] = scale;
}

__global__ void __launch_bounds__(kPrepThreads) zr_ns_start_kernel(const __grid_constant__ PrepLaunch L) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const PieceAt at = find_piece(L);
    const PrepGroup& g = L.g[at.group];
    if (threadIdx.x == 0 && at.piece == 0) {       // the iteration kernel's words
        g.done[at.slot] = 0u;
        if (at.group == 0 && at.slot == 0) *L.abort_word = 0u;
    }
    float2 s;
    if (L.own_scale) {
        __shared__ float2 own;
        const float2 mine = matrix_scale(g, at.slot, L.eps);
        if (threadIdx.x == 0) own = mine;
        __syncthreads();
        s = own;
    } else {
        s = g.scale[at.slot];
    }
    if (at.col >= g.cols) return;
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

// Copies of a batch of cols x rows fp16 matrices, or of `parts` such batches
// part_bytes apart: boxes of box_cols x box_rows x box_parts.  What lies
// outside a matrix reads as zero and is not written.
int encode_map(CUtensorMap* map, int dimensions, void* base, int64_t cols, int64_t rows, int64_t parts, int64_t batch,
               int64_t row_bytes, int64_t part_bytes, int64_t matrix_bytes, int box_cols, int box_rows, int box_parts,
               CUtensorMapSwizzle swizzle) {
    const EncodeTiled fn = encode_tiled();
    if (!fn) return cudaErrorNotSupported;
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(parts),
                          static_cast<cuuint64_t>(batch)};
    cuuint64_t strides[3] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(part_bytes),
                             static_cast<cuuint64_t>(matrix_bytes)};
    cuuint32_t box[4] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows),
                         static_cast<cuuint32_t>(box_parts), 1};
    const cuuint32_t unit[4] = {1, 1, 1, 1};
    if (dimensions == 3) {
        dims[2] = dims[3];
        strides[1] = strides[2];
        box[2] = 1;
    }
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, dimensions, base, dims, strides, box, unit,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

uint64_t align256(uint64_t x) { return (x + 255) & ~uint64_t(255); }

// Tiles of a symmetric result (row blocks of 256, the columns up to the
// diagonal block; only the last row block may have fewer) and of a full one.
int64_t symmetric_tiles(int64_t g, int bn) {
    const int64_t i = (g + kBM - 1) / kBM;
    return i * (i - 1) / 2 * (kBM / bn) + (g + bn - 1) / bn;
}
int64_t full_tiles(int64_t rows, int64_t cols, int bn) { return ((rows + kBM - 1) / kBM) * ((cols + bn - 1) / bn); }

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

// CTA pairs that run at once, with the kernel's shared memory allowed on the
// device; 0 on failure.
template <int NG, bool APPLY>
int resident_pairs() {
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = known[dev].load(std::memory_order_acquire);
    if (n > 0) return n;
    auto kernel = zr_ns_iterate_kernel<NG, APPLY>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kIterSmem) != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kIterThreads);
    cfg.dynamicSmemBytes = kIterSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {2, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) return 0;
    known[dev].store(n, std::memory_order_release);
    return n;
}

// 256-column tiles, or 128 where that gives the pairs an evener share.  In
// cycles: 64 contraction indices take a pair 520 or 400, what follows a wave's
// products some 9000 or 4000.
int pick_columns(int64_t tiles256, int64_t tiles128, int64_t pairs, int64_t k) {
    const int64_t waves256 = (tiles256 + pairs - 1) / pairs, waves128 = (tiles128 + pairs - 1) / pairs;
    const int64_t blocks = (k + kBK - 1) / kBK;
    return waves128 * blocks * 400 + 4000 < waves256 * blocks * 520 + 9000 ? 128 : 256;
}

struct Tiling { int sym_bn, out_bn; };
Tiling tiling(const NsGroup* groups, int32_t n, int64_t pairs) {
    int64_t sym[2] = {0, 0}, out[2] = {0, 0}, k_sym = 0, k_out = 0;
    for (int32_t i = 0; i < n; ++i) {
        for (int h = 0; h < 2; ++h) {
            sym[h] += groups[i].batch * symmetric_tiles(groups[i].gram_dim(), kBN >> h);
            out[h] += groups[i].batch * full_tiles(groups[i].m, groups[i].n, kBN >> h);
        }
        k_sym = std::max(k_sym, std::max(groups[i].m, groups[i].n));
        k_out = std::max(k_out, groups[i].gram_dim());
    }
    return {pick_columns(sym[0], sym[1], pairs, k_sym), pick_columns(out[0], out[1], pairs, k_out)};
}

void fill_maps(IterMaps& o, const NsGroup& s, Tiling t) {
    const NsMaps& m = s.maps;
    const bool sym_half = t.sym_bn != kBN, out_half = t.out_bn != kBN, tall = s.m > s.n;
    for (int j = 0; j < 2; ++j) {
        o.gram1[j] = tall ? m.x_chunks[j] : m.x_rows[j];
        o.gram2[j] = sym_half ? m.x_box[j] : o.gram1[j];
        o.update1[j] = tall ? m.x_rows[j] : m.poly_rows;
        o.update2[j] = tall ? (out_half ? m.poly_box : m.poly_rows) : out_half ? m.x_box[j] : m.x_chunks[j];
        o.ex[j] = m.ex[j];
    }
    o.poly1 = m.gram_rows;
    o.poly2 = sym_half ? m.gram_box : m.gram_rows;
    o.egram = m.egram;
    o.epoly = m.epoly;
    o.mgram = m.mgram;
    o.mpoly = m.mpoly;
}

template <int NG, bool APPLY>
int launch_iterate(const NsGroup* groups, int32_t n, const IterMaps* maps, int32_t steps, const float coeffs[3],
                   const NsApply& apply, uint32_t* gave_up, void* stream) {
    const int most = resident_pairs<NG, APPLY>();
    if (most == 0) return cudaErrorLaunchOutOfResources;
    IterLaunch<NG> L{};
    L.n_groups = n;
    L.steps = steps;
    ns_factors(L.k, coeffs);
    const Tiling t = tiling(groups, n, resident_pairs<NG, APPLY>());
    L.sym_bn = t.sym_bn;
    L.out_bn = t.out_bn;
    if constexpr (NG == 1) fill_maps(L.maps.one, groups[0], t);
    else L.maps.all = maps;
    L.decay = apply.decay;
    L.abort_word = groups[0].done + groups[0].batch;
    L.gave_up = gave_up;
    L.master = apply.master;
    L.param_out = apply.param_out;
    L.targets = apply.targets;
    L.n_targets = apply.n_targets;
    for (int32_t i = 0; i < n; ++i) {
        const NsGroup& s = groups[i];
        IterGroup& g = L.g[i];
        g.m = static_cast<int32_t>(s.m);
        g.n = static_cast<int32_t>(s.n);
        g.dim = static_cast<int32_t>(s.gram_dim());
        g.tall = s.m > s.n;
        g.sym_tiles = static_cast<int32_t>(symmetric_tiles(s.gram_dim(), L.sym_bn));
        g.out_tiles = static_cast<int32_t>(full_tiles(s.m, s.n, L.out_bn));
        g.out_tiles_n = static_cast<int32_t>((s.n + L.out_bn - 1) / L.out_bn);
        g.first_sym = L.sym_total;
        g.first_out = L.out_total;
        L.sym_total += s.batch * g.sym_tiles;
        L.out_total += s.batch * g.out_tiles;
        g.done = s.done;
        g.gram_diag = s.gram_diag;
        g.poly_diag = s.poly_diag;
        g.out = s.out;
        g.out_row = s.out_row;
        g.out_batch = s.out_batch;
        g.out_vec = reinterpret_cast<uintptr_t>(s.out) % 16 == 0 && s.out_row % 8 == 0 && s.out_batch % 8 == 0;
        g.master_offsets = s.master_offsets;
        g.param_offsets = s.param_offsets;
        g.step_size = s.step_size;
    }
    L.pairs = static_cast<int32_t>(std::min<int64_t>(most, std::max(L.sym_total, L.out_total)));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2 * static_cast<unsigned>(L.pairs));
    cfg.blockDim = dim3(kIterThreads);
    cfg.dynamicSmemBytes = kIterSmem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;       // every pair resident: see the kernel's waits
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, zr_ns_iterate_kernel<NG, APPLY>, L);
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
        g.done = s.done;
        pieces += s.batch * g.pieces_per_matrix;
        matrices += s.batch;
    }
    L.total_matrices = static_cast<int32_t>(matrices);
    L.abort_word = groups[0].done + groups[0].batch;
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
    // the counter of a matrix over 32 steps stays below 2^32
    if (2 * symmetric_tiles(g, kBN / 2) + full_tiles(m, n, kBN / 2) >= (1ll << 32) / (32 * 2 * kEpiWarps)) return false;
    return batch * ns_partials_per_matrix(m, n) < (1ll << 31);
}

uint64_t ns_scratch_bytes(int64_t batch, int64_t m, int64_t n) {
    NsGroup g;
    g.batch = batch;
    g.m = m;
    g.n = n;
    const uint64_t x = align256(static_cast<uint64_t>(batch) * m * g.ld() * 2);
    const uint64_t a = align256(static_cast<uint64_t>(batch) * g.gram_dim() * g.ldg() * 2);
    return 4 * x + 2 * a + 2 * align256(static_cast<uint64_t>(batch) * g.gram_dim() * sizeof(float)) +
           align256((static_cast<uint64_t>(batch) + 1) * sizeof(uint32_t));
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
    const uint64_t d = align256(static_cast<uint64_t>(g.batch) * g.gram_dim() * sizeof(float));
    g.poly_diag = reinterpret_cast<float*>(p + 4 * x + 2 * a + d);
    g.done = reinterpret_cast<uint32_t*>(p + 4 * x + 2 * a + 2 * d);
    NsMaps& t = g.maps;
    int e = cudaSuccess;
    const int64_t dim = g.gram_dim(), x_row = 2 * g.ld(), a_row = 2 * g.ldg();
    constexpr CUtensorMapSwizzle k128 = CU_TENSOR_MAP_SWIZZLE_128B, kNone = CU_TENSOR_MAP_SWIZZLE_NONE;
    auto box = [&](CUtensorMap* map, void* at, bool gram, int rows) {          // an operand's: 64 x rows
        if (e != cudaSuccess) return;
        e = gram ? encode_map(map, 4, at, dim, dim, 1, g.batch, a_row, dim * a_row, dim * a_row, 64, rows, 1, k128)
                 : encode_map(map, 4, at, g.n, g.m, 1, g.batch, x_row, g.m * x_row, g.m * x_row, 64, rows, 1, k128);
    };
    auto share = [&](CUtensorMap* map, void* at, int cols, int rows, CUtensorMapSwizzle swizzle) {
        if (e == cudaSuccess)
            e = encode_map(map, 3, at, dim, dim, 1, g.batch, a_row, 0, dim * a_row, cols, rows, 1, swizzle);
    };
    for (int i = 0; i < 2; ++i) {
        box(&t.x_box[i], g.xh[i], false, 64);
        box(&t.x_rows[i], g.xh[i], false, 128);
        // chunks of 64 columns, two at a time: the last reaches into the rows'
        // padding, whose columns are rows or columns of a product that no
        // result keeps
        if (e == cudaSuccess)
            e = encode_map(&t.x_chunks[i], 4, g.xh[i], 64, g.m, (g.n + 63) / 64, g.batch, x_row, 128, g.m * x_row, 64, 64, 2, k128);
        if (e == cudaSuccess)
            e = encode_map(&t.ex[i], 4, g.xh[i], g.n, g.m, 2, g.batch, x_row, static_cast<int64_t>(x), g.m * x_row, 64, 32, 2, k128);
    }
    box(&t.gram_box, g.gram, true, 64);
    box(&t.gram_rows, g.gram, true, 128);
    box(&t.poly_box, g.poly, true, 64);
    box(&t.poly_rows, g.poly, true, 128);
    share(&t.egram, g.gram, 64, 32, k128);
    share(&t.epoly, g.poly, 64, 32, k128);
    share(&t.mgram, g.gram, 32, 64, kNone);
    share(&t.mpoly, g.poly, 32, 64, kNone);
    return e;
}

int launch_ns_sumsq(const NsGroup& group, uint32_t* gave_up, void* stream) {
    PrepLaunch L{};
    const int64_t pieces = fill_prep(L, &group, 1);
    if (pieces > 0x7FFFFFFF) return cudaErrorInvalidValue;
    L.gave_up = gave_up;
    Dependent<PrepLaunch> d(static_cast<unsigned>(pieces), kPrepThreads, 0, stream);
    return d.run(zr_ns_sumsq_kernel, L);
}

int launch_ns_iterations(const NsGroup* groups, int32_t n_groups, int32_t steps, const float coeffs[3], double eps,
                         const NsApply& apply, const void* device_maps, uint32_t* gave_up, void* stream) {
    const IterMaps* maps = static_cast<const IterMaps*>(device_maps);
    if (!apply.master && n_groups > 1) return cudaErrorInvalidValue;
    for (int32_t at = 0; at < n_groups; at += kMaxGroups) {
        const NsGroup* gs = groups + at;
        const int32_t n = std::min(kMaxGroups, n_groups - at);
        PrepLaunch P{};
        const int64_t pieces = fill_prep(P, gs, n);
        if (pieces > 0x7FFFFFFF) return cudaErrorInvalidValue;
        P.eps = eps;
        // Up to 4 partials a thread cost less than a launch.
        int64_t partials = 0;
        for (int32_t i = 0; i < n; ++i) partials = std::max<int64_t>(partials, gs[i].n_partials);
        P.own_scale = partials <= 4 * kPrepThreads;
        if (!P.own_scale) {
            Dependent<PrepLaunch> d(static_cast<unsigned>(P.total_matrices), kPrepThreads, 0, stream);
            const cudaError_t e = d.run(zr_ns_scale_kernel, P);
            if (e != cudaSuccess) return e;
        }
        Dependent<PrepLaunch> d(static_cast<unsigned>(pieces), kPrepThreads, 0, stream);
        int e = d.run(zr_ns_start_kernel, P);
        if (e != cudaSuccess) return e;
        if (!apply.master)                 // one group (zr_orthogonalize)
            e = launch_iterate<1, false>(gs, 1, nullptr, steps, coeffs, apply, gave_up, stream);
        else if (n == 1)
            e = launch_iterate<1, true>(gs, n, nullptr, steps, coeffs, apply, gave_up, stream);
        else
            e = launch_iterate<kMaxGroups, true>(gs, n, maps + at, steps, coeffs, apply, gave_up, stream);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

uint64_t ns_maps_bytes(int32_t n_groups) { return sizeof(IterMaps) * static_cast<uint64_t>(n_groups); }

int ns_fill_maps(const NsGroup* groups, int32_t n_groups, void* host) {
    const int pairs = resident_pairs<kMaxGroups, true>();
    if (pairs == 0) return cudaErrorLaunchOutOfResources;
    char* to = static_cast<char*>(host);          // of any alignment
    for (int32_t at = 0; at < n_groups; at += kMaxGroups) {
        const int32_t n = std::min(kMaxGroups, n_groups - at);
        const Tiling t = tiling(groups + at, n, pairs);
        for (int32_t i = 0; i < n; ++i) {
            IterMaps maps;
            fill_maps(maps, groups[at + i], t);
            std::memcpy(to + sizeof maps * static_cast<size_t>(at + i), &maps, sizeof maps);
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
