// The Muon step's elementwise passes for B200 (sm_100a): the replica fold
// with the momentum update, and the conversions of an 8-bit momentum.
//
// Per owned element the momentum pass reads W bf16 gradients and the
// momentum (4 bytes, or 1 + 4/256 in 8 bits), writes the momentum back and
// the fp32 update U that the orthogonalisation starts from.  Nothing is
// reused, so it is bound by HBM like the AdamW step, and takes that kernel's
// form: a 128-thread CTA per 2048 elements, eight consecutive elements per
// thread and iteration, the loads of a group of replicas issued together.
//
// An 8-bit block is 256 elements, which is one warp's share of an iteration:
// its largest magnitude is one warp reduction, and the block is read back and
// rewritten without leaving registers.
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "zr_fold.cuh"
#include "zr_internal.hpp"
#include "zr_muon.hpp"

namespace zr {
namespace {

static_assert(kMuonBlock == 32 * kElemsPerThreadIter, "a block is one warp's share");
static_assert(kMuonTileElems == kTileElems, "the tile of the AdamW step");

enum class Op : int { kMomentum = 0, kQuantize = 1, kDequantize = 2 };

__device__ __forceinline__ void load_f32(const float* p, bool vec, int n, float (&x)[8]) {
    if (vec) {
        const float4 a = ld_state16(p), b = ld_state16(p + 4);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = k < n ? p[k] : 0.0f;
    }
}
__device__ __forceinline__ void store_f32(float* p, bool vec, int n, const float (&x)[8]) {
    if (vec) {
        st_state16(p, make_float4(x[0], x[1], x[2], x[3]));
        st_state16(p + 4, make_float4(x[4], x[5], x[6], x[7]));
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) p[k] = x[k];
    }
}

// Eight codes of a block and its scale; absent elements read as zero.
__device__ __forceinline__ void load_codes(const int8_t* p, bool vec, int n, float scale, float (&x)[8]) {
    if (vec) {
        const uint2 q = __ldcs(reinterpret_cast<const uint2*>(p));
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int8_t c = static_cast<int8_t>((k < 4 ? q.x : q.y) >> (8 * (k & 3)));
            x[k] = __fmul_rn(static_cast<float>(c), scale);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = k < n ? __fmul_rn(static_cast<float>(p[k]), scale) : 0.0f;
    }
}

// The warp's 256 values as a block: scale = max|x| / 127, codes rounded to
// nearest even of x / scale.  Magnitudes are compared as integers, which
// orders NaN above infinity above every number, so a block that holds either
// gets a scale that reads back as NaN everywhere (code 0).
__device__ __forceinline__ void store_block(int8_t* p, float* scale_out, bool vec, int n, int lane, const float (&x)[8]) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, k < n ? __float_as_uint(x[k]) & 0x7FFFFFFFu : 0u);
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    const float scale = __fdiv_rn(__uint_as_float(top), 127.0f);
    const bool regular = scale > 0.0f && top < 0x7F800000u;
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        int c = regular ? __float2int_rn(__fdiv_rn(x[k], scale)) : 0;
        c = max(-127, min(127, c));      // a subnormal scale rounds by more than half a code
        w[k >> 2] |= (static_cast<uint32_t>(c) & 0xFFu) << (8 * (k & 3));
    }
    if (vec) {
        __stcs(reinterpret_cast<uint2*>(p), make_uint2(w[0], w[1]));
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) p[k] = static_cast<int8_t>(w[k >> 2] >> (8 * (k & 3)));
    }
    if (lane == 0) *scale_out = scale;
}

template <int CAP, int G, Op OP, bool EIGHT_BIT>
__global__ void __launch_bounds__(kThreads) zr_muon_kernel(const GradPtrs<CAP> gp, const MuonArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const MuonTile tile = a.tiles[blockIdx.x];
    const int lane = threadIdx.x & 31;
    double sq = 0.0;
    if constexpr (OP == Op::kQuantize) {
        // All of a thread's loads before its first store: 5.6 TB/s (147 ->
        // 136 us for 151 M elements; the other way round it costs 8 %, 152 us
        // against 141 one iteration at a time).
        constexpr int kIters = kMuonTileElems / (kThreads * 8);
        float x[kIters][8];
#pragma unroll
        for (int it = 0; it < kIters; ++it) {
            const int e = (it * kThreads + static_cast<int>(threadIdx.x)) * 8;
            const int n = max(0, min(8, tile.len - e));
            load_f32(a.momentum + tile.owned + e, n == 8 && tile.aligned, n, x[it]);
        }
#pragma unroll
        for (int it = 0; it < kIters; ++it) {
            const int e = (it * kThreads + static_cast<int>(threadIdx.x)) * 8;
            if ((e & ~(kMuonBlock - 1)) >= tile.len) break;       // the whole warp
            const int n = max(0, min(8, tile.len - e));
            store_block(a.codes + tile.owned + e, a.scales + tile.scale + e / kMuonBlock, n == 8 && tile.aligned, n, lane, x[it]);
        }
    } else {
        for (int it = 0; it < kMuonTileElems / (kThreads * 8); ++it) {
            const int e = (it * kThreads + static_cast<int>(threadIdx.x)) * 8;
            if ((e & ~(kMuonBlock - 1)) >= tile.len) break;       // the whole warp
            const int n = max(0, min(8, tile.len - e));
            const bool vec = n == 8 && tile.aligned;
            const int64_t o = tile.owned + e;
            const int64_t block = tile.scale + e / kMuonBlock;
            float x[8];
            if constexpr (OP == Op::kDequantize) {
                load_codes(a.codes + o, vec, n, a.scales[block], x);
                store_f32(a.momentum + o, vec, n, x);
            } else {
                if constexpr (EIGHT_BIT) load_codes(a.codes + o, vec, n, a.scales[block], x);
                else load_f32(a.momentum + o, vec, n, x);
                float g[8];
                if (vec) {
                    fold8<CAP, G>(gp, a.world_size, o, g);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) g[k] = k < n ? fold1<CAP>(gp, a.world_size, o + k) : 0.0f;
                }
                float u[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    g[k] = average(g[k], a);
                    x[k] = __fadd_rn(__fmul_rn(a.mu, x[k]), g[k]);
                    u[k] = a.nesterov ? __fadd_rn(g[k], __fmul_rn(a.mu, x[k])) : x[k];
                    if (k < n) sq += static_cast<double>(u[k]) * static_cast<double>(u[k]);
                }
                if constexpr (EIGHT_BIT) store_block(a.codes + o, a.scales + block, vec, n, lane, x);
                else store_f32(a.momentum + o, vec, n, x);
                // (the update's matrices start 8 elements apart: always aligned)
                store_f32(a.update + tile.update + e, n == 8, n, u);
            }
        }
    }
    if constexpr (OP == Op::kMomentum) {
        const double total = block_sum(sq);
        if (threadIdx.x == 0) a.partials[blockIdx.x] = total;
    }
}

template <int CAP, int G, Op OP, bool EIGHT_BIT>
cudaError_t launch_one(const MuonArgs& a, const void* const* grad_ptrs, cudaStream_t stream) {
    GradPtrs<CAP> gp;
    for (int w = 0; w < CAP; ++w)
        gp.p[w] = (grad_ptrs != nullptr && w < a.world_size) ? static_cast<const uint16_t*>(grad_ptrs[w]) : nullptr;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.n_tiles));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, zr_muon_kernel<CAP, G, OP, EIGHT_BIT>, gp, a);
}

template <bool EIGHT_BIT>
cudaError_t dispatch_w(const MuonArgs& a, const void* const* grad_ptrs, cudaStream_t s) {
    const int W = a.world_size;
    if (W <= 2) return launch_one<2, 2, Op::kMomentum, EIGHT_BIT>(a, grad_ptrs, s);
    if (W <= 4) return launch_one<4, 4, Op::kMomentum, EIGHT_BIT>(a, grad_ptrs, s);
    if (W <= 8) return launch_one<8, 8, Op::kMomentum, EIGHT_BIT>(a, grad_ptrs, s);
    if (W <= 16) return launch_one<16, 8, Op::kMomentum, EIGHT_BIT>(a, grad_ptrs, s);
    if (W <= 64) return launch_one<64, 8, Op::kMomentum, EIGHT_BIT>(a, grad_ptrs, s);
    return launch_one<ZR_MAX_WORLD_SIZE, 8, Op::kMomentum, EIGHT_BIT>(a, grad_ptrs, s);
}

}  // namespace

int launch_muon_momentum(const MuonArgs& a, const void* const* grad_ptrs, bool eight_bit, void* stream) {
    if (a.n_tiles == 0) return cudaSuccess;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return eight_bit ? dispatch_w<true>(a, grad_ptrs, s) : dispatch_w<false>(a, grad_ptrs, s);
}

int launch_muon_quantize(const MuonArgs& a, void* stream) {
    if (a.n_tiles == 0) return cudaSuccess;
    return launch_one<1, 1, Op::kQuantize, true>(a, nullptr, static_cast<cudaStream_t>(stream));
}

int launch_muon_dequantize(const MuonArgs& a, void* stream) {
    if (a.n_tiles == 0) return cudaSuccess;
    return launch_one<1, 1, Op::kDequantize, true>(a, nullptr, static_cast<cudaStream_t>(stream));
}

}  // namespace zr
