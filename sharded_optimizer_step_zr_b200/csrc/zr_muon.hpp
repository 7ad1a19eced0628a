// The Muon step's elementwise passes (zr_muon.cu).
#pragma once

#include <cstdint>

namespace zr {

constexpr int32_t kMuonTileElems = 2048;
constexpr int32_t kMuonBlock = 256;        // elements that share a scale of an 8-bit momentum

// Up to kMuonTileElems consecutive elements of one matrix, starting at a
// multiple of kMuonTileElems in it.
struct MuonTile {
    int64_t owned;     // first element in owned order
    int64_t update;    // first element in the workspace's fp32 update
    int64_t scale;     // first block's entry of the scales
    int32_t len;
    int32_t aligned;   // owned % 8 == 0: 16-byte accesses
};
static_assert(sizeof(MuonTile) == 32, "MuonTile is 32 bytes");

struct MuonArgs {
    const MuonTile* tiles;
    int32_t n_tiles;
    int32_t world_size;
    int32_t w_is_pow2;
    float inv_w;
    float mu;
    int32_t nesterov;
    float* momentum;         // fp32 state, or the conversions' fp32 side
    int8_t* codes;           // 8-bit state
    float* scales;
    float* update;
    double* partials;        // one per tile
};

// Fold, average, momentum (fp32, or 8-bit when `eight_bit`), the update and
// its sum of squares.  grad_ptrs: host array of W device pointers.
int launch_muon_momentum(const MuonArgs& a, const void* const* grad_ptrs, bool eight_bit, void* stream);
// momentum -> codes, scales, and back.
int launch_muon_quantize(const MuonArgs& a, void* stream);
int launch_muon_dequantize(const MuonArgs& a, void* stream);

}  // namespace zr
