// Newton-Schulz orthogonalisation of batches of matrices: the groups that
// the API layers (muon.cpp) describe and zr_newton.cu runs.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace zr {

// Tensor maps of a group's scratch.  The products' operands: boxes of 64
// columns x 64 or 128 rows, and two chunks of 64 columns x 64 rows.  An
// epilogue warp's share of X with its rounding error, of A and of B: 64
// columns x 32 rows, and the transposed shares of A and B.
struct NsMaps {
    CUtensorMap x_box[2], x_rows[2], x_chunks[2], gram_box, gram_rows, poly_box, poly_rows;
    CUtensorMap ex[2], egram, epoly, mgram, mpoly;
};

// Matrices of one shape: source, scratch and destination.  Gram matrices
// have the smaller extent g = min(m, n): X X^T for m <= n, X^T X otherwise.
struct NsGroup {
    int64_t batch = 0, m = 0, n = 0;

    // source: element (b, i, j) at src[b * src_batch + i * src_row + j]
    const void* src = nullptr;
    int32_t src_dtype = 0;                 // ZR_DTYPE_*
    int64_t src_row = 0, src_batch = 0;

    // destination of the last product: bf16 with strides, or the update of
    // the fp32 master weights at master_offsets[b] + i * n + j
    uint16_t* out = nullptr;
    int64_t out_row = 0, out_batch = 0;
    const int64_t* master_offsets = nullptr;   // device, batch entries
    const int64_t* param_offsets = nullptr;    // device, batch entries
    float step_size = 0.0f;

    // scratch (device)
    uint16_t *xh[2] = {nullptr, nullptr};  // X, fp16, rows of ld elements
    uint16_t *xl[2] = {nullptr, nullptr};  // its rounding error
    uint16_t *gram = nullptr, *poly = nullptr;   // A and B without their diagonals, fp16, rows of ldg elements
    float *gram_diag = nullptr, *poly_diag = nullptr;   // the diagonals, fp32
    double* partials = nullptr;            // sums of squares, n_partials per matrix
    int32_t n_partials = 0;
    const int32_t* first_partial = nullptr;   // device: batch + 1 entries, or NULL for b * n_partials
    float2* scale = nullptr;               // batch entries: X_0 = (src * x) * y, times kNsScaleX
    uint32_t* done = nullptr;              // batch + 1 words: finished shares of tiles, and a launch's abort word
    NsMaps maps;

    int64_t gram_dim() const { return m < n ? m : n; }
    int64_t ld() const { return (n + 63) / 64 * 64; }
    int64_t ldg() const { return (gram_dim() + 63) / 64 * 64; }
};

// Where the last product of the iteration goes.
struct NsApply {
    float* master = nullptr;               // NULL: bf16 to each group's out
    uint16_t* param_out = nullptr;
    uint16_t* const* targets = nullptr;    // device array of n_targets buffers, in place of param_out
    int32_t n_targets = 0;
    float decay = 1.0f;                    // 1 - lr * weight_decay
};

// Scratch of one group, in bytes: X twice with its rounding errors, A, B and
// their diagonals.
uint64_t ns_scratch_bytes(int64_t batch, int64_t m, int64_t n);
// The second X and its rounding error are first written after X_0 has been
// formed, so until then their place (4 bytes per element and more, matrices
// ns_source_pitch elements apart) can hold an fp32 source: its byte offset in
// the scratch.
uint64_t ns_source_offset(int64_t batch, int64_t m, int64_t n);
inline int64_t ns_source_pitch(int64_t m, int64_t n) { return (m * n + 7) / 8 * 8; }
// Points the group's scratch into `base` (ns_scratch_bytes, 256-byte
// aligned) and encodes its tensor maps.  Returns a cudaError_t.
int ns_bind_scratch(NsGroup& g, void* base);
// How many partial sums of squares launch_ns_sumsq writes for one matrix.
int64_t ns_partials_per_matrix(int64_t m, int64_t n);

// Sums of squares of every source matrix into partials (one CTA per piece),
// and *gave_up cleared.
int launch_ns_sumsq(const NsGroup& group, uint32_t* gave_up, void* stream);
// The scales 1 / (norm + eps) from the partials, X_0, then `steps` iterations, then the destination.  *gave_up (device) is
// set to 1 if a wait inside a kernel ran out.  Several groups only with `apply`.
int launch_ns_iterations(const NsGroup* groups, int32_t n_groups, int32_t steps, const float coeffs[3], double eps,
                         const NsApply& apply, const void* device_maps, uint32_t* gave_up, void* stream);
// What several groups' launches need in device memory (device_maps; 128-byte
// aligned), filled on the host for the current device; a single group needs none.
uint64_t ns_maps_bytes(int32_t n_groups);
int ns_fill_maps(const NsGroup* groups, int32_t n_groups, void* host);
// The same from the sources alone, in clusters that keep a matrix on the chip:
// for groups whose smaller extents are at most 128 and whose larger ones fit
// a cluster (ns_small says whether).  Nothing of the scratch is used.  With
// `clear`, *gave_up is cleared first.
bool ns_small(const NsGroup* groups, int32_t n_groups, bool apply);
int launch_ns_small(const NsGroup* groups, int32_t n_groups, int32_t steps, const float coeffs[3], double eps,
                    const NsApply& apply, uint32_t* gave_up, bool clear, void* stream);
// Whether the fp16 range of the scratch holds every iterate that the
// coefficients produce from singular values in [0, 1].
bool ns_coefficients_fit(const float coeffs[3], int32_t steps);
// Whether every tile count and offset of a shape fits the kernels' indices.
bool ns_shape_fits(int64_t batch, int64_t m, int64_t n);

}  // namespace zr
