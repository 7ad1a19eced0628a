// C ABI of the matrix optimizer (declared in include/zr.h): argument checks,
// the groups of equal shapes, the caller's workspace, and the launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "zr_internal.hpp"
#include "zr_muon.hpp"
#include "zr_newton.hpp"

namespace {

uint64_t align256(uint64_t x) { return (x + 255) & ~uint64_t(255); }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
zr_status cuda_status(int e) { return e == cudaSuccess ? ZR_OK : ZR_ERR_CUDA; }

zr_status current_b200(int* dev) {
    int major = 0;
    if (cudaGetDevice(dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *dev) != cudaSuccess)
        return ZR_ERR_CUDA;
    return major == 10 ? ZR_OK : ZR_ERR_UNSUPPORTED;
}

bool iteration_ok(const zr_newton_schulz& ns) {
    if (ns.steps < 1 || ns.steps > 32) return false;
    if (!(ns.eps >= 1e-30f && ns.eps <= 1.0f)) return false;
    const float k[3] = {ns.a, ns.b, ns.c};
    return zr::ns_coefficients_fit(k, ns.steps);
}

// Whether the result would certainly be written over a source that is still
// read: the two start at one address, or are both without gaps and meet.
// Elements of 16 bits replaced one by one are not (a matrix is read whole
// before its result is written).
bool overwrites(const void* x, uint64_t x_size, int64_t x_row, int64_t x_batch, const void* out, int64_t out_row,
                int64_t out_batch, int64_t batch, int64_t m, int64_t n) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(out);
    if (a == b) return x_size != 2 || x_row != out_row || x_batch != out_batch;
    const bool dense = x_row == n && out_row == n && (batch == 1 || (x_batch == m * n && out_batch == m * n));
    const uint64_t count = static_cast<uint64_t>(batch) * m * n;
    return dense && a < b + 2 * count && b < a + x_size * count;
}

// A matrix of this rank, in owned order.
struct Matrix {
    int64_t owned, global;    // first element
    int64_t scale;            // first block's scale
    int32_t group, slot;
};

}  // namespace

struct zr_muon {
    const zr_plan* plan = nullptr;
    zr_muon_params hp{};
    int32_t format = ZR_MOMENTUM_F32;
    std::vector<zr::NsGroup> groups;          // one per shape, in order of first appearance
    std::vector<Matrix> matrices;             // by group, then slot
    int64_t n_scales = 0;
    std::vector<zr::MuonTile> tiles;          // in the order of matrices
    std::vector<int32_t> first_tile;          // per matrix, and the end
    std::vector<int64_t> owned_offsets, global_offsets;   // per matrix

    // workspace regions
    uint64_t at_status = 0, at_tiles = 0, at_first = 0, at_owned = 0, at_global = 0, at_scale = 0, at_partials = 0, at_maps = 0,
             total = 0;
    std::vector<uint64_t> at_group;

    int device = -1;
    char* d_workspace = nullptr;
};

namespace {

void lay_out(zr_muon& u) {
    uint64_t off = 0;
    auto take = [&](uint64_t& at, uint64_t bytes) {
        at = off;
        off = align256(off + bytes);
    };
    const uint64_t n = u.matrices.size();
    take(u.at_status, sizeof(uint32_t));
    take(u.at_tiles, sizeof(zr::MuonTile) * u.tiles.size());
    take(u.at_first, sizeof(int32_t) * (n + 1));
    take(u.at_owned, sizeof(int64_t) * n);
    take(u.at_global, sizeof(int64_t) * n);
    take(u.at_scale, sizeof(float2) * n);
    take(u.at_partials, sizeof(double) * u.tiles.size());
    take(u.at_maps, zr::ns_maps_bytes(static_cast<int32_t>(u.groups.size())));
    u.at_group.clear();
    for (const zr::NsGroup& g : u.groups) {
        uint64_t at;
        take(at, zr::ns_scratch_bytes(g.batch, g.m, g.n));
        u.at_group.push_back(at);
    }
    u.total = std::max<uint64_t>(off, 256);
}

// Groups, matrices, tiles and the workspace's layout from the plan.
zr_status build(zr_muon& u) {
    const zr_plan& p = *u.plan;
    struct Owned { int64_t owned, global, count, m, n; };
    std::vector<Owned> mine;
    int64_t owned = 0;
    for (int32_t t = 0; t < p.n_tensors; ++t) {
        if (p.numel[t] == 0) continue;
        if (p.rows[t] < 0) return ZR_ERR_INVALID_ARG;
        const bool own = p.mode != ZR_PARTITION_WHOLE_TENSOR || p.tensor_owner[t] == p.rank;
        if (!own) continue;
        const int64_t size = p.rows[t] * p.cols[t];
        mine.push_back({owned, p.goff[t], p.numel[t] / size, p.rows[t], p.cols[t]});
        owned += p.numel[t];
    }
    if (owned != p.owned_numel()) return ZR_ERR_INVALID_ARG;
    std::vector<std::vector<Matrix>> by_group;
    for (const Owned& t : mine) {
        size_t gi = 0;
        while (gi < u.groups.size() && !(u.groups[gi].m == t.m && u.groups[gi].n == t.n)) ++gi;
        if (gi == u.groups.size()) {
            zr::NsGroup g;
            g.m = t.m;
            g.n = t.n;
            u.groups.push_back(g);
            by_group.emplace_back();
        }
        for (int64_t b = 0; b < t.count; ++b) {
            Matrix x;
            x.owned = t.owned + b * t.m * t.n;
            x.global = t.global + b * t.m * t.n;
            x.scale = u.n_scales;
            u.n_scales += (t.m * t.n + zr::kMuonBlock - 1) / zr::kMuonBlock;
            x.group = static_cast<int32_t>(gi);
            x.slot = static_cast<int32_t>(by_group[gi].size());
            by_group[gi].push_back(x);
            if (by_group[gi].size() > (1u << 24)) return ZR_ERR_UNSUPPORTED;
        }
    }
    for (size_t gi = 0; gi < u.groups.size(); ++gi) {
        zr::NsGroup& g = u.groups[gi];
        g.batch = static_cast<int64_t>(by_group[gi].size());
        if (!zr::ns_shape_fits(g.batch, g.m, g.n)) return ZR_ERR_UNSUPPORTED;
        u.matrices.insert(u.matrices.end(), by_group[gi].begin(), by_group[gi].end());
    }
    int64_t tiles = 0;
    for (const Matrix& x : u.matrices) {
        const zr::NsGroup& g = u.groups[x.group];
        tiles += (g.m * g.n + zr::kMuonTileElems - 1) / zr::kMuonTileElems;
    }
    if (tiles > 0x7FFFFFFF || u.matrices.size() > 0x7FFFFFFFu) return ZR_ERR_UNSUPPORTED;
    u.tiles.reserve(tiles);
    for (const Matrix& x : u.matrices) {
        const zr::NsGroup& g = u.groups[x.group];
        const int64_t size = g.m * g.n;
        u.first_tile.push_back(static_cast<int32_t>(u.tiles.size()));
        u.owned_offsets.push_back(x.owned);
        u.global_offsets.push_back(x.global);
        for (int64_t e = 0; e < size; e += zr::kMuonTileElems) {
            zr::MuonTile t;
            t.owned = x.owned + e;
            t.update = 0;      // with the group's place, below
            t.scale = x.scale + e / zr::kMuonBlock;
            t.len = static_cast<int32_t>(std::min<int64_t>(zr::kMuonTileElems, size - e));
            t.aligned = t.owned % 8 == 0 ? 1 : 0;
            u.tiles.push_back(t);
        }
    }
    u.first_tile.push_back(static_cast<int32_t>(u.tiles.size()));
    lay_out(u);
    size_t at = 0;
    for (const Matrix& x : u.matrices) {
        const zr::NsGroup& g = u.groups[x.group];
        const uint64_t base = u.at_group[x.group] + zr::ns_source_offset(g.batch, g.m, g.n);
        const int64_t first = static_cast<int64_t>(base / sizeof(float)) + x.slot * zr::ns_source_pitch(g.m, g.n);
        for (int64_t e = 0; e < g.m * g.n; e += zr::kMuonTileElems) u.tiles[at++].update = first + e;
    }
    return ZR_OK;
}

bool params_ok(const zr_muon_params& hp) {
    return std::isfinite(hp.lr) && hp.lr >= 0.0f && hp.momentum >= 0.0f && hp.momentum < 1.0f &&
           std::isfinite(hp.weight_decay) && hp.weight_decay >= 0.0f &&
           (hp.scale == ZR_MUON_SCALE_SPECTRAL || hp.scale == ZR_MUON_SCALE_RMS) && iteration_ok(hp.ns);
}

double update_scale(const zr_muon_params& hp, int64_t m, int64_t n) {
    const double r = static_cast<double>(m), c = static_cast<double>(n);
    return hp.scale == ZR_MUON_SCALE_RMS ? 0.2 * std::sqrt(std::max(r, c)) : std::sqrt(std::max(1.0, r / c));
}

zr_status check_bound(const zr_muon* u) {
    if (!u) return ZR_ERR_INVALID_ARG;
    if (!u->d_workspace) return ZR_ERR_NO_WORKSPACE;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return ZR_ERR_CUDA;
    return dev == u->device && dev == u->plan->device ? ZR_OK : ZR_ERR_INVALID_ARG;
}

zr::MuonArgs base_args(const zr_muon* u) {
    zr::MuonArgs a{};
    a.tiles = reinterpret_cast<const zr::MuonTile*>(u->d_workspace + u->at_tiles);
    a.n_tiles = static_cast<int32_t>(u->tiles.size());
    zr::set_world_size(a, u->plan->world_size);
    a.mu = u->hp.momentum;
    a.nesterov = u->hp.nesterov;
    a.update = reinterpret_cast<float*>(u->d_workspace);
    a.partials = reinterpret_cast<double*>(u->d_workspace + u->at_partials);
    return a;
}

}  // namespace

extern "C" {

zr_status zr_orthogonalize_workspace_bytes(int64_t batch, int64_t m, int64_t n, uint64_t* bytes) {
    if (!bytes || batch < 0 || m < 0 || n < 0) return ZR_ERR_INVALID_ARG;
    *bytes = 256;
    if (batch == 0 || m == 0 || n == 0) return ZR_OK;
    if (!zr::ns_shape_fits(batch, m, n)) return ZR_ERR_UNSUPPORTED;
    *bytes = 256 + align256(sizeof(float2) * static_cast<uint64_t>(batch)) +
             align256(sizeof(double) * static_cast<uint64_t>(batch * zr::ns_partials_per_matrix(m, n))) +
             zr::ns_scratch_bytes(batch, m, n);
    return ZR_OK;
}

zr_status zr_orthogonalize(const void* x, int32_t dtype, int64_t batch, int64_t m, int64_t n, int64_t x_batch_stride,
                           int64_t x_row_stride, void* out, int64_t out_batch_stride, int64_t out_row_stride,
                           const zr_newton_schulz* ns, void* d_ws, uint64_t ws_bytes, zr_stream_t stream) {
    if (!ns || batch < 0 || m < 0 || n < 0 || !iteration_ok(*ns)) return ZR_ERR_INVALID_ARG;
    if (dtype != ZR_DTYPE_F32 && dtype != ZR_DTYPE_BF16 && dtype != ZR_DTYPE_F16) return ZR_ERR_INVALID_ARG;
    if (batch == 0 || m == 0 || n == 0) return ZR_OK;
    uint64_t need = 0;
    zr_status st = zr_orthogonalize_workspace_bytes(batch, m, n, &need);
    if (st != ZR_OK) return st;
    if (m == 1) x_row_stride = out_row_stride = n;
    if (batch == 1) {
        x_batch_stride = 0;
        out_batch_stride = 0;
    }
    constexpr int64_t kMostStride = int64_t(1) << 48;      // with at most 2^24 rows and matrices: no overflow below
    if (x_batch_stride < 0 || x_row_stride < 0 || out_row_stride < n || x_batch_stride > (kMostStride >> 10) ||
        x_row_stride > (kMostStride >> 10) || out_batch_stride > (kMostStride >> 10) ||
        out_row_stride > (kMostStride >> 10))
        return ZR_ERR_INVALID_ARG;
    if (batch > 1 && out_batch_stride < (m - 1) * out_row_stride + n) return ZR_ERR_INVALID_ARG;
    if (!x || !out) return ZR_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(x) % (dtype == ZR_DTYPE_F32 ? 4 : 2) != 0 || reinterpret_cast<uintptr_t>(out) % 2 != 0)
        return ZR_ERR_ALIGNMENT;
    if (!d_ws) return ZR_ERR_NO_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(d_ws) & 255u) != 0) return ZR_ERR_ALIGNMENT;
    if (ws_bytes < need) return ZR_ERR_NO_WORKSPACE;
    if (overwrites(x, dtype == ZR_DTYPE_F32 ? 4 : 2, x_row_stride, x_batch_stride, out, out_row_stride, out_batch_stride,
                   batch, m, n))
        return ZR_ERR_INVALID_ARG;
    int dev = 0;
    if ((st = current_b200(&dev)) != ZR_OK) return st;

    char* base = static_cast<char*>(d_ws);
    zr::NsGroup g;
    g.batch = batch;
    g.m = m;
    g.n = n;
    g.src = x;
    g.src_dtype = dtype;
    g.src_row = x_row_stride;
    g.src_batch = x_batch_stride;
    g.out = static_cast<uint16_t*>(out);
    g.out_row = out_row_stride;
    g.out_batch = out_batch_stride;
    g.scale = reinterpret_cast<float2*>(base + 256);
    const uint64_t at_partials = 256 + align256(sizeof(float2) * static_cast<uint64_t>(batch));
    g.n_partials = static_cast<int32_t>(zr::ns_partials_per_matrix(m, n));
    g.partials = reinterpret_cast<double*>(base + at_partials);
    const float coeffs[3] = {ns->a, ns->b, ns->c};
    uint32_t* gave_up = reinterpret_cast<uint32_t*>(base);
    if (zr::ns_small(&g, 1, false))
        return cuda_status(zr::launch_ns_small(&g, 1, ns->steps, coeffs, ns->eps, zr::NsApply(), gave_up, true,
                                              stream));
    if (zr::ns_bind_scratch(g, base + need - zr::ns_scratch_bytes(batch, m, n)) != cudaSuccess) return ZR_ERR_CUDA;
    int e = zr::launch_ns_sumsq(g, gave_up, stream);
    if (e == cudaSuccess) e = zr::launch_ns_iterations(&g, 1, ns->steps, coeffs, ns->eps, zr::NsApply(), nullptr, gave_up, stream);
    return cuda_status(e);
}

zr_status zr_muon_create(const zr_plan* plan, const zr_muon_params* params, int32_t format, zr_muon** out) {
    if (!out) return ZR_ERR_INVALID_ARG;
    *out = nullptr;
    if (!plan || !params || !params_ok(*params)) return ZR_ERR_INVALID_ARG;
    if (format != ZR_MOMENTUM_F32 && format != ZR_MOMENTUM_INT8) return ZR_ERR_INVALID_ARG;
    if (plan->mode != ZR_PARTITION_WHOLE_TENSOR && plan->world_size > 1) return ZR_ERR_UNSUPPORTED;
    if (plan->clip_enabled()) return ZR_ERR_UNSUPPORTED;
    zr_muon* u = new (std::nothrow) zr_muon();
    if (!u) return ZR_ERR_INVALID_ARG;
    u->plan = plan;
    u->hp = *params;
    u->format = format;
    zr_status st;
    try {
        st = build(*u);
    } catch (...) {
        st = ZR_ERR_INVALID_ARG;
    }
    if (st != ZR_OK) {
        delete u;
        return st;
    }
    *out = u;
    return ZR_OK;
}

void zr_muon_destroy(zr_muon* u) { delete u; }

zr_status zr_muon_set_params(zr_muon* u, const zr_muon_params* params) {
    if (!u || !params || !params_ok(*params)) return ZR_ERR_INVALID_ARG;
    u->hp = *params;
    return ZR_OK;
}

zr_status zr_muon_scales(const zr_muon* u, int64_t* n) {
    if (!u || !n) return ZR_ERR_INVALID_ARG;
    *n = u->n_scales;
    return ZR_OK;
}

zr_status zr_muon_workspace_bytes(const zr_muon* u, uint64_t* bytes) {
    if (!u || !bytes) return ZR_ERR_INVALID_ARG;
    *bytes = u->total;
    return ZR_OK;
}

zr_status zr_muon_set_workspace(zr_muon* u, void* d_ws, uint64_t bytes, zr_stream_t stream) {
    if (!u || !d_ws) return ZR_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(d_ws) & 255u) != 0) return ZR_ERR_ALIGNMENT;
    if (bytes < u->total) return ZR_ERR_NO_WORKSPACE;
    if (!u->plan->d_workspace) return ZR_ERR_NO_WORKSPACE;
    int dev = 0;
    const zr_status st = current_b200(&dev);
    if (st != ZR_OK) return st;
    if (dev != u->plan->device) return ZR_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // A graph would read the host's tables again at every replay, long after
    // they changed or went away.
    cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &capture) != cudaSuccess) return ZR_ERR_CUDA;
    if (capture != cudaStreamCaptureStatusNone) return ZR_ERR_UNSUPPORTED;
    u->d_workspace = nullptr;      // until all of it is in place
    char* base = static_cast<char*>(d_ws);
    auto up = [&](uint64_t at, const void* src, size_t n) {
        return n == 0 || cudaMemcpyAsync(base + at, src, n, cudaMemcpyHostToDevice, s) == cudaSuccess;
    };
    if (!up(u->at_tiles, u->tiles.data(), sizeof(zr::MuonTile) * u->tiles.size()) ||
        !up(u->at_first, u->first_tile.data(), sizeof(int32_t) * u->first_tile.size()) ||
        !up(u->at_owned, u->owned_offsets.data(), sizeof(int64_t) * u->owned_offsets.size()) ||
        !up(u->at_global, u->global_offsets.data(), sizeof(int64_t) * u->global_offsets.size()) ||
        cudaMemsetAsync(base + u->at_status, 0, sizeof(uint32_t), s) != cudaSuccess)
        return ZR_ERR_CUDA;
    int64_t first = 0;
    for (size_t gi = 0; gi < u->groups.size(); ++gi) {
        zr::NsGroup& g = u->groups[gi];
        char* scratch = base + u->at_group[gi];
        if (zr::ns_bind_scratch(g, scratch) != cudaSuccess) return ZR_ERR_CUDA;
        g.src = scratch + zr::ns_source_offset(g.batch, g.m, g.n);
        g.src_dtype = ZR_DTYPE_F32;
        g.src_row = g.n;
        g.src_batch = zr::ns_source_pitch(g.m, g.n);
        g.n_partials = static_cast<int32_t>((g.m * g.n + zr::kMuonTileElems - 1) / zr::kMuonTileElems);
        g.scale = reinterpret_cast<float2*>(base + u->at_scale) + first;
        g.partials = reinterpret_cast<double*>(base + u->at_partials);
        g.first_partial = reinterpret_cast<const int32_t*>(base + u->at_first) + first;
        g.master_offsets = reinterpret_cast<const int64_t*>(base + u->at_owned) + first;
        first += g.batch;
    }
    std::vector<char> maps;
    try {
        maps.resize(zr::ns_maps_bytes(static_cast<int32_t>(u->groups.size())));
    } catch (...) {
        return ZR_ERR_INVALID_ARG;
    }
    if (!maps.empty() && (zr::ns_fill_maps(u->groups.data(), static_cast<int32_t>(u->groups.size()), maps.data()) != cudaSuccess ||
                          !up(u->at_maps, maps.data(), maps.size())))
        return ZR_ERR_CUDA;
    u->device = dev;
    u->d_workspace = base;
    return ZR_OK;
}

zr_status zr_muon_step(const zr_muon* u, const void* const* grad_ptrs, float* master, void* momentum, float* scales,
                       void* param_out, zr_stream_t stream) {
    zr_status st = check_bound(u);
    if (st != ZR_OK) return st;
    const zr_plan* p = u->plan;
    if (p->owned_numel() == 0) return ZR_OK;
    if (!grad_ptrs) return ZR_ERR_INVALID_ARG;
    for (int32_t w = 0; w < p->world_size; ++w) {
        if (!grad_ptrs[w]) return ZR_ERR_INVALID_ARG;
        if (!aligned16(grad_ptrs[w])) return ZR_ERR_ALIGNMENT;
    }
    const bool eight = u->format == ZR_MOMENTUM_INT8;
    if (!master || !momentum || (eight && !scales) || (p->n_gather_targets == 0 && !param_out)) return ZR_ERR_INVALID_ARG;
    if (!aligned16(master) || !aligned16(momentum) || (eight && !aligned16(scales)) || !aligned16(param_out))
        return ZR_ERR_ALIGNMENT;

    zr::MuonArgs a = base_args(u);
    if (eight) {
        a.codes = static_cast<int8_t*>(momentum);
        a.scales = scales;
    } else {
        a.momentum = static_cast<float*>(momentum);
    }
    // A copy of the groups: the step's parameters and the plan's current
    // layout go into it.
    std::vector<zr::NsGroup> groups;
    try {
        groups = u->groups;
    } catch (...) {
        return ZR_ERR_INVALID_ARG;
    }
    const uint64_t at_param = p->param_layout == ZR_PARAMS_OWNED ? u->at_owned : u->at_global;
    int64_t first = 0;
    for (zr::NsGroup& g : groups) {
        g.param_offsets = reinterpret_cast<const int64_t*>(u->d_workspace + at_param) + first;
        g.step_size = static_cast<float>(static_cast<double>(u->hp.lr) * update_scale(u->hp, g.m, g.n));
        first += g.batch;
    }
    zr::NsApply apply;
    apply.master = master;
    apply.param_out = static_cast<uint16_t*>(param_out);
    apply.targets = p->d_gather_targets;
    apply.n_targets = p->n_gather_targets;
    apply.decay = static_cast<float>(1.0 - static_cast<double>(u->hp.lr) * static_cast<double>(u->hp.weight_decay));
    const int32_t n = static_cast<int32_t>(groups.size());
    int e = zr::launch_muon_momentum(a, grad_ptrs, eight, stream);
    if (e != cudaSuccess) return ZR_ERR_CUDA;
    const float coeffs[3] = {u->hp.ns.a, u->hp.ns.b, u->hp.ns.c};
    uint32_t* gave_up = reinterpret_cast<uint32_t*>(u->d_workspace + u->at_status);
    // Small matrices beside large ones cost the persistent kernel nothing:
    // they run while the large ones' products wait for one another.
    if (zr::ns_small(groups.data(), n, true))
        return cuda_status(zr::launch_ns_small(groups.data(), n, u->hp.ns.steps, coeffs, u->hp.ns.eps, apply, gave_up,
                                              false, stream));
    e = zr::launch_ns_iterations(groups.data(), n, u->hp.ns.steps, coeffs, u->hp.ns.eps, apply, u->d_workspace + u->at_maps, gave_up,
                                     stream);
    return cuda_status(e);
}

static zr_status convert(const zr_muon* u, float* momentum, void* codes, float* scales, bool quantize,
                         zr_stream_t stream) {
    const zr_status st = check_bound(u);
    if (st != ZR_OK) return st;
    if (u->plan->owned_numel() == 0) return ZR_OK;
    if (!momentum || !codes || !scales) return ZR_ERR_INVALID_ARG;
    if (!aligned16(momentum) || !aligned16(codes) || !aligned16(scales)) return ZR_ERR_ALIGNMENT;
    zr::MuonArgs a = base_args(u);
    a.momentum = momentum;
    a.codes = static_cast<int8_t*>(codes);
    a.scales = scales;
    return cuda_status(quantize ? zr::launch_muon_quantize(a, stream) : zr::launch_muon_dequantize(a, stream));
}

zr_status zr_muon_quantize_momentum(const zr_muon* u, const float* momentum, void* codes, float* scales,
                                    zr_stream_t stream) {
    return convert(u, const_cast<float*>(momentum), codes, scales, true, stream);
}

zr_status zr_muon_dequantize_momentum(const zr_muon* u, const void* codes, const float* scales, float* momentum,
                                      zr_stream_t stream) {
    return convert(u, momentum, const_cast<void*>(codes), const_cast<float*>(scales), false, stream);
}

zr_status zr_muon_check_result(const zr_muon* u, int32_t* gave_up, zr_stream_t stream) {
    if (!gave_up) return ZR_ERR_INVALID_ARG;
    const zr_status st = check_bound(u);
    if (st != ZR_OK) return st;
    uint32_t word = 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (cudaMemcpyAsync(&word, u->d_workspace + u->at_status, sizeof word, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return ZR_ERR_CUDA;
    *gave_up = word != 0 ? 1 : 0;
    return ZR_OK;
}

}  // extern "C"
