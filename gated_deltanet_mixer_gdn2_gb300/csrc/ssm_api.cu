// ssm_api.cu -- the extern "C" entry points of the selective state-space scan: argument checks (all on the
// host, before anything is enqueued) and the choice of the kernel family.
#include <climits>

#include "ssm_common.cuh"

namespace gdn2 {
namespace {

bool dtype_known(gdn2_dtype dt) { return dt == GDN2_F32 || dt == GDN2_BF16; }

bool scan_shape_ok(int P, int N) { return P % 8 == 0 && P <= 256 && (N == 16 || N == 32 || N == 64 || N == 128 || N == 256); }

// Indices and grid dimensions: rows and units fit an int, (sequence, head) and (unit, head) planes their grids.
bool scan_sizes_ok(const ScanShape& sh) {
    return sh.seqs.rows() < (1LL << 30) && sh.seqs.units(32) < (1LL << 30) && sh.seqs.B <= 65535 && sh.H <= 32767;
}

gdn2_status scan_check(gdn2_path path, const ScanShape& sh) {
    if (!dtype_known(sh.dt) || (path != GDN2_PATH_AUTO && path != GDN2_PATH_SIMT && path != GDN2_PATH_TCGEN05))
        return GDN2_ERR_INVALID_ARG;
    if (sh.seqs.B < 0 || sh.seqs.T < 0 || sh.H <= 0 || sh.G <= 0 || sh.P <= 0 || sh.N <= 0 || sh.H % sh.G)
        return GDN2_ERR_INVALID_ARG;
    if (!scan_shape_ok(sh.P, sh.N) || !scan_sizes_ok(sh)) return GDN2_ERR_UNSUPPORTED;
    if (path == GDN2_PATH_TCGEN05 && !ssm_tc_shape(sh)) return GDN2_ERR_UNSUPPORTED;
    return GDN2_OK;
}

bool on_tensor_cores(gdn2_path path, const ScanShape& sh) { return path != GDN2_PATH_SIMT && ssm_tc_shape(sh); }

// Row stride of a token tensor of `width` dense elements: at least the width, rows on 16-byte boundaries.
gdn2_status row_check(const void* p, long long ld, long long width) {
    if (!p || ld < width) return GDN2_ERR_INVALID_ARG;
    if (ld >= (1LL << 31)) return GDN2_ERR_UNSUPPORTED;
    return aligned16(p) && ld % 8 == 0 ? GDN2_OK : GDN2_ERR_MISALIGNED;
}

const int kFakeOffset = 0;  // workspace sizes depend on whether the sequences are packed, not on the offsets

}  // namespace
}  // namespace gdn2

using namespace gdn2;

extern "C" {

size_t gdn2_ssm_chunk_fwd_workspace_size(gdn2_path path, int B, int T, int H, int G, int P, int N, int packed, gdn2_dtype dt) {
    const ScanShape sh{{packed ? &kFakeOffset : nullptr, B, T}, H, G, P, N, dt};
    if (scan_check(path, sh) != GDN2_OK || B == 0 || sh.seqs.rows() == 0) return 0;
    return on_tensor_cores(path, sh) ? ssm_tc_fwd_workspace(sh) : ssm_simt_fwd_workspace(sh);
}

size_t gdn2_ssm_backward_workspace_size(gdn2_path path, int B, int T, int H, int G, int P, int N, int packed, gdn2_dtype dt) {
    const ScanShape sh{{packed ? &kFakeOffset : nullptr, B, T}, H, G, P, N, dt};
    if (scan_check(path, sh) != GDN2_OK || B == 0 || sh.seqs.rows() == 0) return 0;
    return on_tensor_cores(path, sh) ? ssm_tc_bwd_workspace(sh) : ssm_simt_bwd_workspace(sh);
}

gdn2_status gdn2_ssm_chunk_fwd(gdn2_path path, const void* x, long long ld_x, const void* step, const void* g,
                               const void* bm, long long ld_b, const void* cm, long long ld_c, const float* d,
                               const float* initial_state, float* final_state, const int32_t* offsets, void* y, int B,
                               int T, int H, int G, int P, int N, gdn2_dtype dt, void* workspace, size_t ws_bytes,
                               void* stream) {
    const ScanShape sh{{offsets, B, T}, H, G, P, N, dt};
    gdn2_status st = scan_check(path, sh);
    if (st != GDN2_OK) return st;
    if ((initial_state && !aligned16(initial_state)) || (final_state && !aligned16(final_state)) || (d && !aligned_to(d, 4)) ||
        (offsets && !aligned_to(offsets, 4)))
        return GDN2_ERR_MISALIGNED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (B == 0) return GDN2_OK;
    if (sh.seqs.rows() == 0) {  // no tokens: the states stay
        const size_t bytes = sizeof(float) * (size_t)B * H * N * P;
        cudaError_t e = cudaSuccess;
        if (final_state && !initial_state) e = cudaMemsetAsync(final_state, 0, bytes, s);
        else if (final_state && final_state != initial_state)
            e = cudaMemcpyAsync(final_state, initial_state, bytes, cudaMemcpyDeviceToDevice, s);
        return e == cudaSuccess ? GDN2_OK : GDN2_ERR_CUDA;
    }
    if (!step || !g || !y) return GDN2_ERR_INVALID_ARG;
    if ((st = row_check(x, ld_x, (long long)H * P)) != GDN2_OK || (st = row_check(bm, ld_b, (long long)G * N)) != GDN2_OK ||
        (st = row_check(cm, ld_c, (long long)G * N)) != GDN2_OK)
        return st;
    const size_t esz = dt == GDN2_BF16 ? 2 : 4;
    if (!aligned_to(step, esz) || !aligned_to(g, esz) || !aligned16(y)) return GDN2_ERR_MISALIGNED;
    const size_t need = gdn2_ssm_chunk_fwd_workspace_size(path, B, T, H, G, P, N, offsets != nullptr, dt);
    if (need && (!workspace || ws_bytes < need)) return GDN2_ERR_WORKSPACE;
    if (need && !aligned16(workspace)) return GDN2_ERR_MISALIGNED;
    const ScanIn in{{x, ld_x}, {bm, ld_b}, {cm, ld_c}, step, g, d, initial_state};
    const cudaError_t e = on_tensor_cores(path, sh) ? launch_ssm_tc_fwd(sh, in, y, final_state, workspace, s, wait_limit_ns())
                                                    : launch_ssm_simt_fwd(sh, in, y, final_state, workspace, s);
    return e == cudaSuccess ? GDN2_OK : GDN2_ERR_CUDA;
}

gdn2_status gdn2_ssm_backward(gdn2_path path, const void* x, long long ld_x, const void* step, const void* g,
                              const void* bm, long long ld_b, const void* cm, long long ld_c, const float* d,
                              const float* initial_state, const void* d_y, long long ld_dy, const float* d_final_state,
                              const int32_t* offsets, void* dx, long long ld_dx, void* dstep, void* dg, void* dbm,
                              long long ld_db, void* dcm, long long ld_dc, float* dd, float* d_initial_state, int B, int T,
                              int H, int G, int P, int N, gdn2_dtype dt, void* workspace, size_t ws_bytes, void* stream) {
    const ScanShape sh{{offsets, B, T}, H, G, P, N, dt};
    gdn2_status st = scan_check(path, sh);
    if (st != GDN2_OK) return st;
    if ((initial_state && !aligned16(initial_state)) || (d_final_state && !aligned16(d_final_state)) ||
        (d_initial_state && !aligned16(d_initial_state)) || (d && !aligned_to(d, 4)) || (dd && !aligned_to(dd, 4)) ||
        (offsets && !aligned_to(offsets, 4)))
        return GDN2_ERR_MISALIGNED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (B == 0 || sh.seqs.rows() == 0) {  // no tokens: the state's gradient passes through
        const size_t bytes = sizeof(float) * (size_t)B * H * N * P;
        cudaError_t e = cudaSuccess;
        if (dd) e = cudaMemsetAsync(dd, 0, sizeof(float) * H, s);
        if (e == cudaSuccess && d_initial_state && bytes) {
            if (!d_final_state) e = cudaMemsetAsync(d_initial_state, 0, bytes, s);
            else if (d_final_state != d_initial_state)
                e = cudaMemcpyAsync(d_initial_state, d_final_state, bytes, cudaMemcpyDeviceToDevice, s);
        }
        return e == cudaSuccess ? GDN2_OK : GDN2_ERR_CUDA;
    }
    if (!step || !g || !dstep || !dg) return GDN2_ERR_INVALID_ARG;
    const struct { const void* p; long long ld, w; } rows[] = {
        {x, ld_x, (long long)H * P}, {bm, ld_b, (long long)G * N}, {cm, ld_c, (long long)G * N}, {d_y, ld_dy, (long long)H * P},
        {dx, ld_dx, (long long)H * P}, {dbm, ld_db, (long long)G * N}, {dcm, ld_dc, (long long)G * N}};
    for (const auto& r : rows)
        if ((st = row_check(r.p, r.ld, r.w)) != GDN2_OK) return st;
    const size_t esz = dt == GDN2_BF16 ? 2 : 4;
    if (!aligned_to(step, esz) || !aligned_to(g, esz) || !aligned_to(dstep, esz) || !aligned_to(dg, esz)) return GDN2_ERR_MISALIGNED;
    const size_t need = gdn2_ssm_backward_workspace_size(path, B, T, H, G, P, N, offsets != nullptr, dt);
    if (need && (!workspace || ws_bytes < need)) return GDN2_ERR_WORKSPACE;
    if (need && !aligned16(workspace)) return GDN2_ERR_MISALIGNED;
    const ScanIn in{{x, ld_x}, {bm, ld_b}, {cm, ld_c}, step, g, d, initial_state};
    const ScanGrads gr{{d_y, ld_dy}, d_final_state, {dx, ld_dx}, {dbm, ld_db}, {dcm, ld_dc}, dstep, dg, dd, d_initial_state};
    const cudaError_t e = on_tensor_cores(path, sh) ? launch_ssm_tc_bwd(sh, in, gr, workspace, s, wait_limit_ns())
                                                    : launch_ssm_simt_bwd(sh, in, gr, workspace, s);
    return e == cudaSuccess ? GDN2_OK : GDN2_ERR_CUDA;
}

}  // extern "C"
