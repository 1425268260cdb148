// block_norm.cu -- the residual stream around a block in one pass per direction:
//     t = x silu(z),  p = post t / rms_group(t),  r = residual + scale p,  n = pre r / rms(r)
// Each of the gate, the norm after the block, the residual, its scale and the norm before the next block
// may be absent. Rows are independent; every row is read once and written once, so HBM bounds it.
#include <initializer_list>

#include "ssm_common.cuh"

namespace gdn2 {
namespace {

constexpr int kMaxD = 8192;

struct NormArgs {
    const float *post, *scale, *pre;
    long long rows;
    int d, groups;
    float eps;
};

// Sum over the block; the same value in every thread. `red` holds one float per warp.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    const int warps = blockDim.x >> 5;
    __syncthreads();  // earlier readers of red are done
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    for (int w = 0; w < warps; ++w) s += red[w];
    return s;
}

// Sums over each group of 8-element vectors: vec[] holds every vector's part, out[] the groups' sums.
__device__ __forceinline__ void group_sums(float* vec, float* out, int nvec, int groups) {
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5, per = nvec / groups;
    for (int g = warp; g < groups; g += warps) {
        float v = 0.f;
        for (int i = lane; i < per; i += 32) v += vec[g * per + i];
#pragma unroll
        for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        if (lane == 0) out[g] = v;
    }
    __syncthreads();
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) { Vec8<T>::load(p, x); }

__device__ __forceinline__ void weights8(const float* w, int c, bool in, float (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = w && in ? __ldg(w + c + e) : 1.f;
}

// One row per block and trip, VPT vectors of eight elements per thread; the weights stay in registers
// over the block's rows.
template <typename T, int VPT>
__global__ void __launch_bounds__(512)
    norm_kernel(NormArgs a, const T* __restrict__ x, const T* __restrict__ z, const T* __restrict__ residual, T* __restrict__ r_out,
                T* __restrict__ n_out) {
    __shared__ float red[32], vec[kMaxD / 8], gsum[kMaxD / 8];
    const int tid = threadIdx.x, nvec = a.d / 8;
    float post[VPT][8], scale[VPT][8], pre[VPT][8];
    bool in[VPT];
    int group[VPT];
#pragma unroll
    for (int m = 0; m < VPT; ++m) {
        const int i = tid + m * blockDim.x;
        in[m] = i < nvec;
        group[m] = in[m] ? i / (nvec / a.groups) : 0;
        weights8(a.post, 8 * i, in[m], post[m]);
        weights8(a.scale, 8 * i, in[m], scale[m]);
        weights8(a.pre, 8 * i, in[m], pre[m]);
    }
    const float inv_width = static_cast<float>(a.groups) / a.d;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const size_t base = static_cast<size_t>(row) * a.d;
        float t[VPT][8], res[VPT][8];
        float ss = 0.f;
#pragma unroll
        for (int m = 0; m < VPT; ++m) {
            const size_t at = base + 8 * (tid + m * static_cast<int>(blockDim.x));
#pragma unroll
            for (int e = 0; e < 8; ++e) t[m][e] = res[m][e] = 0.f;
            if (!in[m]) continue;
            load8(x + at, t[m]);
            if (residual) load8(residual + at, res[m]);
            if (z) {
                float zz[8];
                load8(z + at, zz);
#pragma unroll
                for (int e = 0; e < 8; ++e) t[m][e] *= zz[e] * ssm_sigmoid(zz[e]);
            }
            float v = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) v = fmaf(t[m][e], t[m][e], v);
            ss += v;
            if (a.post && a.groups > 1) vec[tid + m * blockDim.x] = v;
        }
        if (a.post) {
            float all = 0.f;
            if (a.groups > 1) group_sums(vec, gsum, nvec, a.groups);
            else all = block_sum(ss, red);
#pragma unroll
            for (int m = 0; m < VPT; ++m) {
                const float inv = rsqrtf(fmaf(a.groups > 1 ? gsum[group[m]] : all, inv_width, a.eps));
#pragma unroll
                for (int e = 0; e < 8; ++e) t[m][e] *= inv * post[m][e];
            }
        }
        float rr = 0.f;
#pragma unroll
        for (int m = 0; m < VPT; ++m) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                t[m][e] = fmaf(t[m][e], scale[m][e], res[m][e]);
                rr = fmaf(t[m][e], t[m][e], rr);
            }
            if (r_out && in[m]) Vec8<T>::store(r_out + base + 8 * (tid + m * static_cast<int>(blockDim.x)), t[m]);
        }
        if (n_out) {
            const float inv = rsqrtf(block_sum(rr, red) / a.d + a.eps);
#pragma unroll
            for (int m = 0; m < VPT; ++m) {
                if (!in[m]) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e) t[m][e] *= inv * pre[m][e];
                Vec8<T>::store(n_out + base + 8 * (tid + m * static_cast<int>(blockDim.x)), t[m]);
            }
        }
    }
}

struct NormGradArgs {
    NormArgs n;
    float* part;  // [blocks][3][d]: dpost, dscale, dpre
};

// The forward's row again, then backwards through it: with nh = r / rms(r) and th = t / rms_group(t),
//     dr = d_r + (k - nh mean(k nh)) / rms(r),    k = d_n pre
//     dt = (q - th mean_group(q th)) / rms_group(t), q = dr scale post
// dx = dt silu(z), dz = dt x silu'(z); the parameters' sums stay in registers over the block's rows.
template <typename T, int VPT, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads)
    norm_grad_kernel(NormGradArgs ga, const T* __restrict__ x, const T* __restrict__ z, const T* __restrict__ residual,
                     const T* __restrict__ d_r, const T* __restrict__ d_n, T* __restrict__ dx, T* __restrict__ dz,
                     T* __restrict__ dres) {
    const NormArgs& a = ga.n;
    __shared__ float red[32], vec[kMaxD / 8], gsum[kMaxD / 8];
    const int tid = threadIdx.x, nvec = a.d / 8;
    float apost[VPT][8] = {}, ascale[VPT][8] = {}, apre[VPT][8] = {};
    bool in[VPT];
    int group[VPT];
#pragma unroll
    for (int m = 0; m < VPT; ++m) {
        const int i = tid + m * blockDim.x;
        in[m] = i < nvec;
        group[m] = in[m] ? i / (nvec / a.groups) : 0;
    }
    const float inv_width = static_cast<float>(a.groups) / a.d, inv_d = 1.f / a.d;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const size_t base = static_cast<size_t>(row) * a.d;
        float xv[VPT][8], zv[VPT][8], t[VPT][8], r[VPT][8], dr[VPT][8], k[VPT][8], inv_t[VPT];
        float ss = 0.f;
#pragma unroll
        for (int m = 0; m < VPT; ++m) {
            const size_t at = base + 8 * (tid + m * static_cast<int>(blockDim.x));
#pragma unroll
            for (int e = 0; e < 8; ++e) xv[m][e] = zv[m][e] = r[m][e] = dr[m][e] = k[m][e] = 0.f;
            if (in[m]) {
                load8(x + at, xv[m]);
                if (z) load8(z + at, zv[m]);
                if (residual) load8(residual + at, r[m]);
                if (d_r) load8(d_r + at, dr[m]);
                if (d_n) load8(d_n + at, k[m]);
            }
            float v = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                t[m][e] = z ? xv[m][e] * zv[m][e] * ssm_sigmoid(zv[m][e]) : xv[m][e];
                v = fmaf(t[m][e], t[m][e], v);
            }
            ss += v;
            inv_t[m] = 1.f;
            if (a.post && a.groups > 1 && in[m]) vec[tid + m * blockDim.x] = v;
        }
        if (a.post) {
            float all = 0.f;
            if (a.groups > 1) group_sums(vec, gsum, nvec, a.groups);
            else all = block_sum(ss, red);
#pragma unroll
            for (int m = 0; m < VPT; ++m) inv_t[m] = rsqrtf(fmaf(a.groups > 1 ? gsum[group[m]] : all, inv_width, a.eps));
        }
        float rr = 0.f, kr = 0.f;
#pragma unroll
        for (int m = 0; m < VPT; ++m) {
            float post[8], scale[8], pre[8];
            const int c = 8 * (tid + m * static_cast<int>(blockDim.x));
            weights8(a.post, c, in[m], post);
            weights8(a.scale, c, in[m], scale);
            weights8(a.pre, c, in[m], pre);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                r[m][e] = fmaf(t[m][e] * inv_t[m] * post[e], scale[e], r[m][e]);
                rr = fmaf(r[m][e], r[m][e], rr);
                kr = fmaf(k[m][e] * pre[e], r[m][e], kr);
            }
        }
        if (d_n) {
            const float inv = rsqrtf(fmaf(block_sum(rr, red), inv_d, a.eps));
            const float mean = block_sum(kr, red) * inv * inv_d;  // mean(k nh)
#pragma unroll
            for (int m = 0; m < VPT; ++m) {
                float pre[8];
                weights8(a.pre, 8 * (tid + m * static_cast<int>(blockDim.x)), in[m], pre);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float nh = r[m][e] * inv;
                    apre[m][e] = fmaf(k[m][e], nh, apre[m][e]);
                    dr[m][e] = fmaf(inv, fmaf(-nh, mean, k[m][e] * pre[e]), dr[m][e]);
                }
            }
        }
        float qs = 0.f;
#pragma unroll
        for (int m = 0; m < VPT; ++m) {
            float post[8], scale[8];
            const int c = 8 * (tid + m * static_cast<int>(blockDim.x));
            weights8(a.post, c, in[m], post);
            weights8(a.scale, c, in[m], scale);
            if (dres && in[m]) Vec8<T>::store(dres + base + c, dr[m]);
            float v = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float th = t[m][e] * inv_t[m];
                ascale[m][e] = fmaf(dr[m][e], th * post[e], ascale[m][e]);
                const float dp = dr[m][e] * scale[e];
                apost[m][e] = fmaf(dp, th, apost[m][e]);
                k[m][e] = dp * post[e];
                v = fmaf(k[m][e], th, v);
            }
            qs += v;
            if (a.post && a.groups > 1 && in[m]) vec[tid + m * blockDim.x] = v;
        }
        float all = 0.f;
        if (a.post) {
            if (a.groups > 1) group_sums(vec, gsum, nvec, a.groups);
            else all = block_sum(qs, red);
        }
#pragma unroll
        for (int m = 0; m < VPT; ++m) {
            if (!in[m]) continue;
            const size_t at = base + 8 * (tid + m * static_cast<int>(blockDim.x));
            const float mean = a.post ? (a.groups > 1 ? gsum[group[m]] : all) * inv_width : 0.f;
            float dzv[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float th = t[m][e] * inv_t[m];
                float dt = a.post ? inv_t[m] * fmaf(-th, mean, k[m][e]) : k[m][e];
                if (z) {
                    const float sg = ssm_sigmoid(zv[m][e]);
                    dzv[e] = dt * xv[m][e] * sg * fmaf(zv[m][e], 1.f - sg, 1.f);
                    dt *= zv[m][e] * sg;
                }
                k[m][e] = dt;
            }
            Vec8<T>::store(dx + at, k[m]);
            if (z) Vec8<T>::store(dz + at, dzv);
        }
    }
    float* to = ga.part + static_cast<size_t>(blockIdx.x) * 3 * a.d;
#pragma unroll
    for (int m = 0; m < VPT; ++m) {
        if (!in[m]) continue;
        const int c = 8 * (tid + m * static_cast<int>(blockDim.x));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            to[c + e] = apost[m][e];
            to[a.d + c + e] = ascale[m][e];
            to[2 * a.d + c + e] = apre[m][e];
        }
    }
}

// The blocks' parameter sums in a fixed order.
__global__ void __launch_bounds__(256)
    norm_sum_kernel(const float* __restrict__ part, int blocks, int d, float* __restrict__ dpost, float* __restrict__ dscale,
                    float* __restrict__ dpre) {
    __shared__ float red[8][33];
    float* const outs[3] = {dpost, dscale, dpre};
    float* out = outs[blockIdx.y];
    if (!out) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (c < d)
        for (int k = warp; k < blocks; k += 8) v += part[(static_cast<size_t>(k) * 3 + blockIdx.y) * d + c];
    red[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < d)
        out[c] = ((red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane])) + ((red[4][lane] + red[5][lane]) + (red[6][lane] + red[7][lane]));
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 152;
    return n;
}

struct NormLaunch {
    int vpt, threads, blocks;
};
// Whole warps over the row's vectors, at most 512 threads; as many blocks as `threads_per_sm` allows, each
// walking over rows.
NormLaunch norm_launch(long long rows, int d, int threads_per_sm) {
    NormLaunch l;
    const int nvec = d / 8;
    l.vpt = nvec <= 512 ? 1 : 2;
    l.threads = ((nvec + l.vpt - 1) / l.vpt + 31) / 32 * 32;
    int per = threads_per_sm / l.threads;
    if (per < 1) per = 1;
    if (per > 32) per = 32;
    const long long most = (long long)sm_count() * per;
    l.blocks = static_cast<int>(rows < most ? rows : most);
    return l;
}
constexpr int kFwdThreadsPerSm = 1024, kGradThreadsPerSm = 512;

gdn2_status norm_check(long long rows, int d, int groups, float eps, const void* post, gdn2_dtype dt) {
    if ((dt != GDN2_F32 && dt != GDN2_BF16) || rows < 0 || d <= 0 || groups <= 0 || !(eps >= 0.f)) return GDN2_ERR_INVALID_ARG;
    if (groups > 1 && !post) return GDN2_ERR_INVALID_ARG;
    if (d % 8 || d > kMaxD || d % (8 * groups) || rows >= (1LL << 40) / d) return GDN2_ERR_UNSUPPORTED;
    return GDN2_OK;
}

bool all_aligned(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (!aligned16(p)) return false;
    return true;
}

}  // namespace
}  // namespace gdn2

using namespace gdn2;

extern "C" {

gdn2_status gdn2_block_norm(const void* x, const void* z, const float* post_weight, const void* residual, const float* scale,
                            const float* pre_weight, void* r, void* n, long long rows, int d, int groups, float eps,
                            gdn2_dtype dt, void* stream) {
    gdn2_status st = norm_check(rows, d, groups, eps, post_weight, dt);
    if (st != GDN2_OK) return st;
    if ((!r && !n) || (n != nullptr) != (pre_weight != nullptr)) return GDN2_ERR_INVALID_ARG;
    if (rows == 0) return GDN2_OK;
    if (!x) return GDN2_ERR_INVALID_ARG;
    if (!all_aligned({x, z, post_weight, residual, scale, pre_weight, r, n})) return GDN2_ERR_MISALIGNED;
    const NormLaunch l = norm_launch(rows, d, kFwdThreadsPerSm);
    const NormArgs a{post_weight, scale, pre_weight, rows, d, groups, eps};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto go = [&](auto zero) {
        using T = decltype(zero);
        auto* k = l.vpt == 1 ? norm_kernel<T, 1> : norm_kernel<T, 2>;
        k<<<l.blocks, l.threads, 0, s>>>(a, static_cast<const T*>(x), static_cast<const T*>(z), static_cast<const T*>(residual),
                                         static_cast<T*>(r), static_cast<T*>(n));
    };
    if (dt == GDN2_BF16) go(__nv_bfloat16{}); else go(0.f);
    return cudaGetLastError() == cudaSuccess ? GDN2_OK : GDN2_ERR_CUDA;
}

size_t gdn2_block_norm_backward_workspace_size(long long rows, int d) {
    if (rows <= 0 || d <= 0 || d % 8 || d > kMaxD) return 0;
    return align_up(sizeof(float) * 3 * d * static_cast<size_t>(norm_launch(rows, d, kGradThreadsPerSm).blocks), 256);
}

gdn2_status gdn2_block_norm_backward(const void* x, const void* z, const float* post_weight, const void* residual,
                                     const float* scale, const float* pre_weight, const void* d_r, const void* d_n, void* dx,
                                     void* dz, float* dpost_weight, void* dresidual, float* dscale, float* dpre_weight,
                                     long long rows, int d, int groups, float eps, gdn2_dtype dt, void* workspace,
                                     size_t ws_bytes, void* stream) {
    gdn2_status st = norm_check(rows, d, groups, eps, post_weight, dt);
    if (st != GDN2_OK) return st;
    if ((z != nullptr) != (dz != nullptr) || (post_weight != nullptr) != (dpost_weight != nullptr) ||
        (scale != nullptr) != (dscale != nullptr) || (pre_weight != nullptr) != (dpre_weight != nullptr) ||
        (d_n != nullptr) != (pre_weight != nullptr) || (dresidual && !residual))
        return GDN2_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0) {  // sums over no rows
        float* const sums[] = {dpost_weight, dscale, dpre_weight};
        for (float* p : sums)
            if (p && cudaMemsetAsync(p, 0, sizeof(float) * d, s) != cudaSuccess) return GDN2_ERR_CUDA;
        return GDN2_OK;
    }
    if (!x || !dx || (!d_r && !d_n)) return GDN2_ERR_INVALID_ARG;
    if (!all_aligned({x, z, post_weight, residual, scale, pre_weight, d_r, d_n, dx, dz, dpost_weight, dresidual, dscale, dpre_weight}))
        return GDN2_ERR_MISALIGNED;
    if (!workspace || ws_bytes < gdn2_block_norm_backward_workspace_size(rows, d)) return GDN2_ERR_WORKSPACE;
    if (!aligned16(workspace)) return GDN2_ERR_MISALIGNED;
    const NormLaunch l = norm_launch(rows, d, kGradThreadsPerSm);
    const NormGradArgs a{{post_weight, scale, pre_weight, rows, d, groups, eps}, static_cast<float*>(workspace)};
    auto go = [&](auto zero) {
        using T = decltype(zero);
        auto* k = l.vpt == 2 ? norm_grad_kernel<T, 2, 512> : l.threads <= 256 ? norm_grad_kernel<T, 1, 256> : norm_grad_kernel<T, 1, 512>;
        k<<<l.blocks, l.threads, 0, s>>>(a, static_cast<const T*>(x), static_cast<const T*>(z), static_cast<const T*>(residual),
                                         static_cast<const T*>(d_r), static_cast<const T*>(d_n), static_cast<T*>(dx),
                                         static_cast<T*>(dz), static_cast<T*>(dresidual));
    };
    if (dt == GDN2_BF16) go(__nv_bfloat16{}); else go(0.f);
    if (cudaGetLastError() != cudaSuccess) return GDN2_ERR_CUDA;
    if (dpost_weight || dscale || dpre_weight)
        norm_sum_kernel<<<dim3((d + 31) / 32, 3), 256, 0, s>>>(a.part, l.blocks, d, dpost_weight, dscale, dpre_weight);
    return cudaGetLastError() == cudaSuccess ? GDN2_OK : GDN2_ERR_CUDA;
}

}  // extern "C"
