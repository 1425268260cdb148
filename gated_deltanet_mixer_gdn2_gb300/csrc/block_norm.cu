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

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// Room for the sums over a row and over its groups. Every sum takes the other slot than the sum before it, of whatever kind
// and in whichever row (`slot` changes with each), so that one barrier per sum is enough: a sum's writes to a slot lie
// behind the barrier of the sum between, and that one behind all reads of the slot's last sum.
struct RowSums {
    float part[2][2][kMaxD / 8 / 32];  // [slot][which][32 vectors or a warp]
    float vec[kMaxD / 8], group[kMaxD / 8];
};

// Sums over the whole row of kWhich values per thread, the same in every thread.
template <int kWhich>
__device__ __forceinline__ void row_total(RowSums& rs, int& slot, float (&v)[kWhich]) {
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    float (&part)[2][kMaxD / 8 / 32] = rs.part[slot];
    slot ^= 1;
#pragma unroll
    for (int w = 0; w < kWhich; ++w) {
        const float t = warp_sum(v[w]);
        if ((threadIdx.x & 31) == 0) part[w][warp] = t;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWhich; ++w)
        v[w] = warp_sum(static_cast<int>(threadIdx.x & 31) < warps ? part[w][threadIdx.x & 31] : 0.f);
}

// Where a thread's vectors lie among the groups. Where groups are whole warps' worth of vectors (every common width)
// their sums take a warp sum per 32 vectors and one barrier; else every vector's part and two more barriers.
template <int VPT>
struct Groups {
    int per, blocks, first[VPT];  // vectors per group; 32-vector blocks per group and this vector's first one, or its group
    bool whole;
    __device__ __forceinline__ Groups(int nvec, int groups) {
        per = nvec / groups;
        whole = per % 32 == 0;
        blocks = per / 32;
#pragma unroll
        for (int m = 0; m < VPT; ++m) {
            const int i = threadIdx.x + m * blockDim.x, g = i < nvec ? i / per : 0;
            first[m] = whole ? g * blocks : g;
        }
    }
};
template <int VPT>
__device__ __forceinline__ void group_sums(RowSums& rs, int& slot, const Groups<VPT>& gr, int groups, const bool (&in)[VPT], float (&v)[VPT]) {
    const int tid = threadIdx.x;
    float (&part)[kMaxD / 8 / 32] = rs.part[slot][0];
    slot ^= 1;
    if (gr.whole) {
#pragma unroll
        for (int m = 0; m < VPT; ++m) {
            const float t = warp_sum(v[m]);
            if (in[m] && (tid & 31) == 0) part[(tid + m * blockDim.x) >> 5] = t;
        }
        __syncthreads();
#pragma unroll
        for (int m = 0; m < VPT; ++m) {
            float t = 0.f;
            for (int k = 0; k < gr.blocks; ++k) t += part[gr.first[m] + k];
            v[m] = t;
        }
        return;
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < VPT; ++m)
        if (in[m]) rs.vec[tid + m * blockDim.x] = v[m];
    __syncthreads();
    const int warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
    for (int g = warp; g < groups; g += warps) {
        float t = 0.f;
        for (int i = lane; i < gr.per; i += 32) t += rs.vec[g * gr.per + i];
        t = warp_sum(t);
        if (lane == 0) rs.group[g] = t;
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < VPT; ++m) v[m] = rs.group[gr.first[m]];
}

// Eight elements as they lie in memory.
template <typename T>
struct alignas(16) Raw8 {
    uint4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw8<T> load_raw(const T* p) {
    Raw8<T> r;
#pragma unroll
    for (int k = 0; k < static_cast<int>(sizeof(T) / 2); ++k) r.w[k] = reinterpret_cast<const uint4*>(p)[k];
    return r;
}
template <typename T>
__device__ __forceinline__ void widen8(const Raw8<T>& r, float (&x)[8]) {
    if constexpr (sizeof(T) == 2) {
        const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
        const float* f = reinterpret_cast<const float*>(&r);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = f[i];
    }
}

__device__ __forceinline__ void weights8(const float* w, int c, bool in, float (&x)[8]) {
    if (w && in) {
        const float4 a = reinterpret_cast<const float4*>(w + c)[0], b = reinterpret_cast<const float4*>(w + c)[1];
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 1.f;
    }
}

// One row per block and trip, VPT vectors of eight elements per thread. The weights lie in shared memory, so that one
// vector per thread fits 64 registers and 32 warps cover the loads and the two barriers of a row: at 16384 x 4096,
// 122 us (5.5 TB/s, 81% of the copy rate); with two vectors per thread and 24 warps 140 us, with the weights in the
// registers of 16 warps 159 us. The next row's loads are in flight while a row is summed.
template <typename T, int VPT, int kMaxThreads, int kPerSm>
__global__ void __launch_bounds__(kMaxThreads, kPerSm)
    norm_kernel(NormArgs a, const T* x, const T* z, const T* residual, T* r_out, T* n_out) {
    __shared__ RowSums rs;
    const int tid = threadIdx.x, nvec = a.d / 8;
    extern __shared__ float4 weights_f4[];
    float* const weights = reinterpret_cast<float*>(weights_f4);  // post, scale, pre; ones where absent
    for (int i = tid; i < a.d; i += blockDim.x) {
        weights[i] = a.post ? a.post[i] : 1.f;
        weights[a.d + i] = a.scale ? a.scale[i] : 1.f;
        weights[2 * a.d + i] = a.pre ? a.pre[i] : 1.f;
    }
    __syncthreads();
    bool in[VPT];
    int at[VPT];
#pragma unroll
    for (int m = 0; m < VPT; ++m) {
        const int i = tid + m * blockDim.x;
        in[m] = i < nvec;
        at[m] = in[m] ? 8 * i : 0;
    }
    auto weight = [&](int which, int m, float (&w)[8]) {
        const float4* p = reinterpret_cast<const float4*>(weights + which * a.d + at[m]);
        const float4 u = p[0], v = p[1];
        w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w; w[4] = v.x; w[5] = v.y; w[6] = v.z; w[7] = v.w;
    };
    const float inv_width = static_cast<float>(a.groups) / a.d, inv_d = 1.f / a.d;
    const Groups<VPT> gr(nvec, a.groups);
    Raw8<T> rx[VPT], rz[VPT], rr[VPT];
    auto fetch = [&](long long row) {
        if (row >= a.rows) return;
        const size_t base = static_cast<size_t>(row) * a.d;
#pragma unroll
        for (int m = 0; m < VPT; ++m) {
            if (!in[m]) continue;
            rx[m] = load_raw(x + base + at[m]);
            if (z) rz[m] = load_raw(z + base + at[m]);
            if (residual) rr[m] = load_raw(residual + base + at[m]);
        }
    };
    int slot = 0;
    fetch(blockIdx.x);
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const size_t base = static_cast<size_t>(row) * a.d;
        float t[VPT][8], res[VPT][8], part[VPT];
#pragma unroll
        for (int m = 0; m < VPT; ++m) {
            part[m] = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) t[m][e] = res[m][e] = 0.f;
            if (!in[m]) continue;
            widen8(rx[m], t[m]);
            if (residual) widen8(rr[m], res[m]);
            if (z) {
                float zz[8];
                widen8(rz[m], zz);
#pragma unroll
                for (int e = 0; e < 8; ++e) t[m][e] *= zz[e] * ssm_sigmoid(zz[e]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) part[m] = fmaf(t[m][e], t[m][e], part[m]);
        }
        fetch(row + gridDim.x);
        if (a.post) {
            group_sums<VPT>(rs, slot, gr, a.groups, in, part);
#pragma unroll
            for (int m = 0; m < VPT; ++m) {
                const float inv = rsqrtf(fmaf(part[m], inv_width, a.eps));
                float post[8];
                weight(0, m, post);
#pragma unroll
                for (int e = 0; e < 8; ++e) t[m][e] *= inv * post[e];
            }
        }
#pragma unroll
        for (int m = 0; m < VPT; ++m) {
            part[m] = 0.f;
            float scale[8];
            weight(1, m, scale);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                t[m][e] = fmaf(t[m][e], scale[e], res[m][e]);
                part[m] = fmaf(t[m][e], t[m][e], part[m]);
            }
            if (r_out && in[m]) Vec8<T>::store(r_out + base + at[m], t[m]);
        }
        if (n_out) {
            float total[1] = {0.f};
#pragma unroll
            for (int m = 0; m < VPT; ++m) total[0] += part[m];
            row_total<1>(rs, slot, total);
            const float inv = rsqrtf(fmaf(total[0], inv_d, a.eps));
#pragma unroll
            for (int m = 0; m < VPT; ++m) {
                if (!in[m]) continue;
                float pre[8];
                weight(2, m, pre);
#pragma unroll
                for (int e = 0; e < 8; ++e) t[m][e] *= inv * pre[e];
                Vec8<T>::store(n_out + base + at[m], t[m]);
            }
        }
    }
}

struct NormGradArgs {
    NormArgs n;
    float* part;  // [blocks][2][d]: sums of dr th, of d_n nh
};

// The forward's row again, then backwards through it: with nh = r / rms(r) and th = t / rms_group(t),
//     dr = d_r + (k - nh mean(k nh)) / rms(r),    k = d_n pre
//     dt = (q - th mean_group(q th)) / rms_group(t), q = dr scale post
// dx = dt silu(z), dz = dt x silu'(z). dpost and dscale are one sum over the rows, of dr th, times scale and post; it and
// dpre's, and the weights, stay in registers over the block's rows, the next row's loads in flight. 8192 x 2048 bf16 with
// all of its inputs: 67 us with the sums, 4 TB/s, 59% of the copy rate: the sums' registers leave room for 16 warps, and two row sums
// with their barriers stand between a row's loads and its stores. Two vectors per thread (above 4096 columns) do not fit the
// registers and spill: 2048 x 8192 takes 150 us, 2048 x 4096 48 us.
template <typename T, int VPT, int kMaxThreads, int kPerSm>
__global__ void __launch_bounds__(kMaxThreads, kPerSm)
    norm_grad_kernel(NormGradArgs ga, const T* x, const T* z, const T* residual, const T* d_r, const T* d_n, T* dx, T* dz, T* dres) {
    const NormArgs& a = ga.n;
    __shared__ RowSums rs;
    const int tid = threadIdx.x, nvec = a.d / 8;
    float sp[VPT][8], pre[VPT][8];           // scale post, pre
    float asum[VPT][8] = {}, apre[VPT][8] = {};  // sums of dr th (dpost = scale asum, dscale = post asum) and of d_n nh
    bool in[VPT];
    int at[VPT];
#pragma unroll
    for (int m = 0; m < VPT; ++m) {
        in[m] = tid + m * static_cast<int>(blockDim.x) < nvec;
        at[m] = in[m] ? 8 * (tid + m * static_cast<int>(blockDim.x)) : 0;
        float post[8];
        weights8(a.post, at[m], in[m], post);
        weights8(a.scale, at[m], in[m], sp[m]);
        weights8(a.pre, at[m], in[m], pre[m]);
#pragma unroll
        for (int e = 0; e < 8; ++e) sp[m][e] *= post[e];
    }
    const float inv_width = static_cast<float>(a.groups) / a.d, inv_d = 1.f / a.d;
    const Groups<VPT> gr(nvec, a.groups);
    Raw8<T> rx[VPT], rz[VPT], rr[VPT], rdr[VPT], rdn[VPT];
    auto fetch = [&](long long row) {
        if (row >= a.rows) return;
        const size_t base = static_cast<size_t>(row) * a.d;
#pragma unroll
        for (int m = 0; m < VPT; ++m) {
            if (!in[m]) continue;
            rx[m] = load_raw(x + base + at[m]);
            if (z) rz[m] = load_raw(z + base + at[m]);
            if (residual) rr[m] = load_raw(residual + base + at[m]);
            if (d_r) rdr[m] = load_raw(d_r + base + at[m]);
            if (d_n) rdn[m] = load_raw(d_n + base + at[m]);
        }
    };
    int slot = 0;
    fetch(blockIdx.x);
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const size_t base = static_cast<size_t>(row) * a.d;
        float t[VPT][8], r[VPT][8], dr[VPT][8], k[VPT][8], one[VPT], inv_t[VPT], both[2] = {0.f, 0.f};
        Raw8<T> kx[VPT], kz[VPT];  // x and z for the end of the row
#pragma unroll
        for (int m = 0; m < VPT; ++m) {
            kx[m] = rx[m];
            kz[m] = rz[m];
            one[m] = 0.f;
            inv_t[m] = 1.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) t[m][e] = r[m][e] = dr[m][e] = k[m][e] = 0.f;
            if (!in[m]) continue;
            widen8(rx[m], t[m]);
            if (residual) widen8(rr[m], r[m]);
            if (d_r) widen8(rdr[m], dr[m]);
            if (d_n) widen8(rdn[m], k[m]);
            if (z) {
                float zv[8];
                widen8(rz[m], zv);
#pragma unroll
                for (int e = 0; e < 8; ++e) t[m][e] *= zv[e] * ssm_sigmoid(zv[e]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) one[m] = fmaf(t[m][e], t[m][e], one[m]);
        }
        fetch(row + gridDim.x);
        if (a.post) {
            group_sums<VPT>(rs, slot, gr, a.groups, in, one);
#pragma unroll
            for (int m = 0; m < VPT; ++m) {
                inv_t[m] = rsqrtf(fmaf(one[m], inv_width, a.eps));
#pragma unroll
                for (int e = 0; e < 8; ++e) t[m][e] *= inv_t[m];  // th
            }
        }
#pragma unroll
        for (int m = 0; m < VPT; ++m) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                r[m][e] = fmaf(t[m][e], sp[m][e], r[m][e]);
                both[0] = fmaf(r[m][e], r[m][e], both[0]);
                both[1] = fmaf(k[m][e] * pre[m][e], r[m][e], both[1]);
            }
        }
        if (d_n) {
            row_total<2>(rs, slot, both);
            const float inv = rsqrtf(fmaf(both[0], inv_d, a.eps));
            const float mean = both[1] * inv * inv_d;  // mean(k nh)
#pragma unroll
            for (int m = 0; m < VPT; ++m) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float nh = r[m][e] * inv;
                    apre[m][e] = fmaf(k[m][e], nh, apre[m][e]);
                    dr[m][e] = fmaf(inv, fmaf(-nh, mean, k[m][e] * pre[m][e]), dr[m][e]);
                }
            }
        }
#pragma unroll
        for (int m = 0; m < VPT; ++m) {
            if (dres && in[m]) Vec8<T>::store(dres + base + at[m], dr[m]);
            one[m] = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                asum[m][e] = fmaf(dr[m][e], t[m][e], asum[m][e]);
                k[m][e] = dr[m][e] * sp[m][e];
                one[m] = fmaf(k[m][e], t[m][e], one[m]);
            }
        }
        if (a.post) {
            group_sums<VPT>(rs, slot, gr, a.groups, in, one);
#pragma unroll
            for (int m = 0; m < VPT; ++m) {
                const float mean = one[m] * inv_width;
#pragma unroll
                for (int e = 0; e < 8; ++e) k[m][e] = inv_t[m] * fmaf(-t[m][e], mean, k[m][e]);
            }
        }
#pragma unroll
        for (int m = 0; m < VPT; ++m) {
            if (!in[m]) continue;
            if (z) {
                float xv[8], zv[8], dzv[8];
                widen8(kx[m], xv);
                widen8(kz[m], zv);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float sg = ssm_sigmoid(zv[e]);
                    dzv[e] = k[m][e] * xv[e] * sg * fmaf(zv[e], 1.f - sg, 1.f);
                    k[m][e] *= zv[e] * sg;
                }
                Vec8<T>::store(dz + base + at[m], dzv);
            }
            Vec8<T>::store(dx + base + at[m], k[m]);
        }
    }
    float* to = ga.part + static_cast<size_t>(blockIdx.x) * 2 * a.d;
#pragma unroll
    for (int m = 0; m < VPT; ++m) {
        if (!in[m]) continue;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            reinterpret_cast<float4*>(to + at[m])[e] = make_float4(asum[m][4 * e], asum[m][4 * e + 1], asum[m][4 * e + 2], asum[m][4 * e + 3]);
            reinterpret_cast<float4*>(to + a.d + at[m])[e] = make_float4(apre[m][4 * e], apre[m][4 * e + 1], apre[m][4 * e + 2], apre[m][4 * e + 3]);
        }
    }
}

// The blocks' parameter sums in a fixed order.
__global__ void __launch_bounds__(1024)
    norm_sum_kernel(const float* __restrict__ part, int blocks, int d, const float* __restrict__ post, const float* __restrict__ scale,
                    float* __restrict__ dpost, float* __restrict__ dscale, float* __restrict__ dpre) {
    __shared__ float red[32][33];
    if (blockIdx.y ? !dpre : !dpost && !dscale) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (c < d) {
        const float* src = part + static_cast<size_t>(blockIdx.y) * d + c;
        const size_t step = 2 * static_cast<size_t>(d);
        for (int k = warp; k < blocks; k += 32 * 10) {  // ten loads in flight: all of two blocks per SM at once
            float t[10];
#pragma unroll
            for (int q = 0; q < 10; ++q) t[q] = k + 32 * q < blocks ? src[(k + 32 * q) * step] : 0.f;
#pragma unroll
            for (int q = 0; q < 10; ++q) v += t[q];
        }
    }
    red[warp][lane] = v;
    __syncthreads();
    if (warp || c >= d) return;
    v = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) v += red[k][lane];
    if (blockIdx.y) {
        dpre[c] = v;
    } else {
        if (dpost) dpost[c] = scale ? scale[c] * v : v;
        if (dscale) dscale[c] = post ? post[c] * v : v;
    }
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
// Whole warps over the row's vectors, one per thread up to 4096 wide, else two; as many blocks per SM as
// `threads_per_sm` allows, each walking over rows.
NormLaunch norm_launch(long long rows, int d, int threads_per_sm) {
    NormLaunch l;
    const int nvec = d / 8;
    l.vpt = d <= 4096 ? 1 : 2;
    l.threads = ((nvec + l.vpt - 1) / l.vpt + 31) / 32 * 32;
    int per = threads_per_sm / l.threads;
    if (per < 1) per = 1;
    const long long most = (long long)sm_count() * per;
    l.blocks = static_cast<int>(rows < most ? rows : most);
    return l;
}
NormLaunch norm_fwd_launch(long long rows, int d) { return norm_launch(rows, d, d <= 4096 ? 1024 : 512); }
NormLaunch norm_grad_launch(long long rows, int d) { return norm_launch(rows, d, 512); }

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
    const NormLaunch l = norm_fwd_launch(rows, d);
    const int smem = 3 * d * static_cast<int>(sizeof(float));
    const NormArgs a{post_weight, scale, pre_weight, rows, d, groups, eps};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto go = [&](auto zero) {
        using T = decltype(zero);
        auto* k = l.vpt == 1 ? norm_kernel<T, 1, 512, 2> : norm_kernel<T, 2, 512, 1>;
        if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 3 * kMaxD * static_cast<int>(sizeof(float))) != cudaSuccess)
            return false;
        k<<<l.blocks, l.threads, smem, s>>>(a, static_cast<const T*>(x), static_cast<const T*>(z), static_cast<const T*>(residual),
                                            static_cast<T*>(r), static_cast<T*>(n));
        return cudaGetLastError() == cudaSuccess;
    };
    return (dt == GDN2_BF16 ? go(__nv_bfloat16{}) : go(0.f)) ? GDN2_OK : GDN2_ERR_CUDA;
}

size_t gdn2_block_norm_backward_workspace_size(long long rows, int d) {
    if (rows <= 0 || d <= 0 || d % 8 || d > kMaxD) return 0;
    return align_up(sizeof(float) * 2 * d * static_cast<size_t>(norm_grad_launch(rows, d).blocks), 256);
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
    const NormLaunch l = norm_grad_launch(rows, d);
    const NormGradArgs a{{post_weight, scale, pre_weight, rows, d, groups, eps}, static_cast<float*>(workspace)};
    auto go = [&](auto zero) {
        using T = decltype(zero);
        auto* k = l.vpt == 2 ? norm_grad_kernel<T, 2, 512, 1> : l.threads <= 256 ? norm_grad_kernel<T, 1, 256, 2> : norm_grad_kernel<T, 1, 512, 1>;
        k<<<l.blocks, l.threads, 0, s>>>(a, static_cast<const T*>(x), static_cast<const T*>(z), static_cast<const T*>(residual),
                                            static_cast<const T*>(d_r), static_cast<const T*>(d_n), static_cast<T*>(dx),
                                            static_cast<T*>(dz), static_cast<T*>(dresidual));
        return cudaGetLastError() == cudaSuccess;
    };
    if (!(dt == GDN2_BF16 ? go(__nv_bfloat16{}) : go(0.f))) return GDN2_ERR_CUDA;
    if (dpost_weight || dscale || dpre_weight)
        norm_sum_kernel<<<dim3((d + 31) / 32, 2), 1024, 0, s>>>(a.part, l.blocks, d, post_weight, scale, dpost_weight, dscale, dpre_weight);
    return cudaGetLastError() == cudaSuccess ? GDN2_OK : GDN2_ERR_CUDA;
}

}  // extern "C"
