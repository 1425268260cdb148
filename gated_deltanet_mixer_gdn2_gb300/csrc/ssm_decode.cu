// ssm_decode.cu -- one token of the selective state-space mixer between its projections, in one launch:
// the causal convolution with SiLU against its kept samples, the gates, the state update and the readout.
//     u = silu(conv(x; window) + bias) = (xs [H, P], B [G, N], C [G, N]),  step = softplus(delta + delta_bias)
//     S <- e^{a step} S + step B xs^T,   y = S^T C + D xs
#include <cooperative_groups.h>

#include "ssm_common.cuh"

namespace gdn2 {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kTaps = 4;
constexpr int kMaxN = 256, kMaxP = 128;
constexpr int kCluster = 8;  // blocks of one (row, group): the portable cluster size

struct DecodeArgs {
    long long ld_x, ld_delta;
    const float *weight, *bias, *a, *delta_bias, *dskip;
    float* conv_state;  // [slots or B][3][channels]
    const int* slots;
    int n_slots, H, G, P, N, channels, heads;  // heads per block
};

template <typename S>
struct Quad;  // four state elements
template <>
struct Quad<float> {
    __device__ static float4 load(const float* p) { return __ldcs(reinterpret_cast<const float4*>(p)); }
    __device__ static void store(float* p, float4 v) { __stcs(reinterpret_cast<float4*>(p), v); }
};
template <>
struct Quad<__nv_bfloat16> {
    __device__ static float4 load(const __nv_bfloat16* p) {
        const uint2 u = __ldcs(reinterpret_cast<const uint2*>(p));
        return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                           __uint_as_float(u.y & 0xffff0000u));
    }
    __device__ static void store(__nv_bfloat16* p, float4 v) {
        __nv_bfloat162 a[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
        __stcs(reinterpret_cast<uint2*>(p), *reinterpret_cast<const uint2*>(a));
    }
};

// One block runs `heads` heads of one (row, group); the blocks of a (row, group) form a cluster, because
// the group's B and C channels have one convolution window that all of them read and one replaces, after
// a cluster barrier. The state's bytes bound it: every thread issues its loads of eight state rows (four
// columns each) before it does anything else, and the next head's before it finishes this one. 64 rows, 48 heads of 64
// values, N = 128, fp32 states: 44 us, 4.7 TB/s, 70% of the copy rate. One row: 10 us, a chain of two dependent loads, a
// cluster barrier and three block barriers.
template <typename T, typename S>
__global__ void __launch_bounds__(kThreads)
    decode_kernel(DecodeArgs a, const T* __restrict__ x, const T* __restrict__ delta, S* __restrict__ state, T* __restrict__ y) {
    __shared__ __align__(16) float sB[kMaxN], sC[kMaxN], sX[kMaxP], red[kThreads / 32][kMaxP];
    __shared__ float sGate[3];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int parts = gridDim.x / a.G, grp = blockIdx.x / parts, part = blockIdx.x - grp * parts, b = blockIdx.y;
    const int per = a.H / a.G, h_lo = grp * per + part * a.heads, h_hi = min(h_lo + a.heads, (grp + 1) * per);
    const int slot = a.slots ? __ldg(a.slots + b) : b;
    if (a.slots && (slot < 0 || slot >= a.n_slots)) return;  // inactive row: uniform over the cluster
    const int quads = a.P / 4, rpp = kThreads / quads;  // threads per state row; state rows per pass
    const int c4 = 4 * (tid % quads), r0 = tid / quads;
    const int passes = (a.N + rpp - 1) / rpp;
    constexpr int kBatch = 8;
    const size_t plane = static_cast<size_t>(a.N) * a.P;
    S* st = state + (static_cast<size_t>(slot) * a.H + h_lo) * plane;
    float4 s[kBatch];
    auto fetch = [&](const S* base, int i0) {
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            const int n = (i0 + q) * rpp + r0;
            if (n < a.N && i0 + q < passes) s[q] = Quad<S>::load(base + static_cast<size_t>(n) * a.P + c4);
        }
    };
    fetch(st, 0);

    // convolution of one channel; `keep` replaces the channel's window
    float* win = a.conv_state + static_cast<size_t>(slot) * (kTaps - 1) * a.channels;
    const T* xrow = x + static_cast<size_t>(b) * a.ld_x;
    float w1 = 0.f, w2 = 0.f, wx = 0.f;
    auto conv = [&](int c) {
        const float4 w = __ldg(reinterpret_cast<const float4*>(a.weight) + c);
        const float w0 = win[c];
        w1 = win[a.channels + c];
        w2 = win[2 * a.channels + c];
        wx = to_f32(xrow[c]);
        const float v = fmaf(w.w, wx, fmaf(w.z, w2, fmaf(w.y, w1, fmaf(w.x, w0, a.bias ? __ldg(a.bias + c) : 0.f))));
        return v * ssm_sigmoid(v);
    };
    auto keep = [&](int c) {
        win[c] = w1;
        win[a.channels + c] = w2;
        win[2 * a.channels + c] = wx;
    };
    // B and C of the group: 2 N <= 512 channels, at most two per thread
    const int cb = a.H * a.P + grp * a.N, cc = cb + a.G * a.N;
    float k1[2], k2[2], kx[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const int i = tid + m * kThreads;
        if (i < 2 * a.N) {
            const float v = conv(i < a.N ? cb + i : cc + i - a.N);
            if (i < a.N) sB[i] = v; else sC[i - a.N] = v;
            k1[m] = w1; k2[m] = w2; kx[m] = wx;
        }
    }
    const cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();  // every block of the group has read the window
    if (part == 0) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int i = tid + m * kThreads;
            if (i < 2 * a.N) {
                w1 = k1[m]; w2 = k2[m]; wx = kx[m];
                keep(i < a.N ? cb + i : cc + i - a.N);
            }
        }
    }

    for (int h = h_lo; h < h_hi; ++h, st += plane) {
        if (tid < a.P) {
            const int c = h * a.P + tid;
            sX[tid] = conv(c);
            keep(c);
        }
        if (tid == kThreads - 1) {
            const float sp = ssm_softplus(to_f32(delta[static_cast<size_t>(b) * a.ld_delta + h]) + a.delta_bias[h]);
            const float2 e = ssm_decay(ssm_gate(a.a[h] * sp));
            sGate[0] = e.x;
            sGate[1] = e.y;
            sGate[2] = sp;
        }
        __syncthreads();
        const float al = sGate[0], lo = sGate[1], sp = sGate[2];
        const float4 xv = *reinterpret_cast<const float4*>(&sX[c4]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 xs = make_float4(sp * xv.x, sp * xv.y, sp * xv.z, sp * xv.w);
        for (int i0 = 0; i0 < passes; i0 += kBatch) {
            if (i0) fetch(st, i0);
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                const int n = (i0 + q) * rpp + r0;
                if (n >= a.N || i0 + q >= passes) continue;
                const float bv = sB[n], cv = sC[n];
                float4 v = s[q];
                v.x = fmaf(al, v.x, fmaf(lo, v.x, bv * xs.x));
                v.y = fmaf(al, v.y, fmaf(lo, v.y, bv * xs.y));
                v.z = fmaf(al, v.z, fmaf(lo, v.z, bv * xs.z));
                v.w = fmaf(al, v.w, fmaf(lo, v.w, bv * xs.w));
                acc.x = fmaf(cv, v.x, acc.x);
                acc.y = fmaf(cv, v.y, acc.y);
                acc.z = fmaf(cv, v.z, acc.z);
                acc.w = fmaf(cv, v.w, acc.w);
                Quad<S>::store(st + static_cast<size_t>(n) * a.P + c4, v);
            }
        }
        if (h + 1 < h_hi) fetch(st + plane, 0);
        // y: over the threads of a column, within the warp (P / 4 is a power of two up to 32), then over the warps
        for (int d = quads; d < 32; d <<= 1) {
            acc.x += __shfl_xor_sync(0xffffffffu, acc.x, d);
            acc.y += __shfl_xor_sync(0xffffffffu, acc.y, d);
            acc.z += __shfl_xor_sync(0xffffffffu, acc.z, d);
            acc.w += __shfl_xor_sync(0xffffffffu, acc.w, d);
        }
        if (lane < quads) *reinterpret_cast<float4*>(&red[warp][c4]) = acc;
        __syncthreads();
        if (tid < a.P) {
            float v = a.dskip ? a.dskip[h] * sX[tid] : 0.f;
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) v += red[w][tid];
            y[(static_cast<size_t>(b) * a.H + h) * a.P + tid] = from_f32<T>(v);
        }
        __syncthreads();
    }
}

}  // namespace
}  // namespace gdn2

using namespace gdn2;

extern "C" gdn2_status gdn2_ssm_decode_step(const void* xbc, long long ld_xbc, const void* delta, long long ld_delta,
                                            const float* conv_weight, const float* conv_bias, const float* a,
                                            const float* delta_bias, const float* d, float* conv_state, void* state,
                                            gdn2_dtype state_dt, const int32_t* slots, int n_slots, void* y, int B, int H,
                                            int G, int P, int N, gdn2_dtype dt, void* stream) {
    if ((dt != GDN2_F32 && dt != GDN2_BF16) || (state_dt != GDN2_F32 && state_dt != GDN2_BF16) || B < 0 || H <= 0 || G <= 0 ||
        P <= 0 || N <= 0 || H % G || (slots && n_slots < 0))
        return GDN2_ERR_INVALID_ARG;
    if (!(P == 16 || P == 32 || P == 64 || P == 128) || !(N == 16 || N == 32 || N == 64 || N == 128 || N == 256) || B > 65535 || H > 32767)
        return GDN2_ERR_UNSUPPORTED;
    if (B == 0) return GDN2_OK;
    const int channels = H * P + 2 * G * N;
    if (!xbc || !delta || !conv_weight || !a || !delta_bias || !conv_state || !state || !y || ld_xbc < channels || ld_delta < H)
        return GDN2_ERR_INVALID_ARG;
    const size_t esz = dt == GDN2_BF16 ? 2 : 4;
    if (!aligned_to(xbc, esz) || !aligned_to(delta, esz) || !aligned16(conv_weight) || !aligned_to(conv_bias, 4) || !aligned_to(a, 4) ||
        !aligned_to(delta_bias, 4) || !aligned_to(d, 4) || !aligned_to(conv_state, 4) || !aligned16(state) || !aligned_to(slots, 4) ||
        !aligned_to(y, esz))
        return GDN2_ERR_MISALIGNED;
    // Blocks of a (row, group): one head each while they fit a cluster, so a small batch spreads widest.
    const int per = H / G, heads = (per + kCluster - 1) / kCluster, parts = (per + heads - 1) / heads;
    const DecodeArgs args{ld_xbc, ld_delta, conv_weight, conv_bias, a, delta_bias, d, conv_state, slots, n_slots, H, G, P, N, channels, heads};
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(G * parts), B);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(parts);
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    auto go = [&](auto t, auto s) {
        using T = decltype(t);
        using S = decltype(s);
        return cudaLaunchKernelEx(&cfg, decode_kernel<T, S>, args, static_cast<const T*>(xbc), static_cast<const T*>(delta),
                                  static_cast<S*>(state), static_cast<T*>(y));
    };
    using BF = __nv_bfloat16;
    cudaError_t e;
    if (dt == GDN2_BF16) e = state_dt == GDN2_BF16 ? go(BF{}, BF{}) : go(BF{}, 0.f);
    else e = state_dt == GDN2_BF16 ? go(0.f, BF{}) : go(0.f, 0.f);
    return e == cudaSuccess ? GDN2_OK : GDN2_ERR_CUDA;
}
