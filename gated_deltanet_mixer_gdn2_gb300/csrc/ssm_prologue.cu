// ssm_prologue.cu -- what stands between the selective state-space mixer's projection and its scan:
//     v_t = bias + sum_{j=0..3} W_j x_{t-3+j},  u = silu(v)       (depthwise, causal within its sequence)
//     step = softplus(delta + delta_bias),      g = a step
// and the gradients of all of it. Both directions stream rows once and are bound by HBM.
#include <initializer_list>
#include <type_traits>

#include "ssm_common.cuh"

namespace gdn2 {
namespace {

constexpr int kTaps = 4;
constexpr int kThreads = 128;

// CH consecutive channels of a row, moved as one word; fp32 in registers.
template <typename T, int CH>
struct Chan {
    struct alignas(sizeof(T) * CH) Raw {
        T v[CH];
    };
    __device__ static Raw load(const T* p) { return *reinterpret_cast<const Raw*>(p); }
    __device__ static void widen(const Raw& r, float (&x)[CH]) {
        if constexpr (sizeof(T) == 2 && CH % 2 == 0) {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
            for (int i = 0; i < CH / 2; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < CH; ++i) x[i] = to_f32(r.v[i]);
        }
    }
    __device__ static void store(T* p, const float (&x)[CH]) {
        Raw r;
        if constexpr (sizeof(T) == 2 && CH % 2 == 0) {
            uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
            for (int i = 0; i < CH / 2; ++i) w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < CH; ++i) r.v[i] = from_f32<T>(x[i]);
        }
        *reinterpret_cast<Raw*>(p) = r;
    }
};

struct ConvArgs {
    Seqs seqs;
    long long rows;
    int channels, H, run;  // run: token rows per block
    const float *weight, *bias, *state;  // [channels][4], [channels] or null, [B][3][channels] or null
    const float *a, *delta_bias;         // [H]
    long long ld_x, ld_delta;
    int conv_blocks_x, conv_blocks_y;    // channel blocks, runs
    int gate_blocks;                     // the grid's first blocks
};

// The three samples before row r of the sequence that starts at `start`: rows, then the given state, then zeros.
template <typename T, int CH>
__device__ __forceinline__ void window_before(const ConvArgs& a, const T* x, int c, int r, int start, int seq,
                                              float (&w)[kTaps - 1][CH]) {
#pragma unroll
    for (int j = 0; j < kTaps - 1; ++j) {
        const int src = r - (kTaps - 1) + j;
        if (src >= start) {
            Chan<T, CH>::widen(Chan<T, CH>::load(x + static_cast<size_t>(src) * a.ld_x + c), w[j]);
        } else if (a.state) {
            const float* sp = a.state + (static_cast<size_t>(seq) * (kTaps - 1) + (src - start + kTaps - 1)) * a.channels + c;
#pragma unroll
            for (int e = 0; e < CH; ++e) w[j][e] = sp[e];
        } else {
#pragma unroll
            for (int e = 0; e < CH; ++e) w[j][e] = 0.f;
        }
    }
}

// The convolution at one row: taps over the three rows before it and itself.
template <int CH>
__device__ __forceinline__ void taps(const float (&w)[kTaps][CH], const float (&bias)[CH], const float (&a)[CH], const float (&b)[CH],
                                     const float (&c)[CH], const float (&d)[CH], float (&v)[CH]) {
    if constexpr (CH % 2 == 0) {
#pragma unroll
        for (int e = 0; e < CH; e += 2) {
            uint64_t t = fma_f32x2(f32x2(w[0][e], w[0][e + 1]), f32x2(a[e], a[e + 1]), f32x2(bias[e], bias[e + 1]));
            t = fma_f32x2(f32x2(w[1][e], w[1][e + 1]), f32x2(b[e], b[e + 1]), t);
            t = fma_f32x2(f32x2(w[2][e], w[2][e + 1]), f32x2(c[e], c[e + 1]), t);
            t = fma_f32x2(f32x2(w[3][e], w[3][e + 1]), f32x2(d[e], d[e + 1]), t);
            f32x2_split(t, v[e], v[e + 1]);
        }
    } else {
        v[0] = fmaf(w[3][0], d[0], fmaf(w[2][0], c[0], fmaf(w[1][0], b[0], fmaf(w[0][0], a[0], bias[0]))));
    }
}

// One thread holds CH channels and walks down a run of rows with the window of the last three in registers and the next
// four rows in flight. Rows of no sequence are left alone. The first blocks compute the
// gates, so that they do not trail behind. 8192 rows of 6144 bf16 channels and 64 heads: 48 us, 4.3 TB/s, 63% of the copy
// rate; with rows that allow words of two channels 55 us, of one 72 us.
template <typename T, int CH, bool kSilu>
__global__ void __launch_bounds__(kThreads, 8)
    prologue_kernel(ConvArgs a, const T* __restrict__ x, const T* __restrict__ delta, T* __restrict__ u, T* __restrict__ step,
                    T* __restrict__ g) {
    using Ch = Chan<T, CH>;
    if (static_cast<int>(blockIdx.x) < a.gate_blocks) {
        long long lo, hi;
        a.seqs.covered(lo, hi);
        const long long n = hi * a.H, stride = static_cast<long long>(a.gate_blocks) * kThreads;
        for (long long i = lo * a.H + blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x; i < n; i += stride) {
            const long long r = i / a.H;
            const int h = static_cast<int>(i - r * a.H);
            const float st = ssm_softplus(to_f32(delta[r * a.ld_delta + h]) + a.delta_bias[h]);
            step[i] = from_f32<T>(st);
            g[i] = from_f32<T>(a.a[h] * st);
        }
        return;
    }
    const int blk = blockIdx.x - a.gate_blocks;
    const int by = blk / a.conv_blocks_x, bx = blk - by * a.conv_blocks_x;
    const int c = CH * (bx * kThreads + threadIdx.x);
    if (c >= a.channels) return;
    float w[kTaps][CH], bias[CH];
#pragma unroll
    for (int e = 0; e < CH; ++e) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(a.weight) + c + e);
        w[0][e] = v.x; w[1][e] = v.y; w[2][e] = v.z; w[3][e] = v.w;
        bias[e] = a.bias ? __ldg(a.bias + c + e) : 0.f;
    }
    long long first, last;
    a.seqs.covered(first, last);
    const int r0 = static_cast<int>(max(static_cast<long long>(by) * a.run, first)), r1 = static_cast<int>(min((by + 1LL) * a.run, last));
    // one stretch of a sequence after the other; within it four rows at a time, the next four in flight
    for (int lo = r0; lo < r1;) {
        int seq, start, end;
        if (!find_row(a.seqs, lo, seq, start, end)) {
            ++lo;
            continue;
        }
        const int hi = min(end, r1);
        float win[kTaps][CH];  // rows r-3, r-2, r-1 at [r & 3 ..]: rotated by the unrolled loop
        {
            float before[kTaps - 1][CH];
            window_before<T, CH>(a, x, c, lo, start, seq, before);
#pragma unroll
            for (int j = 0; j < kTaps - 1; ++j)
#pragma unroll
                for (int e = 0; e < CH; ++e) win[j][e] = before[j][e];
        }
        const T* xp = x + static_cast<size_t>(lo) * a.ld_x + c;
        T* up = u + static_cast<size_t>(lo) * a.channels + c;
        typename Ch::Raw next[kTaps];
#pragma unroll
        for (int q = 0; q < kTaps; ++q)
            if (lo + q < hi) next[q] = Ch::load(xp + static_cast<size_t>(q) * a.ld_x);
        for (int r = lo; r < hi; r += kTaps) {
            typename Ch::Raw raw[kTaps];
#pragma unroll
            for (int q = 0; q < kTaps; ++q) raw[q] = next[q];
            xp += kTaps * a.ld_x;
#pragma unroll
            for (int q = 0; q < kTaps; ++q)
                if (r + kTaps + q < hi) next[q] = Ch::load(xp + static_cast<size_t>(q) * a.ld_x);
#pragma unroll
            for (int q = 0; q < kTaps; ++q) {
                float v[CH];
                Ch::widen(raw[q], win[(q + 3) & 3]);
                taps<CH>(w, bias, win[q], win[(q + 1) & 3], win[(q + 2) & 3], win[(q + 3) & 3], v);
                if (kSilu) {
#pragma unroll
                    for (int e = 0; e < CH; ++e) v[e] *= ssm_sigmoid(v[e]);
                }
                if (r + q < hi) Ch::store(up + static_cast<size_t>(q) * a.channels, v);
            }
            up += static_cast<size_t>(kTaps) * a.channels;
        }
        lo = hi;
    }
}

// New convolution states: the last three samples of [state, x of the sequence], after every block of the
// convolution has read the old ones. One thread per (sequence, channel).
template <typename T>
__global__ void __launch_bounds__(256) window_kernel(Seqs seqs, const T* __restrict__ x, long long ld_x, float* state, int channels) {
    const long long i = blockIdx.x * 256LL + threadIdx.x;
    if (i >= static_cast<long long>(seqs.B) * channels) return;
    const int b = static_cast<int>(i / channels), c = static_cast<int>(i - static_cast<long long>(b) * channels);
    int start, len;
    seqs.span(b, start, len);
    float* sp = state + static_cast<size_t>(b) * (kTaps - 1) * channels + c;
    float nw[kTaps - 1];
#pragma unroll
    for (int j = 0; j < kTaps - 1; ++j) {
        const int e = len + j;  // index into [old (3), x (len)]
        nw[j] = e < kTaps - 1 ? sp[static_cast<size_t>(e) * channels]
                              : to_f32(x[static_cast<size_t>(start + e - (kTaps - 1)) * ld_x + c]);
    }
#pragma unroll
    for (int j = 0; j < kTaps - 1; ++j) sp[static_cast<size_t>(j) * channels] = nw[j];
}

// ---------------------------------------------------------------------------------------------
// gradients

constexpr int kGateRows = 16;  // token rows of one gate block

struct ConvGradArgs {
    ConvArgs c;
    long long ld_du, ld_dx, ld_ddelta;
    float *part, *gate_part;  // [runs][channels][5]; [gate blocks][H][2]
};

// dv_t = du_t silu'(v_t);  dx_s = sum_j W_j dv_{s+3-j};  dW_j = sum_t dv_t x_{t-3+j};  dbias = sum_t dv_t.
// One thread walks down a run of rows of CH channels with the last three x and dv in registers: at row
// r it forms dv_r and, from it and the three before, dx_{r-3}. The three rows after the run (of its last
// sequence) are formed again here for its own dx and belong to the next run's sums. Sums of a run go
// to `part`; sum_kernel adds the runs in order. 8192 rows of 6144 bf16 channels: 93 us with the sums, 3.3 TB/s, bound by
// 60 multiply-adds per value as much as by memory; words of two channels 123 us, of one 187 us.
template <typename T, int CH, bool kSilu>
__global__ void __launch_bounds__(kThreads, 3)
    prologue_grad_kernel(ConvGradArgs ga, const T* __restrict__ x, const T* __restrict__ delta, const T* __restrict__ du,
                         const T* __restrict__ dstep, const T* __restrict__ dg, T* __restrict__ dx, T* __restrict__ ddelta) {
    using Ch = Chan<T, CH>;
    const ConvArgs& a = ga.c;
    if (static_cast<int>(blockIdx.x) < a.gate_blocks) {
        __shared__ float red[kThreads / 32][32][2];
        const int blk = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const long long lo = static_cast<long long>(blk) * kGateRows;
        long long first, last;  // rows of no sequence enter no sum
        a.seqs.covered(first, last);
        for (int h0 = 0; h0 < a.H; h0 += 32) {
            const int h = h0 + lane;
            float sa = 0.f, sb = 0.f;
            if (h < a.H) {
                const float av = a.a[h], bv = a.delta_bias[h];
#pragma unroll
                for (int k = 0; k < kGateRows / 4; ++k) {
                    const long long r = lo + warp + 4 * k;
                    if (r < first || r >= last) continue;
                    const float v = to_f32(delta[r * a.ld_delta + h]) + bv, dgv = to_f32(dg[r * a.H + h]);
                    const float dv = fmaf(av, dgv, to_f32(dstep[r * a.H + h])) * ssm_sigmoid(v);
                    ddelta[r * ga.ld_ddelta + h] = from_f32<T>(dv);
                    sa = fmaf(dgv, ssm_softplus(v), sa);
                    sb += dv;
                }
            }
            red[warp][lane][0] = sa;
            red[warp][lane][1] = sb;
            __syncthreads();
            if (warp == 0 && h < a.H) {
                float* to = ga.gate_part + (static_cast<size_t>(blk) * a.H + h) * 2;
#pragma unroll
                for (int k = 0; k < 2; ++k) to[k] = (red[0][lane][k] + red[1][lane][k]) + (red[2][lane][k] + red[3][lane][k]);
            }
            __syncthreads();
        }
        return;
    }
    const int cblk = blockIdx.x - a.gate_blocks;
    const int by = cblk / a.conv_blocks_x, bx = cblk - by * a.conv_blocks_x;
    const int c = CH * (bx * kThreads + threadIdx.x);
    if (c >= a.channels) return;
    float w[kTaps][CH], bias[CH], dw[kTaps][CH] = {}, db[CH] = {};
#pragma unroll
    for (int e = 0; e < CH; ++e) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(a.weight) + c + e);
        w[0][e] = v.x; w[1][e] = v.y; w[2][e] = v.z; w[3][e] = v.w;
        bias[e] = a.bias ? __ldg(a.bias + c + e) : 0.f;
    }
    long long first, last;
    a.seqs.covered(first, last);
    const int r0 = static_cast<int>(max(static_cast<long long>(by) * a.run, first)), r1 = static_cast<int>(min((by + 1LL) * a.run, last));
    for (int lo = r0; lo < r1;) {
        int seq, start, end;
        if (!find_row(a.seqs, lo, seq, start, end)) {
            ++lo;
            continue;
        }
        // rows [lo, hi) of the run, then (up to) three more of the sequence for this run's last dx
        const int hi = min(end, r1), stop = min(end, r1 + kTaps - 1);
        float win[kTaps][CH], dvw[kTaps][CH];  // x and dv of rows r-3, r-2, r-1 at [r & 3 ..], rotated by the unrolled loop
        {
            float before[kTaps - 1][CH];
            window_before<T, CH>(a, x, c, lo, start, seq, before);
#pragma unroll
            for (int j = 0; j < kTaps - 1; ++j)
#pragma unroll
                for (int e = 0; e < CH; ++e) {
                    win[j][e] = before[j][e];
                    dvw[j][e] = 0.f;
                }
        }
        const T *xp = x + static_cast<size_t>(lo) * a.ld_x + c, *dp = du + static_cast<size_t>(lo) * ga.ld_du + c;
        T* op = dx + static_cast<size_t>(lo) * ga.ld_dx + c;
        typename Ch::Raw nx[kTaps], nd[kTaps];
#pragma unroll
        for (int q = 0; q < kTaps; ++q)
            if (lo + q < stop) {
                nx[q] = Ch::load(xp + static_cast<size_t>(q) * a.ld_x);
                nd[q] = Ch::load(dp + static_cast<size_t>(q) * ga.ld_du);
            }
        // three rows past the last one, of zero dv, bring out the last dx of the sequence
        for (int r = lo; r < hi + kTaps - 1; r += kTaps) {
            typename Ch::Raw rx[kTaps], rd[kTaps];
#pragma unroll
            for (int q = 0; q < kTaps; ++q) {
                rx[q] = nx[q];
                rd[q] = nd[q];
            }
            xp += kTaps * a.ld_x;
            dp += kTaps * ga.ld_du;
#pragma unroll
            for (int q = 0; q < kTaps; ++q)
                if (r + kTaps + q < stop) {
                    nx[q] = Ch::load(xp + static_cast<size_t>(q) * a.ld_x);
                    nd[q] = Ch::load(dp + static_cast<size_t>(q) * ga.ld_du);
                }
#pragma unroll
            for (int q = 0; q < kTaps; ++q) {
                const int t = r + q;
                float (&cur)[CH] = win[(q + 3) & 3], (&dv)[CH] = dvw[(q + 3) & 3];
                float v[CH];
                const bool real = t < stop;
                Ch::widen(rx[q], cur);
                Ch::widen(rd[q], dv);
                taps<CH>(w, bias, win[q], win[(q + 1) & 3], win[(q + 2) & 3], cur, v);
                if (kSilu) {
#pragma unroll
                    for (int e = 0; e < CH; ++e) {
                        const float sg = ssm_sigmoid(v[e]);
                        dv[e] *= sg * fmaf(v[e], 1.f - sg, 1.f);
                    }
                }
#pragma unroll
                for (int e = 0; e < CH; ++e) dv[e] = real ? dv[e] : 0.f;
                if (t < hi) {
#pragma unroll
                    for (int e = 0; e < CH; ++e) {
                        dw[0][e] = fmaf(dv[e], win[q][e], dw[0][e]);
                        dw[1][e] = fmaf(dv[e], win[(q + 1) & 3][e], dw[1][e]);
                        dw[2][e] = fmaf(dv[e], win[(q + 2) & 3][e], dw[2][e]);
                        dw[3][e] = fmaf(dv[e], cur[e], dw[3][e]);
                        db[e] += dv[e];
                    }
                }
                const int s = t - (kTaps - 1);  // the row whose dx is complete
                if (s >= lo && s < hi) {
                    float out[CH];
                    // dx_s = W_3 dv_s + W_2 dv_{s+1} + W_1 dv_{s+2} + W_0 dv_{s+3}
                    const float (&d0)[CH] = dvw[q], (&d1)[CH] = dvw[(q + 1) & 3], (&d2)[CH] = dvw[(q + 2) & 3];
#pragma unroll
                    for (int e = 0; e < CH; ++e)
                        out[e] = fmaf(w[3][e], d0[e], fmaf(w[2][e], d1[e], fmaf(w[1][e], d2[e], w[0][e] * dv[e])));
                    Ch::store(op + (static_cast<long long>(s) - lo) * ga.ld_dx, out);
                }
            }
        }
        lo = hi;
    }
    float* to = ga.part + (static_cast<size_t>(by) * a.channels + c) * 5;
#pragma unroll
    for (int e = 0; e < CH; ++e) {
#pragma unroll
        for (int j = 0; j < kTaps; ++j) to[5 * e + j] = dw[j][e];
        to[5 * e + 4] = db[e];
    }
}

// The runs' sums in order: parameters of the convolution (first blocks), then of the gates.
__global__ void __launch_bounds__(256)
    sum_kernel(const float* __restrict__ part, const float* __restrict__ gate_part, int runs, int gate_blocks, int channels, int H,
               int conv_blocks, float* __restrict__ dweight, float* __restrict__ dbias, float* __restrict__ da,
               float* __restrict__ ddelta_bias) {
    __shared__ float red[8][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool conv = static_cast<int>(blockIdx.x) < conv_blocks;
    const int i = (conv ? blockIdx.x : blockIdx.x - conv_blocks) * 32 + lane, n = conv ? channels * 5 : H * 2;
    const float* src = conv ? part : gate_part;
    const int count = conv ? runs : gate_blocks;
    float v = 0.f;
    if (i < n) {
        int k = warp;
        for (; k + 56 < count; k += 64) {  // eight loads in flight
            float t[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) t[q] = src[static_cast<size_t>(k + 8 * q) * n + i];
#pragma unroll
            for (int q = 0; q < 8; ++q) v += t[q];
        }
        for (; k < count; k += 8) v += src[static_cast<size_t>(k) * n + i];
    }
    red[warp][lane] = v;
    __syncthreads();
    if (warp || i >= n) return;
    v = ((red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane])) + ((red[4][lane] + red[5][lane]) + (red[6][lane] + red[7][lane]));
    if (conv) {
        const int c = i / 5, j = i - 5 * c;
        if (j < kTaps) dweight[kTaps * c + j] = v;
        else if (dbias) dbias[c] = v;
    } else if (i & 1) {
        ddelta_bias[i >> 1] = v;
    } else {
        da[i >> 1] = v;
    }
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 152;
    return n;
}

// Rows per block: enough blocks for `per_sm` on every SM, at least `least` rows (three more are read).
int run_rows(long long rows, int blocks_x, int per_sm, int least) {
    const long long want = (static_cast<long long>(per_sm) * sm_count() + blocks_x - 1) / blocks_x;
    const long long run = (rows + want - 1) / want;
    return static_cast<int>(run < least ? least : run);
}

ConvArgs conv_args(const Seqs& seqs, int channels, int H, int ch_per_thread, int per_sm, int least) {
    ConvArgs a{};
    a.seqs = seqs;
    a.rows = seqs.rows();
    a.channels = channels;
    a.H = H;
    a.conv_blocks_x = (channels + ch_per_thread * kThreads - 1) / (ch_per_thread * kThreads);
    a.run = run_rows(a.rows, a.conv_blocks_x, per_sm, least);
    a.conv_blocks_y = static_cast<int>((a.rows + a.run - 1) / a.run);
    return a;
}

constexpr int kGradPerSm = 3, kGradLeast = 16;

struct GradPlan {
    ConvArgs c;
    size_t part, gate_part;  // floats
};
GradPlan grad_plan(const Seqs& seqs, int channels, int H, int ch_per_thread) {
    GradPlan p;
    p.c = conv_args(seqs, channels, H, ch_per_thread, kGradPerSm, kGradLeast);
    p.c.gate_blocks = static_cast<int>((p.c.rows + kGateRows - 1) / kGateRows);
    p.part = static_cast<size_t>(p.c.conv_blocks_y) * channels * 5;
    p.gate_part = static_cast<size_t>(p.c.gate_blocks) * H * 2;
    return p;
}

gdn2_status sizes(int B, int T, int channels, int H, gdn2_dtype dt, const Seqs& seqs) {
    if ((dt != GDN2_F32 && dt != GDN2_BF16) || B < 0 || T < 0 || channels <= 0 || H <= 0) return GDN2_ERR_INVALID_ARG;
    if (channels % 8 || channels > (1 << 20) || H > 32767 || seqs.rows() >= (1LL << 30)) return GDN2_ERR_UNSUPPORTED;
    return GDN2_OK;
}

gdn2_status row_check(const void* p, long long ld, long long width, size_t esz) {
    if (!p || ld < width) return GDN2_ERR_INVALID_ARG;
    if (ld >= (1LL << 31)) return GDN2_ERR_UNSUPPORTED;
    return aligned_to(p, esz) ? GDN2_OK : GDN2_ERR_MISALIGNED;
}

// The widest word of up to `most` channels that every row of these tensors starts on: projections whose
// rows carry an odd number of heads behind the channels are read in narrower words.
int word(std::initializer_list<Rows> ts, size_t esz, int most) {
    int w = most;
    for (const Rows& t : ts)
        while (w > 1 && (!aligned_to(t.p, esz * w) || t.ld % w)) w >>= 1;
    return w;
}

const int kFakeOffset = 0;

}  // namespace
}  // namespace gdn2

using namespace gdn2;

extern "C" {

gdn2_status gdn2_ssm_prologue(const void* xbc, long long ld_xbc, const void* delta, long long ld_delta,
                              const float* conv_weight, const float* conv_bias, const float* a, const float* delta_bias,
                              float* conv_state, const int32_t* offsets, void* u, void* step, void* g, int B, int T,
                              int channels, int H, int silu, gdn2_dtype dt, void* stream) {
    const Seqs seqs{offsets, B, T};
    gdn2_status st = sizes(B, T, channels, H, dt, seqs);
    if (st != GDN2_OK) return st;
    if (B == 0 || seqs.rows() == 0) return GDN2_OK;  // no tokens: nothing to write, states unchanged
    const size_t esz = dt == GDN2_BF16 ? 2 : 4;
    if ((st = row_check(xbc, ld_xbc, channels, esz)) != GDN2_OK) return st;
    if (!delta || ld_delta < H || !conv_weight || !a || !delta_bias || !u || !step || !g) return GDN2_ERR_INVALID_ARG;
    if (!aligned_to(delta, esz) || !aligned16(conv_weight) || !aligned_to(conv_bias, 4) || !aligned_to(a, 4) ||
        !aligned_to(delta_bias, 4) || !aligned_to(conv_state, 4) || !aligned_to(offsets, 4) || !aligned16(u) || !aligned_to(step, esz) ||
        !aligned_to(g, esz))
        return GDN2_ERR_MISALIGNED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool bf = dt == GDN2_BF16;
    const int ch = word({{xbc, ld_xbc}}, esz, 4);
    ConvArgs c = conv_args(seqs, channels, H, ch, 24, 8);
    c.weight = conv_weight;
    c.bias = conv_bias;
    c.state = conv_state;
    c.a = a;
    c.delta_bias = delta_bias;
    c.ld_x = ld_xbc;
    c.ld_delta = ld_delta;
    const long long gates = (c.rows * H + 4 * kThreads - 1) / (4 * kThreads), conv = (long long)c.conv_blocks_x * c.conv_blocks_y;
    c.gate_blocks = static_cast<int>(gates < 2048 ? gates : 2048);
    const unsigned grid = static_cast<unsigned>(conv + c.gate_blocks);
    auto go = [&](auto kernel, auto zero) {
        using T = decltype(zero);
        kernel<<<grid, kThreads, 0, s>>>(c, static_cast<const T*>(xbc), static_cast<const T*>(delta), static_cast<T*>(u),
                                         static_cast<T*>(step), static_cast<T*>(g));
    };
    using BF = __nv_bfloat16;
    auto pick = [&](auto act) {
        constexpr bool kSilu = decltype(act)::value;
        if (bf) go(ch == 4 ? prologue_kernel<BF, 4, kSilu> : ch == 2 ? prologue_kernel<BF, 2, kSilu> : prologue_kernel<BF, 1, kSilu>, BF{});
        else go(ch == 4 ? prologue_kernel<float, 4, kSilu> : ch == 2 ? prologue_kernel<float, 2, kSilu> : prologue_kernel<float, 1, kSilu>, 0.f);
    };
    if (silu) pick(std::true_type{}); else pick(std::false_type{});
    if (cudaGetLastError() != cudaSuccess) return GDN2_ERR_CUDA;
    if (conv_state) {
        const unsigned n = static_cast<unsigned>(((long long)B * channels + 255) / 256);
        if (bf) window_kernel<<<n, 256, 0, s>>>(seqs, static_cast<const __nv_bfloat16*>(xbc), ld_xbc, conv_state, channels);
        else window_kernel<<<n, 256, 0, s>>>(seqs, static_cast<const float*>(xbc), ld_xbc, conv_state, channels);
        if (cudaGetLastError() != cudaSuccess) return GDN2_ERR_CUDA;
    }
    return GDN2_OK;
}

size_t gdn2_ssm_prologue_backward_workspace_size(int B, int T, int channels, int H, int packed, gdn2_dtype dt) {
    const Seqs seqs{packed ? &kFakeOffset : nullptr, B, T};
    if (sizes(B, T, channels, H, dt, seqs) != GDN2_OK || B == 0 || seqs.rows() == 0) return 0;
    size_t most = 0;  // whatever the word that the rows' alignment allows
    for (int ch = 1; ch <= 4; ch *= 2) {
        const GradPlan p = grad_plan(seqs, channels, H, ch);
        if (p.part + p.gate_part > most) most = p.part + p.gate_part;
    }
    return align_up(sizeof(float) * most, 256);
}

gdn2_status gdn2_ssm_prologue_backward(const void* xbc, long long ld_xbc, const void* delta, long long ld_delta,
                                       const float* conv_weight, const float* conv_bias, const float* a,
                                       const float* delta_bias, const int32_t* offsets, const void* du, long long ld_du,
                                       const void* dstep, const void* dg, void* dxbc, long long ld_dxbc, void* ddelta,
                                       long long ld_ddelta, float* dconv_weight, float* dconv_bias, float* da,
                                       float* ddelta_bias, int B, int T, int channels, int H, int silu, gdn2_dtype dt,
                                       void* workspace, size_t ws_bytes, void* stream) {
    const Seqs seqs{offsets, B, T};
    gdn2_status st = sizes(B, T, channels, H, dt, seqs);
    if (st != GDN2_OK) return st;
    if (!dconv_weight || !da || !ddelta_bias) return GDN2_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (B == 0 || seqs.rows() == 0) {  // sums over no tokens
        const bool ok = cudaMemsetAsync(dconv_weight, 0, sizeof(float) * 4 * channels, s) == cudaSuccess &&
                        (!dconv_bias || cudaMemsetAsync(dconv_bias, 0, sizeof(float) * channels, s) == cudaSuccess) &&
                        cudaMemsetAsync(da, 0, sizeof(float) * H, s) == cudaSuccess &&
                        cudaMemsetAsync(ddelta_bias, 0, sizeof(float) * H, s) == cudaSuccess;
        return ok ? GDN2_OK : GDN2_ERR_CUDA;
    }
    const size_t esz = dt == GDN2_BF16 ? 2 : 4;
    if ((st = row_check(xbc, ld_xbc, channels, esz)) != GDN2_OK || (st = row_check(du, ld_du, channels, esz)) != GDN2_OK ||
        (st = row_check(dxbc, ld_dxbc, channels, esz)) != GDN2_OK)
        return st;
    if (!delta || ld_delta < H || !ddelta || ld_ddelta < H || !conv_weight || !a || !delta_bias || !dstep || !dg)
        return GDN2_ERR_INVALID_ARG;
    if (!aligned_to(delta, esz) || !aligned_to(ddelta, esz) || !aligned16(conv_weight) || !aligned_to(conv_bias, 4) ||
        !aligned_to(a, 4) || !aligned_to(delta_bias, 4) || !aligned_to(offsets, 4) || !aligned_to(dstep, esz) || !aligned_to(dg, esz) ||
        !aligned_to(dconv_weight, 4) || !aligned_to(dconv_bias, 4) || !aligned_to(da, 4) || !aligned_to(ddelta_bias, 4))
        return GDN2_ERR_MISALIGNED;
    const int ch = word({{xbc, ld_xbc}, {du, ld_du}, {dxbc, ld_dxbc}}, esz, 4);
    GradPlan p = grad_plan(seqs, channels, H, ch);
    if (!workspace || ws_bytes < gdn2_ssm_prologue_backward_workspace_size(B, T, channels, H, offsets != nullptr, dt))
        return GDN2_ERR_WORKSPACE;
    if (!aligned16(workspace)) return GDN2_ERR_MISALIGNED;
    p.c.weight = conv_weight;
    p.c.bias = conv_bias;
    p.c.a = a;
    p.c.delta_bias = delta_bias;
    p.c.ld_x = ld_xbc;
    p.c.ld_delta = ld_delta;
    float* part = static_cast<float*>(workspace);
    const ConvGradArgs ga{p.c, ld_du, ld_dxbc, ld_ddelta, part, part + p.part};
    const unsigned grid = static_cast<unsigned>(p.c.conv_blocks_x * p.c.conv_blocks_y + p.c.gate_blocks);
    auto go = [&](auto kernel, auto zero) {
        using T = decltype(zero);
        kernel<<<grid, kThreads, 0, s>>>(ga, static_cast<const T*>(xbc), static_cast<const T*>(delta), static_cast<const T*>(du),
                                         static_cast<const T*>(dstep), static_cast<const T*>(dg), static_cast<T*>(dxbc),
                                         static_cast<T*>(ddelta));
    };
    using BF = __nv_bfloat16;
    auto pick = [&](auto act) {
        constexpr bool kSilu = decltype(act)::value;
        if (dt == GDN2_BF16)
            go(ch == 4 ? prologue_grad_kernel<BF, 4, kSilu> : ch == 2 ? prologue_grad_kernel<BF, 2, kSilu> : prologue_grad_kernel<BF, 1, kSilu>, BF{});
        else
            go(ch == 4 ? prologue_grad_kernel<float, 4, kSilu> : ch == 2 ? prologue_grad_kernel<float, 2, kSilu> : prologue_grad_kernel<float, 1, kSilu>, 0.f);
    };
    if (silu) pick(std::true_type{}); else pick(std::false_type{});
    if (cudaGetLastError() != cudaSuccess) return GDN2_ERR_CUDA;
    const int conv_blocks = (channels * 5 + 31) / 32, gate_blocks = (H * 2 + 31) / 32;
    sum_kernel<<<conv_blocks + gate_blocks, 256, 0, s>>>(ga.part, ga.gate_part, p.c.conv_blocks_y, p.c.gate_blocks, channels, H,
                                                         conv_blocks, dconv_weight, dconv_bias, da, ddelta_bias);
    return cudaGetLastError() == cudaSuccess ? GDN2_OK : GDN2_ERR_CUDA;
}

}  // extern "C"
