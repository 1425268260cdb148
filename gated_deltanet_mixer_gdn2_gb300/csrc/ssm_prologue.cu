// ssm_prologue.cu -- what stands between the selective state-space mixer's projection and its scan:
//     v_t = bias + sum_{j=0..3} W_j x_{t-3+j},  u = silu(v)       (depthwise, causal within its sequence)
//     step = softplus(delta + delta_bias),      g = a step
// and the gradients of all of it. Both directions stream rows once and are bound by HBM.
#include <initializer_list>

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
#pragma unroll
        for (int i = 0; i < CH; ++i) x[i] = to_f32(r.v[i]);
    }
    __device__ static void store(T* p, const float (&x)[CH]) {
        Raw r;
#pragma unroll
        for (int i = 0; i < CH; ++i) r.v[i] = from_f32<T>(x[i]);
        *reinterpret_cast<Raw*>(p) = r;
    }
};

struct ConvArgs {
    Seqs seqs;
    long long rows;
    int channels, H, silu, run;  // run: token rows per block
    const float *weight, *bias, *state;  // [channels][4], [channels] or null, [B][3][channels] or null
    const float *a, *delta_bias;         // [H]
    long long ld_x, ld_delta;
    int conv_blocks_x, conv_blocks_y;    // channel blocks, runs
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

// One thread holds CH channels and walks down a run of rows with the window of the last three in
// registers; kAhead rows are in flight at a time. Rows between sequences (none, with sound offsets) are
// skipped. The blocks past the conv's compute the gates.
template <typename T, int CH>
__global__ void __launch_bounds__(kThreads)
    prologue_kernel(ConvArgs a, const T* __restrict__ x, const T* __restrict__ delta, T* __restrict__ u, T* __restrict__ step,
                    T* __restrict__ g) {
    constexpr int kAhead = 8;
    const int conv_blocks = a.conv_blocks_x * a.conv_blocks_y;
    if (static_cast<int>(blockIdx.x) >= conv_blocks) {
        const long long n = a.rows * a.H, stride = static_cast<long long>(gridDim.x - conv_blocks) * kThreads;
        for (long long i = (blockIdx.x - conv_blocks) * static_cast<long long>(kThreads) + threadIdx.x; i < n; i += stride) {
            const long long r = i / a.H;
            const int h = static_cast<int>(i - r * a.H);
            const float st = ssm_softplus(to_f32(delta[r * a.ld_delta + h]) + a.delta_bias[h]);
            step[i] = from_f32<T>(st);
            g[i] = from_f32<T>(a.a[h] * st);
        }
        return;
    }
    const int by = blockIdx.x / a.conv_blocks_x, bx = blockIdx.x - by * a.conv_blocks_x;
    const int c = CH * (bx * kThreads + threadIdx.x);
    if (c >= a.channels) return;
    float w[CH][kTaps], bias[CH];
#pragma unroll
    for (int e = 0; e < CH; ++e) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(a.weight) + c + e);
        w[e][0] = v.x; w[e][1] = v.y; w[e][2] = v.z; w[e][3] = v.w;
        bias[e] = a.bias ? __ldg(a.bias + c + e) : 0.f;
    }
    const int r0 = by * a.run, r1 = static_cast<int>(min(static_cast<long long>(r0) + a.run, a.rows));
    float win[kTaps - 1][CH];
    int end = r0;
    bool in = false;
    for (int rb = r0; rb < r1; rb += kAhead) {
        typename Chan<T, CH>::Raw raw[kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; ++q)
            if (rb + q < r1) raw[q] = Chan<T, CH>::load(x + static_cast<size_t>(rb + q) * a.ld_x + c);
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            const int r = rb + q;
            if (r >= r1) break;
            if (r >= end) {  // into another sequence (uniform over the block)
                int seq, start;
                in = find_row(a.seqs, r, seq, start, end);
                if (in) window_before<T, CH>(a, x, c, r, start, seq, win);
                else end = r + 1;
            }
            float cur[CH], out[CH];
            Chan<T, CH>::widen(raw[q], cur);
#pragma unroll
            for (int e = 0; e < CH; ++e) {
                float v = fmaf(w[e][0], win[0][e], bias[e]);
                v = fmaf(w[e][1], win[1][e], v);
                v = fmaf(w[e][2], win[2][e], v);
                v = fmaf(w[e][3], cur[e], v);
                out[e] = a.silu ? v * ssm_sigmoid(v) : v;
                win[0][e] = win[1][e];
                win[1][e] = win[2][e];
                win[2][e] = cur[e];
            }
            if (in) Chan<T, CH>::store(u + static_cast<size_t>(r) * a.channels + c, out);
        }
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

constexpr int kGateRows = 64;  // token rows of one gate block

struct ConvGradArgs {
    ConvArgs c;
    long long ld_du, ld_dx, ld_ddelta;
    int gate_blocks;
    float *part, *gate_part;  // [runs][channels][5]; [gate blocks][H][2]
};

// dv_t = du_t silu'(v_t);  dx_s = sum_j W_j dv_{s+3-j};  dW_j = sum_t dv_t x_{t-3+j};  dbias = sum_t dv_t.
// One thread walks down a run of rows of CH channels with the last three x and dv in registers: at row
// r it forms dv_r and, from it and the three before, dx_{r-3}. The three rows after the run (of its last
// sequence) are formed again here for its own dx and belong to the next run's sums. Sums of a run go
// to `part`; sum_kernel adds the runs in order.
template <typename T, int CH>
__global__ void __launch_bounds__(kThreads)
    prologue_grad_kernel(ConvGradArgs ga, const T* __restrict__ x, const T* __restrict__ delta, const T* __restrict__ du,
                         const T* __restrict__ dstep, const T* __restrict__ dg, T* __restrict__ dx, T* __restrict__ ddelta) {
    constexpr int kAhead = 8;
    const ConvArgs& a = ga.c;
    const int conv_blocks = a.conv_blocks_x * a.conv_blocks_y;
    if (static_cast<int>(blockIdx.x) >= conv_blocks) {
        __shared__ float red[kThreads / 32][32][2];
        const int blk = blockIdx.x - conv_blocks, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const long long lo = static_cast<long long>(blk) * kGateRows, hi = min(lo + kGateRows, a.rows);
        for (int h0 = 0; h0 < a.H; h0 += 32) {
            const int h = h0 + lane;
            float sa = 0.f, sb = 0.f;
            if (h < a.H) {
                const float av = a.a[h], bv = a.delta_bias[h];
                for (long long r = lo + warp; r < hi; r += kThreads / 32) {
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
    const int by = blockIdx.x / a.conv_blocks_x, bx = blockIdx.x - by * a.conv_blocks_x;
    const int c = CH * (bx * kThreads + threadIdx.x);
    if (c >= a.channels) return;
    float w[CH][kTaps], bias[CH], dw[CH][kTaps] = {}, db[CH] = {};
#pragma unroll
    for (int e = 0; e < CH; ++e) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(a.weight) + c + e);
        w[e][0] = v.x; w[e][1] = v.y; w[e][2] = v.z; w[e][3] = v.w;
        bias[e] = a.bias ? __ldg(a.bias + c + e) : 0.f;
    }
    const int rows = static_cast<int>(a.rows);
    const int r0 = by * a.run, r1 = min(r0 + a.run, rows);
    float win[kTaps - 1][CH], dvw[kTaps - 1][CH];  // x and dv of rows r-3, r-2, r-1
#pragma unroll
    for (int j = 0; j < kTaps - 1; ++j)
#pragma unroll
        for (int e = 0; e < CH; ++e) win[j][e] = dvw[j][e] = 0.f;
    int start = r0, end = r0;
    bool in = false;
    // dx of row s from dvw (rows s .. s+2) and the row after, `last` (zeros past the sequence)
    auto put = [&](int s, const float (&last)[CH]) {
        float out[CH];
#pragma unroll
        for (int e = 0; e < CH; ++e)
            out[e] = fmaf(w[e][3], dvw[0][e], fmaf(w[e][2], dvw[1][e], fmaf(w[e][1], dvw[2][e], w[e][0] * last[e])));
        Chan<T, CH>::store(dx + static_cast<size_t>(s) * ga.ld_dx + c, out);
    };
    auto push = [&](const float (&v)[CH]) {
#pragma unroll
        for (int e = 0; e < CH; ++e) {
            dvw[0][e] = dvw[1][e];
            dvw[1][e] = dvw[2][e];
            dvw[2][e] = v[e];
        }
    };
    const float zero[CH] = {};
    // the last (up to) three rows of a sequence have no rows after them; `upto`: the row after its last
    auto flush = [&](int upto) {
#pragma unroll
        for (int j = 0; j < kTaps - 1; ++j) {
            const int s = upto - (kTaps - 1) + j;
            if (s >= max(start, r0) && s < r1) put(s, zero);
            push(zero);
        }
    };
    const int stop = min(r1 + kTaps - 1, rows);
    bool open = false;  // a sequence whose last dx rows are still to come
    for (int rb = r0; rb < stop; rb += kAhead) {
        typename Chan<T, CH>::Raw rx[kAhead], rd[kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; ++q)
            if (rb + q < stop) {
                rx[q] = Chan<T, CH>::load(x + static_cast<size_t>(rb + q) * a.ld_x + c);
                rd[q] = Chan<T, CH>::load(du + static_cast<size_t>(rb + q) * ga.ld_du + c);
            }
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            const int r = rb + q;
            if (r >= stop) break;
            if (r >= end) {
                if (open) flush(end);
                open = false;
                if (r >= r1) break;  // the rows after the run are another sequence's
                int seq;
                in = find_row(a.seqs, r, seq, start, end);
                if (in) {
                    window_before<T, CH>(a, x, c, r, start, seq, win);
                    open = true;
                } else {
                    end = r + 1;
                }
            }
            if (!in) continue;
            float cur[CH], dv[CH];
            Chan<T, CH>::widen(rx[q], cur);
            Chan<T, CH>::widen(rd[q], dv);
            const bool own = r < r1;
#pragma unroll
            for (int e = 0; e < CH; ++e) {
                float v = fmaf(w[e][0], win[0][e], bias[e]);
                v = fmaf(w[e][1], win[1][e], v);
                v = fmaf(w[e][2], win[2][e], v);
                v = fmaf(w[e][3], cur[e], v);
                if (a.silu) {
                    const float sg = ssm_sigmoid(v);
                    dv[e] *= sg * fmaf(v, 1.f - sg, 1.f);
                }
                if (own) {
                    dw[e][0] = fmaf(dv[e], win[0][e], dw[e][0]);
                    dw[e][1] = fmaf(dv[e], win[1][e], dw[e][1]);
                    dw[e][2] = fmaf(dv[e], win[2][e], dw[e][2]);
                    dw[e][3] = fmaf(dv[e], cur[e], dw[e][3]);
                    db[e] += dv[e];
                }
                win[0][e] = win[1][e];
                win[1][e] = win[2][e];
                win[2][e] = cur[e];
            }
            if (r - (kTaps - 1) >= max(start, r0)) put(r - (kTaps - 1), dv);
            push(dv);
        }
    }
    if (open) {
        if (end <= stop) flush(end);  // the sequence ends within what was read
    }
    float* to = ga.part + (static_cast<size_t>(by) * a.channels + c) * 5;
#pragma unroll
    for (int e = 0; e < CH; ++e) {
#pragma unroll
        for (int j = 0; j < kTaps; ++j) to[5 * e + j] = dw[e][j];
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
    if (i < n)
        for (int k = warp; k < count; k += 8) v += src[static_cast<size_t>(k) * n + i];
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

ConvArgs conv_args(const Seqs& seqs, int channels, int H, int silu, int ch_per_thread, int per_sm, int least) {
    ConvArgs a{};
    a.seqs = seqs;
    a.rows = seqs.rows();
    a.channels = channels;
    a.H = H;
    a.silu = silu ? 1 : 0;
    a.conv_blocks_x = (channels + ch_per_thread * kThreads - 1) / (ch_per_thread * kThreads);
    a.run = run_rows(a.rows, a.conv_blocks_x, per_sm, least);
    a.conv_blocks_y = static_cast<int>((a.rows + a.run - 1) / a.run);
    return a;
}

constexpr int kGradPerSm = 4, kGradLeast = 16;

struct GradPlan {
    ConvArgs c;
    int gate_blocks;
    size_t part, gate_part;  // floats
};
GradPlan grad_plan(const Seqs& seqs, int channels, int H, int silu, int ch_per_thread) {
    GradPlan p;
    p.c = conv_args(seqs, channels, H, silu, ch_per_thread, kGradPerSm, kGradLeast);
    p.gate_blocks = static_cast<int>((p.c.rows + kGateRows - 1) / kGateRows);
    p.part = static_cast<size_t>(p.c.conv_blocks_y) * channels * 5;
    p.gate_part = static_cast<size_t>(p.gate_blocks) * H * 2;
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
    const int ch = word({{xbc, ld_xbc}}, esz, bf ? 8 : 4);
    ConvArgs c = conv_args(seqs, channels, H, silu, ch, 16, 8);
    c.weight = conv_weight;
    c.bias = conv_bias;
    c.state = conv_state;
    c.a = a;
    c.delta_bias = delta_bias;
    c.ld_x = ld_xbc;
    c.ld_delta = ld_delta;
    const long long gates = (c.rows * H + 4 * kThreads - 1) / (4 * kThreads), conv = (long long)c.conv_blocks_x * c.conv_blocks_y;
    const unsigned grid = static_cast<unsigned>(conv + (gates < 4096 ? gates : 4096));
    auto go = [&](auto kernel, auto zero) {
        using T = decltype(zero);
        kernel<<<grid, kThreads, 0, s>>>(c, static_cast<const T*>(xbc), static_cast<const T*>(delta), static_cast<T*>(u),
                                         static_cast<T*>(step), static_cast<T*>(g));
    };
    using BF = __nv_bfloat16;
    if (bf) go(ch == 8 ? prologue_kernel<BF, 8> : ch == 4 ? prologue_kernel<BF, 4> : ch == 2 ? prologue_kernel<BF, 2> : prologue_kernel<BF, 1>, BF{});
    else go(ch == 4 ? prologue_kernel<float, 4> : ch == 2 ? prologue_kernel<float, 2> : prologue_kernel<float, 1>, 0.f);
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
        const GradPlan p = grad_plan(seqs, channels, H, 1, ch);
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
    GradPlan p = grad_plan(seqs, channels, H, silu, ch);
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
    const ConvGradArgs ga{p.c, ld_du, ld_dxbc, ld_ddelta, p.gate_blocks, part, part + p.part};
    const unsigned grid = static_cast<unsigned>(p.c.conv_blocks_x * p.c.conv_blocks_y + p.gate_blocks);
    auto go = [&](auto kernel, auto zero) {
        using T = decltype(zero);
        kernel<<<grid, kThreads, 0, s>>>(ga, static_cast<const T*>(xbc), static_cast<const T*>(delta), static_cast<const T*>(du),
                                         static_cast<const T*>(dstep), static_cast<const T*>(dg), static_cast<T*>(dxbc),
                                         static_cast<T*>(ddelta));
    };
    using BF = __nv_bfloat16;
    if (dt == GDN2_BF16) go(ch == 4 ? prologue_grad_kernel<BF, 4> : ch == 2 ? prologue_grad_kernel<BF, 2> : prologue_grad_kernel<BF, 1>, BF{});
    else go(ch == 4 ? prologue_grad_kernel<float, 4> : ch == 2 ? prologue_grad_kernel<float, 2> : prologue_grad_kernel<float, 1>, 0.f);
    if (cudaGetLastError() != cudaSuccess) return GDN2_ERR_CUDA;
    const int conv_blocks = (channels * 5 + 31) / 32, gate_blocks = (H * 2 + 31) / 32;
    sum_kernel<<<conv_blocks + gate_blocks, 256, 0, s>>>(ga.part, ga.gate_part, p.c.conv_blocks_y, p.gate_blocks, channels, H,
                                                         conv_blocks, dconv_weight, dconv_bias, da, ddelta_bias);
    return cudaGetLastError() == cudaSuccess ? GDN2_OK : GDN2_ERR_CUDA;
}

}  // extern "C"
