// ssm_scan.cu -- the selective state-space scan and its gradients on CUDA cores, any dtype and every supported shape
// (entry points, argument checks and the choice of the kernel family: ssm_api.cu).
//
// Per sequence and head, on a state H in R^{N x P}, with a scalar log-decay g_t <= 0, a step s_t, keys
// B_t and readouts C_t (R^N, shared by the heads of a group) and values x_t (R^P):
//     H_t = e^{g_t} H_{t-1} + s_t B_t x_t^T,        y_t = H_t^T C_t + D x_t.
// The recurrence is linear with a scalar decay, so a sequence splits into units of tokens: every unit's
// own contribution from a zero state (walk_kernel, increments), a walk over the units that turns them
// into the states at the units' starts (chain_kernel), and the units again from those states.
#include "ssm_common.cuh"

namespace gdn2 {
namespace {

constexpr int kWalkTile = 16;     // tokens staged at a time
constexpr int kWalkCols = 32;     // state columns (of P) of one block, one per lane
constexpr int kWalkThreads = 128; // four warps, each a quarter of N

enum Walk { kForward, kIncrement, kIncrementBack };

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}

// Token by token through one unit, the state in registers: warp w holds rows w N/4 .. of 32 columns.
// Four multiply-adds per state element and token (two passes' worth where a sequence is cut) and one shared-memory read
// of B and C for four rows bound it: 8 x 512 tokens, 24 heads of 64 values, N = 128, fp32: 262 us, 10 TFLOP/s; the sum over N crosses the four warps once per tile of tokens.
//   kForward        y, from the unit's starting state (units > 1 per sequence: `states`, else s0)
//   kIncrement      the unit's state from zero into `states`, its total log-decay into `decay`
//   kIncrementBack  the adjoint's: sum_i e^{g_1 + .. + g_i} C_i dy_i^T (bm = C, x = dy, no step)
struct WalkArgs {
    Seqs seqs;
    int unit, use_states, H, G, P;
    Rows x, b, c;
    const void *step, *g;
    const float *d, *s0;
    float* s1;
    void* y;
    float *states, *decay;
};

template <typename T, int NPT, int kMode>
__device__ __forceinline__ void walk_block(const WalkArgs& a, int cols) {
    const Rows xr = a.x, br = a.b, cr = a.c;
    const T *__restrict__ step = static_cast<const T*>(a.step), *__restrict__ g = static_cast<const T*>(a.g);
    T* __restrict__ y = static_cast<T*>(a.y);
    const float *dskip = a.d, *s0 = a.s0;
    float *s1 = a.s1, *states = a.states, *decay = a.decay;
    const int H = a.H, G = a.G, P = a.P;
    constexpr int N = 4 * NPT;
    __shared__ float sB[kWalkTile][N], sC[kMode == kForward ? kWalkTile : 1][N], sX[kWalkTile][kWalkCols];
    __shared__ float sY[kMode == kForward ? kWalkTile : 1][4][kWalkCols], sS[kWalkTile];
    __shared__ float2 sA[kWalkTile];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.y, grp = h / (H / G), p = cols * kWalkCols + lane;
    Unit u;
    if (!find_unit(a.seqs, a.unit, blockIdx.x, u)) return;
    const bool col = p < P;
    const size_t plane = static_cast<size_t>(N) * P;
    const size_t mine = static_cast<size_t>(warp * NPT) * P + (col ? p : 0);

    float st[NPT];
    {
        const float* from = nullptr;
        if (kMode == kForward)
            from = a.use_states ? states + (static_cast<size_t>(blockIdx.x) * H + h) * plane
                              : (s0 ? s0 + (static_cast<size_t>(u.seq) * H + h) * plane : nullptr);
#pragma unroll
        for (int i = 0; i < NPT; ++i) st[i] = from && col ? from[mine + static_cast<size_t>(i) * P] : 0.f;
    }
    const T* xp = static_cast<const T*>(xr.p) + static_cast<size_t>(h) * P;
    const T* bp = static_cast<const T*>(br.p) + static_cast<size_t>(grp) * N;
    const T* cp = static_cast<const T*>(cr.p) + static_cast<size_t>(grp) * N;
    const float dk = kMode == kForward && dskip ? dskip[h] : 0.f;
    float gsum = 0.f;
    const int tiles = (u.len + kWalkTile - 1) / kWalkTile;
    for (int k = 0; k < tiles; ++k) {
        const int t0 = (kMode == kIncrementBack ? tiles - 1 - k : k) * kWalkTile, n = min(kWalkTile, u.len - t0);
        const size_t row = static_cast<size_t>(u.row) + t0;
        __syncthreads();  // the previous tile has been used
        for (int i = tid; i < n * (N / 4); i += kWalkThreads) {
            const int t = i / (N / 4), c = 4 * (i - t * (N / 4));
            *reinterpret_cast<float4*>(&sB[t][c]) = load4(bp + (row + t) * br.ld + c);
            if (kMode == kForward) *reinterpret_cast<float4*>(&sC[t][c]) = load4(cp + (row + t) * cr.ld + c);
        }
        for (int i = tid; i < n * kWalkCols; i += kWalkThreads) {
            const int t = i / kWalkCols, c = i - t * kWalkCols;
            const int pc = cols * kWalkCols + c;
            sX[t][c] = pc < P ? to_f32(xp[(row + t) * xr.ld + pc]) : 0.f;
        }
        if (tid < n) {
            const float gt = ssm_gate(to_f32(g[(row + tid) * H + h]));
            sA[tid] = ssm_decay(gt);
            sS[tid] = kMode == kIncrementBack ? gt : to_f32(step[(row + tid) * H + h]);
            if (kMode == kIncrement) sY[0][0][tid] = gt;
        }
        __syncthreads();
        if (kMode != kForward && tid == 0)
            for (int t = 0; t < n; ++t) gsum += kMode == kIncrement ? sY[0][0][t] : sS[t];
        for (int q = 0; q < n; ++q) {
            const int t = kMode == kIncrementBack ? n - 1 - q : q;
            const float2 al = sA[t];
            const float e = al.x, lo = al.y, x = kMode == kIncrementBack ? sX[t][lane] : sX[t][lane] * sS[t];
            float acc0 = 0.f, acc1 = 0.f;
#pragma unroll
            for (int i = 0; i < NPT; i += 4) {
                const float4 b = *reinterpret_cast<const float4*>(&sB[t][warp * NPT + i]);
                if (kMode == kIncrementBack) {
                    const float u0 = fmaf(b.x, x, st[i]), u1 = fmaf(b.y, x, st[i + 1]);
                    const float u2 = fmaf(b.z, x, st[i + 2]), u3 = fmaf(b.w, x, st[i + 3]);
                    st[i] = fmaf(e, u0, lo * u0);
                    st[i + 1] = fmaf(e, u1, lo * u1);
                    st[i + 2] = fmaf(e, u2, lo * u2);
                    st[i + 3] = fmaf(e, u3, lo * u3);
                } else {
                    st[i] = fmaf(e, st[i], fmaf(lo, st[i], b.x * x));
                    st[i + 1] = fmaf(e, st[i + 1], fmaf(lo, st[i + 1], b.y * x));
                    st[i + 2] = fmaf(e, st[i + 2], fmaf(lo, st[i + 2], b.z * x));
                    st[i + 3] = fmaf(e, st[i + 3], fmaf(lo, st[i + 3], b.w * x));
                }
                if (kMode == kForward) {
                    const float4 c = *reinterpret_cast<const float4*>(&sC[t][warp * NPT + i]);
                    acc0 = fmaf(c.x, st[i], acc0);
                    acc1 = fmaf(c.y, st[i + 1], acc1);
                    acc0 = fmaf(c.z, st[i + 2], acc0);
                    acc1 = fmaf(c.w, st[i + 3], acc1);
                }
            }
            if (kMode == kForward) sY[t][warp][lane] = acc0 + acc1;
        }
        if (kMode == kForward) {
            __syncthreads();
            for (int i = tid; i < n * kWalkCols; i += kWalkThreads) {
                const int t = i / kWalkCols, c = i - t * kWalkCols, pc = cols * kWalkCols + c;
                const float v = (sY[t][0][c] + sY[t][1][c]) + (sY[t][2][c] + sY[t][3][c]);
                if (pc < P) y[((row + t) * H + h) * P + pc] = from_f32<T>(fmaf(dk, sX[t][c], v));
            }
        }
    }
    if (!col && kMode == kForward) return;
    if (kMode == kForward) {
        if (s1 && u.k == u.count - 1) {
            float* to = s1 + (static_cast<size_t>(u.seq) * H + h) * plane;
#pragma unroll
            for (int i = 0; i < NPT; ++i) to[mine + static_cast<size_t>(i) * P] = st[i];
        }
    } else {
        if (col) {
            float* to = states + (static_cast<size_t>(blockIdx.x) * H + h) * plane;
#pragma unroll
            for (int i = 0; i < NPT; ++i) to[mine + static_cast<size_t>(i) * P] = st[i];
        }
        if (tid == 0 && cols == 0) decay[static_cast<size_t>(blockIdx.x) * H + h] = gsum;
    }
}

template <typename T, int NPT, int kMode>
__global__ void __launch_bounds__(kWalkThreads) walk_kernel(WalkArgs a) {
    walk_block<T, NPT, kMode>(a, blockIdx.z);
}
// Both directions' increments in one launch: the adjoint's beside the state's.
template <typename T, int NPT>
__global__ void __launch_bounds__(kWalkThreads) walk_pair_kernel(WalkArgs f, WalkArgs b) {
    const int half = gridDim.z / 2;
    if (blockIdx.z < half) walk_block<T, NPT, kIncrement>(f, blockIdx.z);
    else walk_block<T, NPT, kIncrementBack>(b, blockIdx.z - half);
}

// From the units' increments to the states at their starts (back: the adjoints at their ends), in
// place: four state elements per thread, eight units' loads in flight. Memory-bound: each increment is
// read once and replaced once. `last`: the state after the final unit (back: before the first). The two directions
// of a gradient run in one launch.
__global__ void __launch_bounds__(256) chain_kernel(Seqs seqs, int unit, int room, ChainJob j0, ChainJob j1, int H, int plane4) {
    const ChainJob& job = blockIdx.y < H ? j0 : j1;
    const float* first = job.first;
    float *last = job.last, *states = job.states;
    const float* decay = job.decay;
    const int back = job.back;
    const int e = blockIdx.x * blockDim.x + threadIdx.x, h = blockIdx.y % H, seq = blockIdx.z;
    int start, len;
    const long long before = units_before(seqs, unit, seq);
    seqs.span(seq, start, len);
    const int count = Seqs::held(before, Seqs::units_of(len, unit), room), base = static_cast<int>(before);
    if (e >= plane4) return;
    const size_t at = (static_cast<size_t>(seq) * H + h) * plane4 + e;
    float4 cur = first ? reinterpret_cast<const float4*>(first)[at] : make_float4(0.f, 0.f, 0.f, 0.f);
    float4* st = reinterpret_cast<float4*>(states);
    constexpr int kAhead = 8;
    for (int k0 = 0; k0 < count; k0 += kAhead) {
        float4 inc[kAhead];
        float gs[kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; ++q)
            if (k0 + q < count) {
                const size_t uh = static_cast<size_t>(base + (back ? count - 1 - k0 - q : k0 + q)) * H + h;
                inc[q] = st[uh * plane4 + e];
                gs[q] = decay[uh];
            }
#pragma unroll
        for (int q = 0; q < kAhead; ++q)
            if (k0 + q < count) {
                const size_t uh = static_cast<size_t>(base + (back ? count - 1 - k0 - q : k0 + q)) * H + h;
                st[uh * plane4 + e] = cur;
                const float a = expf(gs[q]);
                cur.x = fmaf(a, cur.x, inc[q].x);
                cur.y = fmaf(a, cur.y, inc[q].y);
                cur.z = fmaf(a, cur.z, inc[q].z);
                cur.w = fmaf(a, cur.w, inc[q].w);
            }
    }
    if (last) reinterpret_cast<float4*>(last)[at] = cur;
}

// ---------------------------------------------------------------------------------------------
// gradients, one block per (unit of 32 tokens, group, share of the group's heads)

constexpr int kGradUnit = 32;
constexpr int kGradThreads = 256;

template <int N, int PB>
struct GradSmem {
    static constexpr int NS = N + 4, XS = PB + 4, Q = kGradUnit, PS = Q + 1;
    float b[Q][NS], c[Q][NS], x[Q][XS], dy[Q][XS], h0[N][XS], dh[N][XS];
    float p1[Q][PS], sw[Q][PS], pf[Q][PS];
    float g[Q], eL[Q], wend[Q], stp[Q];     // log-decay, e^L, e^{L_end - L}, step
    float rows[Q], cols[Q], q[Q], v[Q], du[Q];
    float red[kGradThreads / 32][2];
};

// Within a unit, with L the inclusive sum of g, W_ij = e^{L_i - L_j} (i >= j), S = C B^T, R = dY X^T,
// H0 the state before the unit and dH the adjoint of the state after it:
//   dC_i = sum_j R_ij W_ij s_j B_j + e^{L_i} H0 dY_i          (summed over the group's heads)
//   dB_j = s_j (sum_i R_ij W_ij C_i + e^{L_end - L_j} dH x_j)  (summed over the group's heads)
//   U_j  = sum_i S_ij W_ij dY_i + e^{L_end - L_j} dH^T B_j;  dx_j = s_j U_j + D dY_j;  ds_j = x_j . U_j
//   dg_t = sum_{i >= t > j} S R W s + sum_{i >= t} e^{L_i} dY_i . H0^T C_i
//          + sum_{j < t} s_j e^{L_end - L_j} x_j . dH^T B_j + e^{L_end} <dH, H0>
// The double sum is a suffix sum of (row sums - column sums) of one matrix held in fp32, so what
// cancels in it cancels exactly. Every exponent is <= 0, and each is a sum of just the gates that it stands for: as a difference
// of two L it would lose the digits of ordinary decays behind strong ones (fp32, twelve resets before them: 3.5e-4).
// Multiply-adds from shared memory bound it, two blocks per SM: fp32, 1364 packed tokens, 8 heads of 64 values, N = 64,
// 50 us of a call's 74 (walk of both directions 21, chain 10, sums 4), 28000 of each scheduler's 64000 cycles issuing.
// Value columns in halves of 32, which let three blocks share an SM, took 79 us instead of 75.
template <typename T, int N, int PB>
__global__ void __launch_bounds__(kGradThreads, N <= 64 ? 2 : 1)
    grad_kernel(Seqs seqs, Rows xr, Rows br, Rows cr, Rows dyr, const T* __restrict__ step, const T* __restrict__ g,
                const float* __restrict__ dskip, const float* __restrict__ h0, const float* __restrict__ dhe,
                RowsOut dxr, RowsOut dbr, RowsOut dcr, T* __restrict__ dstep, T* __restrict__ dg,
                float* __restrict__ part, float* __restrict__ dd_part, int H, int G, int P, int heads, int splits,
                long long rows) {
    extern __shared__ float4 smem_f4[];
    using Sm = GradSmem<N, PB>;
    Sm& s = *reinterpret_cast<Sm*>(smem_f4);
    constexpr int Q = kGradUnit;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int grp = blockIdx.y / splits, split = blockIdx.y - grp * splits, per = H / G;
    Unit u;
    const bool real = find_unit(seqs, Q, blockIdx.x, u);
    const int h_lo = grp * per + split * heads, h_hi = min(h_lo + heads, (grp + 1) * per);
    const int n = real ? u.len : 0;
    if (n == 0) {  // no such unit, or an empty sequence: nothing but its share of dD
        if (dd_part)
            for (int h = h_lo + tid; h < h_hi; h += kGradThreads) dd_part[static_cast<size_t>(blockIdx.x) * H + h] = 0.f;
        return;
    }
    const size_t row = u.row;
    {
        const T* bp = static_cast<const T*>(br.p) + static_cast<size_t>(grp) * N;
        const T* cp = static_cast<const T*>(cr.p) + static_cast<size_t>(grp) * N;
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = tid; i < Q * (N / 4); i += kGradThreads) {
            const int t = i / (N / 4), c = 4 * (i - t * (N / 4));
            *reinterpret_cast<float4*>(&s.b[t][c]) = t < n ? load4(bp + (row + t) * br.ld + c) : zero;
            *reinterpret_cast<float4*>(&s.c[t][c]) = t < n ? load4(cp + (row + t) * cr.ld + c) : zero;
        }
    }
    __syncthreads();
    // this thread's entries (pi, pj + 8 e) of the Q x Q matrices: neighbouring lanes read neighbouring rows of b and x, whose
    // stride of 4 floats past a multiple of 32 keeps them in different banks
    const int pi = tid >> 3, pj = tid & 7;
    float sc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < N; k += 4) {
        const float4 c = *reinterpret_cast<const float4*>(&s.c[pi][k]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float4 b = *reinterpret_cast<const float4*>(&s.b[pj + 8 * e][k]);
            sc[e] += c.x * b.x + c.y * b.y + c.z * b.z + c.w * b.w;
        }
    }
    // tiles of 4 tokens x 4 states (n0 + N / 4 e) of dB and dC: lanes run over the states, so token rows are read once for
    // all of them and the rows of H and A without bank conflicts (four neighbouring states per thread took 4 times as long)
    constexpr int kTiles = 8 * (N / 4), kPer = (kTiles + kGradThreads - 1) / kGradThreads;
    float ab[kPer][4][4] = {}, ac[kPer][4][4] = {};

    const size_t plane = static_cast<size_t>(N) * P;
    for (int h = h_lo; h < h_hi; ++h) {
        const size_t uh = static_cast<size_t>(blockIdx.x) * H + h;
        if (warp == 0) {
            const float gt = lane < n ? ssm_gate(to_f32(g[(row + lane) * H + h])) : 0.f;
            float L = gt, rest = gt;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const float v = __shfl_up_sync(0xffffffffu, L, d), w = __shfl_down_sync(0xffffffffu, rest, d);
                if (lane >= d) L += v;
                if (lane + d < 32) rest += w;
            }
            rest = __shfl_down_sync(0xffffffffu, rest, 1);
            s.g[lane] = gt;
            s.eL[lane] = expf(L);
            s.wend[lane] = lane < 31 ? expf(rest) : 1.f;
            s.stp[lane] = lane < n ? to_f32(step[(row + lane) * H + h]) : 0.f;
            s.rows[lane] = s.cols[lane] = s.q[lane] = s.v[lane] = s.du[lane] = 0.f;
        }
        const float dk = dskip ? dskip[h] : 0.f;
        float e_acc = 0.f, dd_acc = 0.f, wp[4];  // wp: W of this thread's entries
        for (int p0 = 0; p0 < P; p0 += PB) {
            const T* xp = static_cast<const T*>(xr.p) + static_cast<size_t>(h) * P + p0;
            const T* dyp = static_cast<const T*>(dyr.p) + static_cast<size_t>(h) * P + p0;
            const int pw = min(PB, P - p0);
            const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int i = tid; i < Q * (PB / 4); i += kGradThreads) {
                const int t = i / (PB / 4), c = 4 * (i - t * (PB / 4));
                const bool in = t < n && c < pw;
                *reinterpret_cast<float4*>(&s.x[t][c]) = in ? load4(xp + (row + t) * xr.ld + c) : zero;
                *reinterpret_cast<float4*>(&s.dy[t][c]) = in ? load4(dyp + (row + t) * dyr.ld + c) : zero;
            }
            for (int i = tid; i < N * (PB / 4); i += kGradThreads) {
                const int t = i / (PB / 4), c = 4 * (i - t * (PB / 4));
                const size_t at = uh * plane + static_cast<size_t>(t) * P + p0 + c;
                const float4 a = c < pw ? *reinterpret_cast<const float4*>(h0 + at) : zero;
                const float4 b = c < pw ? *reinterpret_cast<const float4*>(dhe + at) : zero;
                *reinterpret_cast<float4*>(&s.h0[t][c]) = a;
                *reinterpret_cast<float4*>(&s.dh[t][c]) = b;
                e_acc += a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w;
            }
            __syncthreads();
            if (p0 == 0) {
                float sum = 0.f;  // of the gates behind token j up to token pi, eight at a time
#pragma unroll
                for (int e = 3; e >= 0; --e) {
                    float eight = 0.f;
#pragma unroll
                    for (int k = pj + 8 * e + 1, d = 0; d < 8; ++k, ++d) eight += k <= pi ? s.g[k] : 0.f;
                    sum += eight;
                    wp[e] = pi >= pj + 8 * e ? expf(sum) : 0.f;
                }
            }
            {
                float r[4] = {0.f, 0.f, 0.f, 0.f};
                for (int k = 0; k < PB; k += 4) {
                    const float4 a = *reinterpret_cast<const float4*>(&s.dy[pi][k]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float4 b = *reinterpret_cast<const float4*>(&s.x[pj + 8 * e][k]);
                        r[e] += a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w;
                    }
                }
                float rs = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = pj + 8 * e;
                    const float p1 = r[e] * wp[e] * s.stp[j], pf = pi > j ? sc[e] * p1 : 0.f;
                    s.p1[pi][j] = p1;
                    s.sw[pi][j] = sc[e] * wp[e];
                    s.pf[pi][j] = pf;
                    rs += pf;
                }
#pragma unroll
                for (int d = 1; d < 8; d <<= 1) rs += __shfl_xor_sync(0xffffffffu, rs, d);
                if ((tid & 7) == 0) s.rows[pi] += rs;
            }
            __syncthreads();
            if (warp == 0) {
                float cs = 0.f;
                for (int i = 0; i < Q; ++i) cs += s.pf[i][lane];
                s.cols[lane] += cs;
            }
#pragma unroll
            for (int m = 0; m < kPer; ++m) {
                const int tile = tid + m * kGradThreads;
                if (kTiles % kGradThreads == 0 || tile < kTiles) {
                    const int n0 = tile % (N / 4), t0 = 4 * (tile / (N / 4));
                    for (int j = 0; j < t0 + 4; ++j) {  // p1 is lower triangular
                        float b[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) b[e] = s.b[j][n0 + N / 4 * e];
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const float w = s.p1[t0 + t][j];
#pragma unroll
                            for (int e = 0; e < 4; ++e) ac[m][t][e] += w * b[e];
                        }
                    }
                    for (int j = t0; j < Q; ++j) {
                        float c[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) c[e] = s.c[j][n0 + N / 4 * e];
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const float z = s.p1[j][t0 + t];
#pragma unroll
                            for (int e = 0; e < 4; ++e) ab[m][t][e] += z * c[e];
                        }
                    }
                    float xb[4][4] = {}, xc[4][4] = {};
                    for (int k = 0; k < PB; k += 4) {
                        float4 hh[4], dd[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            hh[e] = *reinterpret_cast<const float4*>(&s.h0[n0 + N / 4 * e][k]);
                            dd[e] = *reinterpret_cast<const float4*>(&s.dh[n0 + N / 4 * e][k]);
                        }
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const float4 a = *reinterpret_cast<const float4*>(&s.dy[t0 + t][k]);
                            const float4 b = *reinterpret_cast<const float4*>(&s.x[t0 + t][k]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                xc[t][e] += a.x * hh[e].x + a.y * hh[e].y + a.z * hh[e].z + a.w * hh[e].w;
                                xb[t][e] += b.x * dd[e].x + b.y * dd[e].y + b.z * dd[e].z + b.w * dd[e].w;
                            }
                        }
                    }
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const float wc = s.eL[t0 + t], wb = s.stp[t0 + t] * s.wend[t0 + t];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            ac[m][t][e] = fmaf(wc, xc[t][e], ac[m][t][e]);
                            ab[m][t][e] = fmaf(wb, xb[t][e], ab[m][t][e]);
                        }
                    }
                }
            }
            // dx and the per-token sums over P: PB / 4 lanes per token
            constexpr int kQuads = PB / 4, kRows = kGradThreads / kQuads, kPerT = Q / kRows;
            const int pq = 4 * (tid % kQuads);
            float a2[kPerT][4] = {}, a3[kPerT][4] = {};
            for (int k = 0; k < N; ++k) {  // A and H are read once for all of a thread's tokens
                const float4 d = *reinterpret_cast<const float4*>(&s.dh[k][pq]);
                const float4 e = *reinterpret_cast<const float4*>(&s.h0[k][pq]);
#pragma unroll
                for (int m = 0; m < kPerT; ++m) {
                    const float bv = s.b[tid / kQuads + m * kRows][k], cv = s.c[tid / kQuads + m * kRows][k];
                    a2[m][0] += bv * d.x; a2[m][1] += bv * d.y; a2[m][2] += bv * d.z; a2[m][3] += bv * d.w;
                    a3[m][0] += cv * e.x; a3[m][1] += cv * e.y; a3[m][2] += cv * e.z; a3[m][3] += cv * e.w;
                }
            }
#pragma unroll
            for (int m = 0; m < kPerT; ++m) {
                const int j = tid / kQuads + m * kRows;
                float a1[4] = {};
                for (int i = j; i < Q; ++i) {
                    const float w = s.sw[i][j];
                    const float4 d = *reinterpret_cast<const float4*>(&s.dy[i][pq]);
                    a1[0] += w * d.x; a1[1] += w * d.y; a1[2] += w * d.z; a1[3] += w * d.w;
                }
                const float we = s.wend[j], sj = s.stp[j];
                float du = 0.f, v = 0.f, q = 0.f, out[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float xv = s.x[j][pq + e], dv = s.dy[j][pq + e], U = a1[e] + we * a2[m][e];
                    out[e] = sj * U + dk * dv;
                    du += xv * U;
                    v += xv * a2[m][e];
                    q += dv * a3[m][e];
                    dd_acc += xv * dv;
                }
                if (j < n && pq < pw) {
                    T* to = static_cast<T*>(dxr.p) + (row + j) * dxr.ld + static_cast<size_t>(h) * P + p0 + pq;
#pragma unroll
                    for (int e = 0; e < 4; ++e) to[e] = from_f32<T>(out[e]);
                }
#pragma unroll
                for (int d = 1; d < kQuads; d <<= 1) {
                    du += __shfl_xor_sync(0xffffffffu, du, d);
                    v += __shfl_xor_sync(0xffffffffu, v, d);
                    q += __shfl_xor_sync(0xffffffffu, q, d);
                }
                if (pq == 0) {
                    s.du[j] += du;
                    s.v[j] += sj * we * v;
                    s.q[j] += s.eL[j] * q;
                }
            }
            __syncthreads();
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            e_acc += __shfl_xor_sync(0xffffffffu, e_acc, d);
            dd_acc += __shfl_xor_sync(0xffffffffu, dd_acc, d);
        }
        if (lane == 0) {
            s.red[warp][0] = e_acc;
            s.red[warp][1] = dd_acc;
        }
        __syncthreads();
        if (warp == 0) {
            float E = 0.f, D = 0.f;
#pragma unroll
            for (int w = 0; w < kGradThreads / 32; ++w) {
                E += s.red[w][0];
                D += s.red[w][1];
            }
            if (dd_part && lane == 0) dd_part[uh] = D;
            float suf = s.rows[lane] - s.cols[lane] + s.q[lane], pre = s.v[lane];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const float a = __shfl_down_sync(0xffffffffu, suf, d), b = __shfl_up_sync(0xffffffffu, pre, d);
                if (lane + d < 32) suf += a;
                if (lane >= d) pre += b;
            }
            pre -= s.v[lane];  // j < t only
            if (lane < n) {
                dg[(row + lane) * H + h] = from_f32<T>(suf + pre + s.eL[31] * E);
                dstep[(row + lane) * H + h] = from_f32<T>(s.du[lane]);
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int m = 0; m < kPer; ++m) {
        const int tile = tid + m * kGradThreads;
        if (tile >= kTiles) continue;
        const int n0 = tile % (N / 4), t0 = 4 * (tile / (N / 4));
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (t0 + t >= n) continue;
            const size_t r = row + t0 + t;
            if (splits == 1) {
                T* tb = static_cast<T*>(dbr.p) + r * dbr.ld + static_cast<size_t>(grp) * N + n0;
                T* tc = static_cast<T*>(dcr.p) + r * dcr.ld + static_cast<size_t>(grp) * N + n0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    tb[N / 4 * e] = from_f32<T>(ab[m][t][e]);
                    tc[N / 4 * e] = from_f32<T>(ac[m][t][e]);
                }
            } else {
                const size_t gn = static_cast<size_t>(G) * N, at = (static_cast<size_t>(split) * rows + r) * gn + static_cast<size_t>(grp) * N + n0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    part[at + N / 4 * e] = ab[m][t][e];
                    part[static_cast<size_t>(splits) * rows * gn + at + N / 4 * e] = ac[m][t][e];
                }
            }
        }
    }
}

// dB and dC: the sum of the head shares in a fixed order, then one rounding; rows of no sequence have no shares. dD, by the third row of blocks: the sum over the
// units, one block per head, in a fixed order.
template <typename T>
__global__ void __launch_bounds__(256)
    sums_kernel(Seqs seqs, const float* __restrict__ part, RowsOut dbr, RowsOut dcr, long long rows, int gn, int splits,
                const float* __restrict__ dd_part, float* __restrict__ dd, int units, int H) {
    if (blockIdx.y == 2) {
        __shared__ float red[8];
        const int h = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (!dd || h >= H) return;
        float v = 0.f;
        for (int k = threadIdx.x; k < units; k += 256) v += dd_part[static_cast<size_t>(k) * H + h];
#pragma unroll
        for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        if (lane == 0) red[warp] = v;
        __syncthreads();
        if (threadIdx.x == 0) dd[h] = ((red[0] + red[1]) + (red[2] + red[3])) + ((red[4] + red[5]) + (red[6] + red[7]));
        return;
    }
    const long long i = blockIdx.x * 256LL + threadIdx.x;
    if (splits <= 1 || i >= rows * (gn / 4)) return;
    const long long r = i / (gn / 4);
    long long first, last;
    seqs.covered(first, last);
    if (r < first || r >= last) return;
    const int c = 4 * static_cast<int>(i - r * (gn / 4));
    const float* src = part + (blockIdx.y ? static_cast<size_t>(splits) * rows * gn : 0);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < splits; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(src + (static_cast<size_t>(k) * rows + r) * gn + c);
        a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
    }
    const RowsOut o = blockIdx.y ? dcr : dbr;
    T* to = static_cast<T*>(o.p) + r * o.ld + c;
    to[0] = from_f32<T>(a.x); to[1] = from_f32<T>(a.y); to[2] = from_f32<T>(a.z); to[3] = from_f32<T>(a.w);
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 152;
    return n;
}

// Tokens per unit of the forward walk: each block walks token by token, so only more blocks shorten a call. Sequences
// stay whole where they are that many by themselves or short (the two further launches cost what five tiles of tokens do:
// 77 tokens of 8 heads 25 us either way, 200 tokens 41 -> 25 us), else they are cut until about twelve blocks per SM run,
// into units of whole tiles (fp32, N = 64, 8 heads: 512 tokens 145 us whole, 30 us cut; 4096 tokens 1133 and 90 us).
int walk_unit(const ScanShape& sh) {
    const long long cols = (sh.P + kWalkCols - 1) / kWalkCols, want = 12LL * sm_count();
    const long long per = sh.H * cols, units = (want + per - 1) / per;
    long long len = (sh.seqs.rows() + units - 1) / units;
    len = (len + 15) / 16 * 16;
    const long long whole = sh.seqs.T > 0 ? sh.seqs.T : 1;
    if (len * 5 > whole || sh.seqs.B >= units) return static_cast<int>(whole);
    return static_cast<int>(len);
}

size_t state_floats(const ScanShape& sh, int unit) {
    return static_cast<size_t>(sh.seqs.units(unit)) * sh.H * (static_cast<size_t>(sh.N) * sh.P + 4);
}

WalkArgs walk_args(const ScanShape& sh, int unit, Rows x, Rows b, Rows c, const ScanIn& in, float* states, float* decay) {
    WalkArgs a{};
    a.seqs = sh.seqs;
    a.unit = unit;
    a.H = sh.H; a.G = sh.G; a.P = sh.P;
    a.x = x; a.b = b; a.c = c;
    a.step = in.step; a.g = in.g;
    a.states = states;
    a.decay = decay;
    return a;
}

// One walk, or with `b` the increments of both directions.
template <typename T, int NPT>
cudaError_t walk(const ScanShape& sh, int mode, const WalkArgs& a, const WalkArgs* b, cudaStream_t s) {
    const unsigned units = static_cast<unsigned>(sh.seqs.units(a.unit)), cols = (sh.P + kWalkCols - 1) / kWalkCols;
    if (b) walk_pair_kernel<T, NPT><<<dim3(units, sh.H, 2 * cols), kWalkThreads, 0, s>>>(a, *b);
    else if (mode == kForward) walk_kernel<T, NPT, kForward><<<dim3(units, sh.H, cols), kWalkThreads, 0, s>>>(a);
    else walk_kernel<T, NPT, kIncrement><<<dim3(units, sh.H, cols), kWalkThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t walk_n(const ScanShape& sh, int mode, const WalkArgs& a, const WalkArgs* b, cudaStream_t s) {
    switch (sh.N) {
        case 16: return walk<T, 4>(sh, mode, a, b, s);
        case 32: return walk<T, 8>(sh, mode, a, b, s);
        case 64: return walk<T, 16>(sh, mode, a, b, s);
        case 128: return walk<T, 32>(sh, mode, a, b, s);
        default: return walk<T, 64>(sh, mode, a, b, s);
    }
}

cudaError_t walk_any(const ScanShape& sh, int mode, const WalkArgs& a, const WalkArgs* b, cudaStream_t s) {
    return sh.dt == GDN2_BF16 ? walk_n<__nv_bfloat16>(sh, mode, a, b, s) : walk_n<float>(sh, mode, a, b, s);
}

// Heads per block of the gradient kernel: all of a group while that alone gives two blocks per SM.
int grad_heads(const ScanShape& sh) {
    const int per = sh.H / sh.G;
    const long long blocks = sh.seqs.units(kGradUnit) * sh.G, want = 2LL * sm_count();
    if (blocks >= want) return per;
    const long long splits = (want + blocks - 1) / blocks;
    return splits >= per ? 1 : static_cast<int>((per + splits - 1) / splits);
}

struct BwdWs {
    size_t h0, dh, decay, decay_b, part, dd, total;
    int heads, splits;
};
BwdWs bwd_ws(const ScanShape& sh) {
    BwdWs w;
    const size_t units = static_cast<size_t>(sh.seqs.units(kGradUnit)), uh = units * sh.H;
    const size_t st = uh * sh.N * sh.P;
    w.heads = grad_heads(sh);
    w.splits = (sh.H / sh.G + w.heads - 1) / w.heads;
    w.h0 = 0;
    w.dh = w.h0 + st;
    w.decay = w.dh + st;
    w.decay_b = w.decay + align_up(uh, 4);
    w.dd = w.decay_b + align_up(uh, 4);
    w.part = w.dd + align_up(uh, 4);
    w.total = w.part + (w.splits > 1 ? 2ull * w.splits * sh.seqs.rows() * sh.G * sh.N : 0);
    return w;
}

template <typename T, int N, int PB>
cudaError_t grad(const ScanShape& sh, const ScanIn& in, const ScanGrads& gr, float* ws, const BwdWs& w, cudaStream_t s) {
    const size_t smem = sizeof(GradSmem<N, PB>);
    static_assert(sizeof(GradSmem<N, PB>) <= 227 * 1024, "gradient kernel shared memory");
    cudaError_t e = cudaFuncSetAttribute(grad_kernel<T, N, PB>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    grad_kernel<T, N, PB><<<dim3(static_cast<unsigned>(sh.seqs.units(kGradUnit)), sh.G * w.splits), kGradThreads, smem, s>>>(
        sh.seqs, in.x, in.bm, in.cm, gr.dy, static_cast<const T*>(in.step), static_cast<const T*>(in.g), in.d, ws + w.h0,
        ws + w.dh, gr.dx, gr.dbm, gr.dcm, static_cast<T*>(gr.dstep), static_cast<T*>(gr.dg), ws + w.part,
        gr.dd ? ws + w.dd : nullptr, sh.H, sh.G, sh.P, w.heads, w.splits, sh.seqs.rows());
    return cudaGetLastError();
}

template <typename T>
cudaError_t grad_n(const ScanShape& sh, const ScanIn& in, const ScanGrads& gr, float* ws, const BwdWs& w, cudaStream_t s) {
    switch (sh.N) {
        case 16: return grad<T, 16, 64>(sh, in, gr, ws, w, s);
        case 32: return grad<T, 32, 64>(sh, in, gr, ws, w, s);
        case 64: return grad<T, 64, 64>(sh, in, gr, ws, w, s);
        case 128: return grad<T, 128, 64>(sh, in, gr, ws, w, s);
        default: return grad<T, 256, 32>(sh, in, gr, ws, w, s);
    }
}

}  // namespace

cudaError_t launch_ssm_chain(const ScanShape& sh, int unit, const ChainJob* jobs, int n, cudaStream_t s) {
    const int plane4 = sh.N * sh.P / 4;
    chain_kernel<<<dim3((plane4 + 255) / 256, n * sh.H, sh.seqs.B), 256, 0, s>>>(sh.seqs, unit, static_cast<int>(sh.seqs.units(unit)),
                                                                                     jobs[0], jobs[n - 1], sh.H, plane4);
    return cudaGetLastError();
}

cudaError_t launch_ssm_grad_sums(const ScanShape& sh, const ScanGrads& gr, const float* part, int splits, const float* dd_part, int units,
                                 cudaStream_t s) {
    if (splits <= 1 && !gr.dd) return cudaSuccess;
    const long long rows = sh.seqs.rows(), n = splits > 1 ? (rows * (sh.G * sh.N / 4) + 255) / 256 : 0;
    const dim3 grid(static_cast<unsigned>(n > sh.H ? n : sh.H), 3);
    auto go = [&](auto kernel) { kernel<<<grid, 256, 0, s>>>(sh.seqs, part, gr.dbm, gr.dcm, rows, sh.G * sh.N, splits, dd_part, gr.dd, units, sh.H); };
    if (sh.dt == GDN2_BF16) go(sums_kernel<__nv_bfloat16>);
    else go(sums_kernel<float>);
    return cudaGetLastError();
}

size_t ssm_simt_fwd_workspace(const ScanShape& sh) {
    const int unit = walk_unit(sh);
    return unit >= sh.seqs.T ? 0 : align_up(sizeof(float) * state_floats(sh, unit), 256);
}

cudaError_t launch_ssm_simt_fwd(const ScanShape& sh, const ScanIn& in, void* y, float* s1, void* ws, cudaStream_t s) {
    const int unit = walk_unit(sh);
    const bool cut = unit < sh.seqs.T;
    float* states = static_cast<float*>(ws);
    float* decay = cut ? states + static_cast<size_t>(sh.seqs.units(unit)) * sh.H * sh.N * sh.P : nullptr;
    cudaError_t e;
    WalkArgs a = walk_args(sh, unit, in.x, in.bm, in.cm, in, states, decay);
    if (cut) {
        if ((e = walk_any(sh, kIncrement, a, nullptr, s)) != cudaSuccess) return e;
        const ChainJob job{in.s0, nullptr, states, decay, 0};
        if ((e = launch_ssm_chain(sh, unit, &job, 1, s)) != cudaSuccess) return e;
    }
    a.use_states = cut;
    a.d = in.d;
    a.s0 = in.s0;
    a.s1 = s1;
    a.y = y;
    return walk_any(sh, kForward, a, nullptr, s);
}

size_t ssm_simt_bwd_workspace(const ScanShape& sh) { return align_up(sizeof(float) * bwd_ws(sh).total, 256); }

cudaError_t launch_ssm_simt_bwd(const ScanShape& sh, const ScanIn& in, const ScanGrads& gr, void* wsv, cudaStream_t s) {
    float* ws = static_cast<float*>(wsv);
    const BwdWs w = bwd_ws(sh);
    const WalkArgs fwd = walk_args(sh, kGradUnit, in.x, in.bm, in.cm, in, ws + w.h0, ws + w.decay);
    const WalkArgs bwd = walk_args(sh, kGradUnit, gr.dy, in.cm, in.cm, in, ws + w.dh, ws + w.decay_b);
    cudaError_t e = walk_any(sh, kIncrement, fwd, &bwd, s);
    if (e != cudaSuccess) return e;
    const ChainJob jobs[2] = {{in.s0, nullptr, ws + w.h0, ws + w.decay, 0}, {gr.ds1, gr.ds0, ws + w.dh, ws + w.decay_b, 1}};
    if ((e = launch_ssm_chain(sh, kGradUnit, jobs, 2, s)) != cudaSuccess) return e;
    e = sh.dt == GDN2_BF16 ? grad_n<__nv_bfloat16>(sh, in, gr, ws, w, s) : grad_n<float>(sh, in, gr, ws, w, s);
    if (e != cudaSuccess) return e;
    return launch_ssm_grad_sums(sh, gr, ws + w.part, w.splits, ws + w.dd, static_cast<int>(sh.seqs.units(kGradUnit)), s);
}

}  // namespace gdn2
