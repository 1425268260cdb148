// ssm_tc_grad.cu -- the gradients of the selective state-space scan on the tensor cores, one block per (chunk of
// 128 tokens, group, share of the group's heads), from the state H before the chunk and the adjoint A after it
// (ssm_tc_walk.cu). With W_ij = e^{L_i - L_j} (i >= j), S = C B^T, R = dY X^T, s the steps:
//     dC   = (R W s) B + e^{L} dY H^T            dB   = (R W s)^T C + (s e^{L_end - L} X) A^T      (sum over heads)
//     U    = (S W)^T dY + e^{L_end - L} (B A)    dx_j = s_j U_j + D dY_j,   ds_j = x_j . U_j
//     dg_t = sum_{i >= t > j} S R W s + sum_{i >= t} e^{L_i} dY_i . (C H)_i
//            + sum_{j < t} s_j e^{L_end - L_j} x_j . (B A)_j + e^{L_end} <A, H>
// The pair matrices are formed transposed (a row j of X per thread), so that (R W s)^T and (S W)^T are written back
// over R^T in tensor memory as operands; dB and dC accumulate there over the block's heads, so the sum over a
// group's heads costs nothing. The double sum of dg is a suffix sum of (row sums - column sums) of one fp32
// matrix: what cancels in it cancels exactly.
// Roundings: the pair matrices and the saved states are bf16 operands, once each, of products whose sums are fp32; e^L dY
// and X~, which meet the states, enter as two bf16 parts (2^-16), so that no term of dB or dC has two roundings to bf16 before
// the result's own. Row and column sums, dstep's and dg's sums and dD are fp32 throughout.
// 4 x 2048 tokens, 32 heads of 64 values, N = 128: 96 us of a call's 143 (walk 41, sums 7; CUDA cores: 1870); with one part of e^L dY
// and X~ 90 us, and dC off by 2.9e-3 of its norm instead of 2.4e-3 where given states are most of it (its own rounding: 1.7e-3). A
// head of a chunk takes about 10700 cycles: the pair matrices, 4500 (a fifth of it the sums across lanes), the state's
// shares 1800, U 800, dx 2000, each waiting for the one before; its 60 products take 4200 to issue, beside the rest. What limits
// overlapping two heads is tensor memory: dB, dC and one pair matrix take three quarters of it.
#include <cuda_fp16.h>

#include "ssm_tc.cuh"

namespace gdn2 {
namespace {

// shared memory
namespace sg {
constexpr uint32_t B = 0;                         // 2 tiles
constexpr uint32_t C = B + 2 * kTileBytes;        // 2 tiles
constexpr uint32_t X = C + 2 * kTileBytes;        // 2 stages; X~'s first part replaces X
constexpr uint32_t DY = X + 2 * kTileBytes;       // 2 stages; dx leaves through dY's room
constexpr uint32_t XL = DY + 2 * kTileBytes;      // X~'s second part
constexpr uint32_t H0 = XL + kTileBytes;
constexpr uint32_t DH = H0 + kTileBytes;
constexpr uint32_t P1 = DH + kTileBytes;          // (R W s)^T [j][i]: 2 tiles
constexpr uint32_t GATE = P1 + 2 * kTileBytes;    // 2 stages x {L, s, wend, eL, col}[128]
constexpr uint32_t kGateStage = 5 * 512;
constexpr uint32_t SUM = GATE + 2 * kGateStage;   // a head's {row sums, column sums, v, q, du}[4][128]
constexpr uint32_t RED = SUM + 20 * 512;          // a head's {<A, H>, dD} per warp
constexpr uint32_t BAR = RED + 128;
constexpr uint32_t TOTAL = BAR + 256;
}  // namespace sg
static_assert(sg::TOTAL + 1024 <= 232448, "gradient kernel shared memory");

enum GradBar {
    gBc = 0, gXy = 1, gXyDone = 3, gXyFree = 5, gGate = 7, gGateFree = 9, gHd = 11, gHdFree, gS, gSRead, gR, gTu, gPReady, gDx,
    gURead, gTrFree, gAll, gSumFree, gOut, gDrain = gOut + 2, gBars
};
static_assert(gBars * 8 + 16 <= 256, "barrier room");

// tensor-memory columns: S^T, then each head's R^T and, in its place, per 16 columns 8 packed of (R W s)^T and 8
// of (S W)^T; dB; dC; C H, then in its place, per 16 columns, 8 packed of each part of e^L dY; U
constexpr uint32_t kTR = 0, kTdB = 128, kTdC = 256, kTT = 384, kTU = 448;
constexpr int kGradTc = 640;  // sixteen compute warps, then results, copies, gates, products

struct GradMaps {
    CUtensorMap x, dy, b, c, dx;
};
struct GradTcArgs {
    Seqs seqs;
    int H, G, P, N, heads, splits;
    long long rows;
    const __nv_bfloat16 *step, *g;
    const float* d;
    const uint8_t *h0, *dh;
    __nv_bfloat16 *dx, *db, *dc, *dstep, *dg;
    long long ld_dx, ld_db, ld_dc;
    float *part, *dd_part;
    long long wait_ns;
};

__device__ __forceinline__ float sum_of(uint64_t v) {
    float a, b;
    f32x2_split(v, a, b);
    return a + b;
}
// Pair k of the 16 bf16 values of two 16-byte words, widened.
__device__ __forceinline__ uint64_t pair_of(const uint4 (&v)[2], int k) {
    const uint4& u = v[k >> 2];
    return bf16x2_widen((k & 3) == 0 ? u.x : (k & 3) == 1 ? u.y : (k & 3) == 2 ? u.z : u.w);
}
// A pair times w as two bf16 parts.
__device__ __forceinline__ void scaled_parts(uint32_t u, uint64_t w2, uint32_t& hi, uint32_t& lo) {
    const uint64_t v = mul_f32x2(bf16x2_widen(u), w2);
    hi = bf16x2_narrow(v);
    lo = bf16x2_narrow(sub_f32x2(v, bf16x2_widen(hi)));
}

// Sum over the warp's lanes of each of 32 values: lane l returns the sum of v[l]. Each step halves the values.
__device__ __forceinline__ float transpose_sum(float (&v)[32], int lane) {
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const bool up = lane & d;
#pragma unroll
        for (int k = 0; k < d; ++k) {
            const float keep = up ? v[k + d] : v[k], give = up ? v[k] : v[k + d];
            v[k] = keep + __shfl_xor_sync(0xffffffffu, give, d);
        }
    }
    return v[0];
}

__global__ void __launch_bounds__(kGradTc, 1) grad_tc_kernel(const __grid_constant__ GradMaps maps, const __grid_constant__ GradTcArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + sg::BAR);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + sg::BAR + gBars * 8);
    volatile int* err = reinterpret_cast<volatile int*>(sm + sg::BAR + gBars * 8 + 8);
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    const int grp = blockIdx.x / a.splits, split = blockIdx.x - grp * a.splits, per = a.H / a.G;
    const int h_lo = grp * per + split * a.heads, h_hi = min(h_lo + a.heads, (grp + 1) * per);
    const int pbs = a.P / kCols, NI = uniform((h_hi - h_lo) * pbs);
    Unit u;
    const bool found = find_unit(a.seqs, kQ, blockIdx.y, u);
    if (!found || u.len == 0) {  // no such chunk, or an empty sequence: nothing but its share of dD
        if (a.dd_part)
            for (int h = h_lo + tid; h < h_hi; h += kGradTc) a.dd_part[static_cast<size_t>(blockIdx.y) * a.H + h] = 0.f;
        return;
    }
    const int n = uniform(u.len), row = uniform(u.row);
    const bool tail = n < kQ;
    const long long lim = a.wait_ns;
    const uint32_t tile = a.N * 128;  // bytes of a saved state

    if (tid == 0) {
        for (int i = 0; i < gBars; ++i)
            mbar_init(bars + i, i == gSRead || i == gPReady || i == gURead || i == gOut || i == gOut + 1 ? 16
                                : i == gGateFree || i == gGateFree + 1 || i == gHdFree ? 17 : 1);
        *err = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    if (warp < 16) {
        // ---- row j of the transposed pair matrices (token j): one of their four blocks of 32 columns, and 16 of the
        // 64 value columns, per thread
        const int q = warp & 3, b = warp >> 2, j = 32 * q + lane;
        const uint32_t lane_base = static_cast<uint32_t>(32 * q) << 16, pair = lane_base + kTR + 32 * b, val = lane_base + 16 * b;
        float* const sums = reinterpret_cast<float*>(sm + sg::SUM);
        bool ok = wait_bar(bars + gS, 0, lim, err);
        // This row and block of S^T, kept over the heads in the registers that bf16 would take: fp16 under a power of two
        // that brings its largest entry to 2^14 .. 2^15, so entries down to 2^-29 of that keep 11 bits. It goes into
        // dstep and dg; as bf16 (8 bits) dstep was off by 2.8e-3 of its norm instead of 2.4e-3, for 2 us less.
        uint32_t sp[2][8];
        float unscale = 1.f;
        if (ok) {
            tc_fence_after();
            float x[32], top = 0.f;
            tmem_ld_cols<2>(pair, x);
#pragma unroll
            for (int e = 0; e < 32; ++e) top = fmaxf(top, fabsf(x[e]));
            const int ex = max(static_cast<int>(__float_as_uint(top) >> 23), 15);
            const float scale = __uint_as_float(static_cast<uint32_t>(268 - ex) << 23);
            unscale = __uint_as_float(static_cast<uint32_t>(ex - 14) << 23);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const __half2 v = __floats2half2_rn(x[2 * e] * scale, x[2 * e + 1] * scale);
                sp[e >> 3][e & 7] = *reinterpret_cast<const uint32_t*>(&v);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive1(bars + gSRead);
        }
        auto score = [&](uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); };
        uint64_t e_acc = 0, dd_acc = 0;  // pairs of partial sums
        int pi = 0, h = h_lo;
        for (int it = 0; ok && it < NI; ++it) {
            const int st = it & 1;
            const uint32_t ph = (it >> 1) & 1, ph1 = it & 1;
            const float* arr = reinterpret_cast<const float*>(sm + sg::GATE + st * sg::kGateStage);
            const bool fresh = pi == 0;
            uint8_t *xt = sm + sg::X + st * kTileBytes + j * 128, *yt = sm + sg::DY + st * kTileBytes + j * 128;
            const int cell0 = ((2 * b) ^ (j & 7)) << 4, cell1 = ((2 * b + 1) ^ (j & 7)) << 4;
            if (!(ok = wait_bar(bars + gXy + st, ph, lim, err) && wait_bar(bars + gGate + st, ph, lim, err) && wait_bar(bars + gR, ph1, lim, err))) break;
            tc_fence_after();
            const float Lj = arr[j], sj = arr[128 + j], wej = arr[256 + j], eLj = arr[384 + j];
            float cols = 0.f;
            uint8_t* p1t = sm + sg::P1 + (b >> 1) * kTileBytes + j * 128;
            const float dk = a.d ? __ldg(a.d + h) : 0.f;
            float rsum = 0.f;  // of token i = 32 b + lane, over this warp's rows
            uint32_t m1[2][8] = {};
            if (b < q) {  // every i of the block lies before every j
#pragma unroll
                for (int k = 0; k < 4; ++k) tmem_st8(pair + 8 * k, m1[0]);
            } else {
                const bool off = b > q;
                // Off the diagonal block the decay factors through the start of the column's block, both factors <= 1:
                // an exponential per row and block. On it, an exponential per entry.
                const float rf = off ? ex2_approx(arr[32 * b - 1] - Lj) : 1.f;
                float pf[32];
#pragma unroll
                for (int sub = 0; sub < 2; ++sub) {
                    float x[16];
                    uint32_t m2[8];
                    tmem_ld_cols<1>(pair + 16 * sub, x);
                    if (off) {
                        const uint64_t rf2 = f32x2(rf, rf), sj2 = f32x2(sj, sj), un2 = f32x2(unscale, unscale);
                        uint64_t c2 = 0;
#pragma unroll
                        for (int k4 = 0; k4 < 4; ++k4) {
                            const float4 f = *reinterpret_cast<const float4*>(arr + 512 + 32 * b + 16 * sub + 4 * k4);
                            const uint64_t fv[2] = {f32x2(f.x, f.y), f32x2(f.z, f.w)};
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int k = 2 * k4 + e;
                                const float2 s2 = score(sp[sub][k]);
                                const uint64_t w = mul_f32x2(rf2, fv[e]), S = mul_f32x2(f32x2(s2.x, s2.y), un2);
                                const uint64_t p1 = mul_f32x2(f32x2(x[2 * k], x[2 * k + 1]), mul_f32x2(w, sj2)), pp = mul_f32x2(S, p1);
                                c2 = add_f32x2(c2, pp);
                                f32x2_split(pp, pf[16 * sub + 2 * k], pf[16 * sub + 2 * k + 1]);
                                m1[sub][k] = bf16x2_narrow(p1);
                                m2[k] = bf16x2_narrow(mul_f32x2(S, w));
                            }
                        }
                        float c0, c1;
                        f32x2_split(c2, c0, c1);
                        cols += c0 + c1;
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int i0 = 16 * sub + 2 * k;
                            const float2 f = *reinterpret_cast<const float2*>(arr + 32 * b + i0);
                            float d0, d1, f0, f1;
                            f32x2_split(sub_f32x2(f32x2(f.x, f.y), f32x2(Lj, Lj)), d0, d1);
                            const uint64_t w = f32x2(i0 >= lane ? ex2_approx(d0) : 0.f, i0 + 1 >= lane ? ex2_approx(d1) : 0.f);
                            const float2 s2 = score(sp[sub][k]);
                            const uint64_t S = mul_f32x2(f32x2(s2.x, s2.y), f32x2(unscale, unscale));
                            const uint64_t p1 = mul_f32x2(f32x2(x[2 * k], x[2 * k + 1]), mul_f32x2(w, f32x2(sj, sj)));
                            f32x2_split(mul_f32x2(S, p1), f0, f1);
                            pf[i0] = i0 > lane ? f0 : 0.f;
                            pf[i0 + 1] = i0 + 1 > lane ? f1 : 0.f;
                            cols += pf[i0] + pf[i0 + 1];
                            m1[sub][k] = bf16x2_narrow(p1);
                            m2[k] = bf16x2_narrow(mul_f32x2(S, w));
                        }
                    }
                    tmem_st8(pair + 16 * sub, m1[sub]);
                    tmem_st8(pair + 16 * sub + 8, m2);
                }
                rsum = transpose_sum(pf, lane);
            }
            // the products of the head before have read (R W s) and X~
            if (it && !(ok = wait_bar(bars + gAll, ph1 ^ 1, lim, err))) break;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t(&m)[8] = m1[k >> 1];
                const int e = 4 * (k & 1);
                *reinterpret_cast<uint4*>(p1t + (((4 * (b & 1) + k) ^ (j & 7)) << 4)) = make_uint4(m[e], m[e + 1], m[e + 2], m[e + 3]);
            }
            // the thread's part of the head's sums of token j: column sums, v, q, du
            auto keep = [&](int which, float v) {
                float* to = sums + 512 * which + 128 * b + j;
                *to = fresh ? v : *to + v;
            };
            // the sums of the head before have been used
            if (fresh && it && !(ok = wait_bar(bars + gSumFree, ((it / pbs) & 1) ^ 1, lim, err))) break;
            {
                float* to = sums + 128 * q + 32 * b + lane;
                *to = fresh ? rsum : *to + rsum;
            }
            keep(1, cols);
            // X~: one part in place of X
            const uint4 xr[2] = {*reinterpret_cast<const uint4*>(xt + cell0), *reinterpret_cast<const uint4*>(xt + cell1)};
            const uint4 yr[2] = {*reinterpret_cast<const uint4*>(yt + cell0), *reinterpret_cast<const uint4*>(yt + cell1)};
            uint8_t* xl = sm + sg::XL + j * 128;
            const float wx = sj * wej;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int cell = k ? cell1 : cell0;
                const uint64_t w2 = f32x2(wx, wx);
                uint4 hi, lo;
                scaled_parts(xr[k].x, w2, hi.x, lo.x);
                scaled_parts(xr[k].y, w2, hi.y, lo.y);
                scaled_parts(xr[k].z, w2, hi.z, lo.z);
                scaled_parts(xr[k].w, w2, hi.w, lo.w);
                *reinterpret_cast<uint4*>(xt + cell) = hi;
                *reinterpret_cast<uint4*>(xl + cell) = lo;
            }
            if (!(ok = wait_bar(bars + gTu, ph1, lim, err))) break;
            tc_fence_after();
            {
                // B A in U's columns: its share of dg, then scaled as U's start; C H: its share of dg, then the parts of e^L dY
                uint32_t t[16], c[16];
                tmem_ld16(val + kTU, t);
                tmem_ld16(val + kTT, c);
                tmem_ld_wait();
                uint64_t vs = 0, qs = 0;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint64_t ba = f32x2(__uint_as_float(t[2 * k]), __uint_as_float(t[2 * k + 1]));
                    vs = fma_f32x2(pair_of(xr, k), ba, vs);
                    qs = fma_f32x2(pair_of(yr, k), f32x2(__uint_as_float(c[2 * k]), __uint_as_float(c[2 * k + 1])), qs);
                    float b0, b1;
                    f32x2_split(mul_f32x2(ba, f32x2(wej, wej)), b0, b1);
                    t[2 * k] = __float_as_uint(b0);
                    t[2 * k + 1] = __float_as_uint(b1);
                }
                tmem_st16(val + kTU, t);
                const uint64_t eL2 = f32x2(eLj, eLj);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint4& u = yr[k >> 2];
                    scaled_parts((k & 3) == 0 ? u.x : (k & 3) == 1 ? u.y : (k & 3) == 2 ? u.z : u.w, eL2, c[k], c[8 + k]);
                }
                tmem_st16(val + kTT, c);
                keep(2, sum_of(vs) * wx);
                keep(3, sum_of(qs) * eLj);
            }
            fence_proxy_async_smem();
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive1(bars + gPReady);
            if (!(ok = wait_bar(bars + gHd, ph1, lim, err))) break;
            if (j < a.N) {
                const uint8_t *ht = sm + sg::H0 + j * 128, *dt = sm + sg::DH + j * 128;
                const uint4 hr[2] = {*reinterpret_cast<const uint4*>(ht + cell0), *reinterpret_cast<const uint4*>(ht + cell1)};
                const uint4 ar[2] = {*reinterpret_cast<const uint4*>(dt + cell0), *reinterpret_cast<const uint4*>(dt + cell1)};
#pragma unroll
                for (int k = 0; k < 8; ++k) e_acc = fma_f32x2(pair_of(hr, k), pair_of(ar, k), e_acc);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive1(bars + gHdFree);
            if (!(ok = wait_bar(bars + gDx, ph1, lim, err))) break;
            tc_fence_after();
            {
                float t[16];
                uint64_t du = 0;
                tmem_ld_cols<1>(val + kTU, t);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive1(bars + gURead);
                __nv_bfloat16* to = a.dx + static_cast<size_t>(row + j) * a.ld_dx + static_cast<size_t>(h) * a.P + pi * kCols + 16 * b;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint64_t xv = pair_of(xr, 4 * k + e), yv = pair_of(yr, 4 * k + e), U = f32x2(t[8 * k + 2 * e], t[8 * k + 2 * e + 1]);
                        du = fma_f32x2(xv, U, du);
                        dd_acc = fma_f32x2(xv, yv, dd_acc);
                        w[e] = bf16x2_narrow(fma_f32x2(f32x2(dk, dk), yv, mul_f32x2(f32x2(sj, sj), U)));
                    }
                    const uint4 o = make_uint4(w[0], w[1], w[2], w[3]);
                    if (!tail) *reinterpret_cast<uint4*>(yt + (k ? cell1 : cell0)) = o;
                    else if (j < n) reinterpret_cast<uint4*>(to)[k] = o;
                }
                keep(4, sum_of(du));
            }
            if (++pi == pbs) {
                float es = sum_of(e_acc), ds = sum_of(dd_acc);
#pragma unroll
                for (int d = 16; d; d >>= 1) {
                    es += __shfl_xor_sync(0xffffffffu, es, d);
                    ds += __shfl_xor_sync(0xffffffffu, ds, d);
                }
                if (lane == 0) *reinterpret_cast<float2*>(sm + sg::RED + 8 * warp) = make_float2(es, ds);
                e_acc = dd_acc = 0;
                pi = 0;
                ++h;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive1(bars + gOut + st);
                mbar_arrive1(bars + gGateFree + st);
            }
        }
        // dB and dC: rows j and i, 32 columns per thread
        if (ok) ok = wait_bar(bars + gAll, (NI - 1) & 1, lim, err);
        if (ok && 32 * b < a.N) {
            tc_fence_after();
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
                const int o = k >> 1, c0 = 32 * b + 16 * (k & 1);
                float f[16];
                tmem_ld_cols<1>(lane_base + (o ? kTdC : kTdB) + c0, f);
                const int col = grp * a.N + c0;
                if (j < n) {
                    if (a.splits == 1) {
                        uint4* to = reinterpret_cast<uint4*>((o ? a.dc : a.db) + static_cast<size_t>(row + j) * (o ? a.ld_dc : a.ld_db) + col);
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            to[e] = make_uint4(pack_bf16x2(f[8 * e], f[8 * e + 1]), pack_bf16x2(f[8 * e + 2], f[8 * e + 3]),
                                               pack_bf16x2(f[8 * e + 4], f[8 * e + 5]), pack_bf16x2(f[8 * e + 6], f[8 * e + 7]));
                    } else {
                        const size_t gn = static_cast<size_t>(a.G) * a.N;
                        float4* to = reinterpret_cast<float4*>(a.part + ((static_cast<size_t>(o) * a.splits + split) * a.rows + row + j) * gn + col);
#pragma unroll
                        for (int e = 0; e < 4; ++e) to[e] = make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
                    }
                }
            }
        }
    } else if (warp == 16) {
        // ---- results of an iteration: dx's tile, and at a head's end dg and dstep, four tokens per lane
        const float* sums = reinterpret_cast<const float*>(sm + sg::SUM);
        int pi = 0, h = h_lo;
        for (int it = 0; it < NI; ++it) {
            const int st = it & 1;
            if (!wait_bar(bars + gOut + st, (it >> 1) & 1, lim, err)) break;
            const int pi_done = pi;
            if (++pi < pbs) {
                if (lane == 0 && !tail) {
                    tma_store_3d(&maps.dx, sm + sg::DY + st * kTileBytes, pi_done * kCols, h, row);
                    bulk_commit();
                }
            } else {
                const float* arr = reinterpret_cast<const float*>(sm + sg::GATE + st * sg::kGateStage);
                auto four = [&](int which, float (&v)[4]) {  // the four parts' sum
                    float4 s = reinterpret_cast<const float4*>(sums + 512 * which)[lane];
#pragma unroll
                    for (int k = 1; k < 4; ++k) {
                        const float4 x = reinterpret_cast<const float4*>(sums + 512 * which + 128 * k)[lane];
                        s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
                    }
                    v[0] = s.x; v[1] = s.y; v[2] = s.z; v[3] = s.w;
                };
                float s4[4], c4[4], v4[4], q4[4], d4[4], p4[4];
                four(0, s4);
                four(1, c4);
                four(2, v4);
                four(3, q4);
                four(4, d4);
                const float eEnd = arr[384 + 127];
                float E = 0.f, D = 0.f;
                if (lane < 16) {
                    const float2 r = *reinterpret_cast<const float2*>(sm + sg::RED + 8 * lane);
                    E = r.x;
                    D = r.y;
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive1(bars + gSumFree);  // the next head's sums wait for this
                    if (!tail) {
                        tma_store_3d(&maps.dx, sm + sg::DY + st * kTileBytes, pi_done * kCols, h, row);
                        bulk_commit();
                    }
                }
#pragma unroll
                for (int d = 8; d; d >>= 1) {
                    E += __shfl_xor_sync(0xffffffffu, E, d);
                    D += __shfl_xor_sync(0xffffffffu, D, d);
                }
                E = __shfl_sync(0xffffffffu, E, 0);
                if (a.dd_part && lane == 0) a.dd_part[static_cast<size_t>(blockIdx.y) * a.H + h] = D;
#pragma unroll
                for (int e = 0; e < 4; ++e) s4[e] += q4[e] - c4[e];
                s4[2] += s4[3]; s4[1] += s4[2]; s4[0] += s4[1];
                p4[0] = 0.f; p4[1] = v4[0]; p4[2] = p4[1] + v4[1]; p4[3] = p4[2] + v4[2];
                float suf = s4[0], pre = p4[3] + v4[3];
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const float x = __shfl_down_sync(0xffffffffu, suf, d), y = __shfl_up_sync(0xffffffffu, pre, d);
                    if (lane + d < 32) suf += x;
                    if (lane >= d) pre += y;
                }
                const float after = __shfl_down_sync(0xffffffffu, suf, 1), before = __shfl_up_sync(0xffffffffu, pre, 1);
                const float behind = lane < 31 ? after : 0.f, ahead = (lane ? before : 0.f) + eEnd * E;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = 4 * lane + e;
                    if (t < n) {
                        const size_t at = static_cast<size_t>(row + t) * a.H + h;
                        a.dg[at] = __float2bfloat16_rn((s4[e] + behind) + (p4[e] + ahead));
                        a.dstep[at] = __float2bfloat16_rn(d4[e]);
                    }
                }
                pi = 0;
                ++h;
            }
            if (lane == 0) bulk_wait_read_all();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive1(bars + gXyFree + st);
                mbar_arrive1(bars + gGateFree + st);
            }
        }
        if (lane == 0) bulk_wait_all();
    } else if (warp == 19) {
        // ---- products (rows 96-127 have three blocks of zeros: its scheduler is the least loaded)
        const uint32_t lead = elect_one();
        const uint32_t dk = desc_lo(sb, 16), dm = desc_lo(sb, kTileBytes);
        const uint32_t id_kk = idesc_bf16(128, 128, false, false), id_t = idesc_bf16(128, 64, false, true);
        const uint32_t id_nk = idesc_bf16(128, a.N, false, false), id_nm = idesc_bf16(128, a.N, false, true), id_mm = idesc_bf16(128, a.N, true, true);
        const int ks = a.N / 16;
        auto wait = [&](int bar, uint32_t parity) {
            const bool w = wait_bar(bars + bar, parity, lim, err);
            tc_fence_after();
            return w;
        };
        bool ok = wait(gBc, 0) && (!tail || wait(gGate, 0));
        if (ok) {
            mma_steps<false, kStepK, kStepK, kJumpK, kJumpK>(lead, kTR, dk + (sg::B >> 4), dk + (sg::C >> 4), id_kk, 0, ks);
            commit_by(lead, bars + gS);
        }
        auto pairs = [&](int it) {  // R^T = X dY^T
            const int st = it & 1;
            const uint32_t ph = (it >> 1) & 1, xo = (sg::X + st * kTileBytes) >> 4, yo = (sg::DY + st * kTileBytes) >> 4;
            if (!(wait(gXy + st, ph) && (!tail || wait(gGate + st, ph)))) return false;
            mma_steps<false, kStepK, kStepK, 0, 0>(lead, kTR, dk + xo, dk + yo, id_kk, 0, 4);
            commit_by(lead, bars + gR);
            return true;
        };
        ok = ok && wait(gSRead, 0) && pairs(0);
        for (int it = 0; ok && it < NI; ++it) {
            const int st = it & 1;
            const uint32_t ph1 = it & 1, xo = (sg::X + st * kTileBytes) >> 4, yo = (sg::DY + st * kTileBytes) >> 4;
            if (!(ok = wait(gHd, ph1) && (it == 0 || wait(gURead, ph1 ^ 1)))) break;
            // C H and B A
            mma_steps<false, kStepK, kStepMn, kJumpK, 0>(lead, kTT, dk + (sg::C >> 4), dm + (sg::H0 >> 4), id_t, 0, ks);
            mma_steps<false, kStepK, kStepMn, kJumpK, 0>(lead, kTU, dk + (sg::B >> 4), dm + (sg::DH >> 4), id_t, 0, ks);
            commit_by(lead, bars + gTu);
            if (!(ok = wait(gPReady, ph1))) break;
            // what the block waits for first: U += (S W)^T dY; then dB += (R W s)^T C, the last reader of the pair matrices'
            // room, which the next head's R^T takes; the rest beside the next head's pair matrices
            mma_steps<true, 16, kStepMn, 0, 0>(lead, kTU, kTR + 8, dm + yo, id_t, 1, 8);
            commit_by(lead, bars + gDx);
            mma_steps<true, 16, kStepMn, 0, 0>(lead, kTdB, kTR, dm + (sg::C >> 4), id_nm, it > 0, 8);
            commit_by(lead, bars + gTrFree);
            if (it + 1 < NI && !(ok = wait(gTrFree, ph1) && pairs(it + 1))) break;
            // the states' products first, for the next H and A wait for their room: dB += X~ A^T, dC += (e^L dY) H^T. C H of the next
            // head, which takes the room of e^L dY, waits for that copy
            mma_steps<false, kStepK, kStepK, 0, 0>(lead, kTdB, dk + xo, dk + (sg::DH >> 4), id_nk, 1, 4);
            mma_steps<false, kStepK, kStepK, 0, 0>(lead, kTdB, dk + (sg::XL >> 4), dk + (sg::DH >> 4), id_nk, 1, 4);
            mma_steps<true, 16, kStepK, 0, 0>(lead, kTdC, kTT, dk + (sg::H0 >> 4), id_nk, it > 0, 4);
            mma_steps<true, 16, kStepK, 0, 0>(lead, kTdC, kTT + 8, dk + (sg::H0 >> 4), id_nk, 1, 4);
            commit_by(lead, bars + gHdFree);
            // dC += (R W s) B
            mma_steps<false, kStepMn, kStepMn, 0, 0>(lead, kTdC, dm + (sg::P1 >> 4), dm + (sg::B >> 4), id_mm, 1, 8);
            commit_by(lead, bars + gAll);
            commit_by(lead, bars + gXyDone + st);
        }
        commit_by(lead, bars + gDrain);
        mbar_wait(bars + gDrain, 0, kDefaultWaitNs);
    } else if (warp == 17) {
        // ---- copies
        if (lane == 0) {
            const int halves = a.N / 64;
            mbar_arrive_expect_tx(bars + gBc, kTileBytes * 2 * halves);
            for (int k = 0; k < halves; ++k) {
                tma_load_3d(sm + sg::B + k * kTileBytes, &maps.b, 64 * k, grp, row, bars + gBc);
                tma_load_3d(sm + sg::C + k * kTileBytes, &maps.c, 64 * k, grp, row, bars + gBc);
            }
            int xy = 0, hd = 0;
            auto load_xy = [&](int it) {
                const int st = it & 1, hh = h_lo + it / pbs, pi = it % pbs;
                const uint32_t ph = (it >> 1) & 1;
                if (it >= 2 && !(mbar_wait_or_abort(bars + gXyDone + st, ph ^ 1, lim, err) && mbar_wait_or_abort(bars + gXyFree + st, ph ^ 1, lim, err)))
                    return false;
                mbar_arrive_expect_tx(bars + gXy + st, 2 * kTileBytes);
                tma_load_3d(sm + sg::X + st * kTileBytes, &maps.x, pi * kCols, hh, row, bars + gXy + st);
                tma_load_3d(sm + sg::DY + st * kTileBytes, &maps.dy, pi * kCols, hh, row, bars + gXy + st);
                ++xy;
                return true;
            };
            bool ok = load_xy(0);
            for (int it = 0; ok && it < NI; ++it) {
                // H and A have one buffer: asked for once this block's previous products and sums have read it
                if (it >= 1 && !(ok = mbar_wait_or_abort(bars + gHdFree, (it - 1) & 1, lim, err))) break;
                const size_t at = ((static_cast<size_t>(blockIdx.y) * a.H + h_lo + it / pbs) * pbs + it % pbs) * tile;
                mbar_arrive_expect_tx(bars + gHd, 2 * tile);
                bulk_load(sm + sg::H0, a.h0 + at, tile, bars + gHd);
                bulk_load(sm + sg::DH, a.dh + at, tile, bars + gHd);
                ++hd;
                if (it + 1 < NI) ok = load_xy(it + 1);
            }
            if (!ok) note_failure(err);
            mbar_wait(bars + gBc, 0, kDefaultWaitNs);  // nothing in flight when the block ends
            for (int it = xy > 2 ? xy - 2 : 0; it < xy; ++it) mbar_wait(bars + gXy + (it & 1), (it >> 1) & 1, kDefaultWaitNs);
            if (hd) mbar_wait(bars + gHd, (hd - 1) & 1, kDefaultWaitNs);
        }
    } else {
        // ---- gates: four tokens per lane; and the rows past the sequence cleared
        float gn[4], sn[4];
        auto fetch = [&](int it) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = 4 * lane + e;
                const size_t at = static_cast<size_t>(row + t) * a.H + h_lo + it / pbs;
                gn[e] = t < n ? ssm_gate(__bfloat162float(a.g[at])) * kLog2e : 0.f;
                sn[e] = t < n ? __bfloat162float(a.step[at]) : 0.f;
            }
        };
        fetch(0);
        for (int it = 0; it < NI; ++it) {
            const int st = it & 1;
            const uint32_t ph = (it >> 1) & 1;
            if (it >= 2 && !wait_bar(bars + gGateFree + st, ph ^ 1, lim, err)) break;
            if (tail) {
                const uint4 z = make_uint4(0, 0, 0, 0);
                if (it == 0) {
                    if (!wait_bar(bars + gBc, 0, lim, err)) break;
                    for (int k = 0; k < 4; ++k)
                        for (int i = n * 8 + lane; i < kQ * 8; i += 32) reinterpret_cast<uint4*>(sm + sg::B + k * kTileBytes)[i] = z;
                }
                if (!wait_bar(bars + gXy + st, ph, lim, err)) break;
                for (int i = n * 8 + lane; i < kQ * 8; i += 32) {
                    reinterpret_cast<uint4*>(sm + sg::X + st * kTileBytes)[i] = z;
                    reinterpret_cast<uint4*>(sm + sg::DY + st * kTileBytes)[i] = z;
                }
                fence_proxy_async_smem();
            }
            float* arr = reinterpret_cast<float*>(sm + sg::GATE + st * sg::kGateStage);
            float p[4], sfx[4];
            p[0] = gn[0]; p[1] = p[0] + gn[1]; p[2] = p[1] + gn[2]; p[3] = p[2] + gn[3];
            sfx[3] = 0.f; sfx[2] = gn[3]; sfx[1] = sfx[2] + gn[2]; sfx[0] = sfx[1] + gn[1];
            float pre = p[3], suf = p[3];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const float x = __shfl_up_sync(0xffffffffu, pre, d), y = __shfl_down_sync(0xffffffffu, suf, d);
                if (lane >= d) pre += x;
                if (lane + d < 32) suf += y;
            }
            const float before = __shfl_up_sync(0xffffffffu, pre, 1), after = __shfl_down_sync(0xffffffffu, suf, 1);
            const float lo = lane ? before : 0.f, hi = lane < 31 ? after : 0.f;
            const float start = __shfl_sync(0xffffffffu, lo, lane & ~7);  // L before the 32-token block
            const float4 L = make_float4(lo + p[0], lo + p[1], lo + p[2], lo + p[3]);
            reinterpret_cast<float4*>(arr)[lane] = L;
            reinterpret_cast<float4*>(arr + 128)[lane] = make_float4(sn[0], sn[1], sn[2], sn[3]);
            reinterpret_cast<float4*>(arr + 256)[lane] = exp2_4(make_float4(hi + sfx[0], hi + sfx[1], hi + sfx[2], hi + sfx[3]));
            reinterpret_cast<float4*>(arr + 384)[lane] = exp2_4(L);
            reinterpret_cast<float4*>(arr + 512)[lane] = exp2_4(make_float4(L.x - start, L.y - start, L.z - start, L.w - start));
            __syncwarp();
            if (lane == 0) mbar_arrive1(bars + gGate + st);
            if (it + 1 < NI) fetch(it + 1);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(*tmem_slot, 512);
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 152;
    return n;
}

// Heads per block: the number of waves times (heads + the block's own cost, about a head and a half) is least.
int grad_heads_tc(const ScanShape& sh) {
    const int per = sh.H / sh.G, sms = sm_count();
    const long long chunks = sh.seqs.units(kQ) * sh.G;
    int best = per;
    double cost = 1e30;
    for (int splits = 1; splits <= per; ++splits) {
        const int heads = (per + splits - 1) / splits;
        if ((per + heads - 1) / heads != splits) continue;
        const double waves = static_cast<double>((chunks * splits + sms - 1) / sms);
        const double c = waves * (heads * (sh.P / kCols) + 1.5) * (1 + 0.02 * splits);
        if (c < cost) {
            cost = c;
            best = heads;
        }
    }
    return best;
}

// The walk over chunks: whole sequences while both directions' blocks about fill the SMs, else units of 1024 tokens
// or more whose starting states come from a pass over their increments first.
int walk_unit_tc(const ScanShape& sh) {
    const long long chains = 2LL * sh.seqs.B * sh.H * (sh.P / kCols), sms = sm_count();
    const int whole = (sh.seqs.T + kQ - 1) / kQ * kQ;
    if (10 * chains >= 8 * sms) return whole;
    const long long rows = sh.seqs.rows(), units = (2 * sms * sh.seqs.B + chains - 1) / chains;
    long long len = ((rows + units - 1) / units + kQ - 1) / kQ * kQ;
    if (len < 1024) len = 1024;
    return len >= whole ? whole : static_cast<int>(len);
}

struct BwdTc {
    int unit, heads, splits;
    bool cut;
    size_t h0, dh, dd, part, states, states_b, decay, decay_b, total;  // bytes
};
BwdTc bwd_plan(const ScanShape& sh) {
    BwdTc p;
    p.unit = walk_unit_tc(sh);
    p.cut = p.unit < sh.seqs.T;
    p.heads = grad_heads_tc(sh);
    p.splits = (sh.H / sh.G + p.heads - 1) / p.heads;
    const size_t chunks = static_cast<size_t>(sh.seqs.units(kQ)), st = chunks * sh.H * sh.N * sh.P * 2;
    const size_t units = p.cut ? static_cast<size_t>(sh.seqs.units(p.unit)) : 0, us = units * sh.H * sh.N * sh.P * 4;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += align_up(bytes, 256);
        return here;
    };
    p.h0 = take(st);
    p.dh = take(st);
    p.dd = take(chunks * sh.H * 4);
    p.part = take(p.splits > 1 ? 2ull * p.splits * sh.seqs.rows() * sh.G * sh.N * 4 : 0);
    p.states = take(us);
    p.states_b = take(us);
    p.decay = take(units * sh.H * 4);
    p.decay_b = take(units * sh.H * 4);
    p.total = at;
    return p;
}

}  // namespace

size_t ssm_tc_bwd_workspace(const ScanShape& sh) { return bwd_plan(sh).total; }

cudaError_t launch_ssm_tc_bwd(const ScanShape& sh, const ScanIn& in, const ScanGrads& gr, void* wsv, cudaStream_t s, long long wait_ns) {
    uint8_t* ws = static_cast<uint8_t*>(wsv);
    const BwdTc p = bwd_plan(sh);
    auto f = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
    const WalkJob jobs[2] = {{in.bm, in.x, in.s0, nullptr, f(p.states), f(p.decay), ws + p.h0, 0},
                             {in.cm, gr.dy, gr.ds1, gr.ds0, f(p.states_b), f(p.decay_b), ws + p.dh, 1}};
    cudaError_t e;
    // d_initial_state is a result in fp32; the saved states feed bf16 results
    const int exact = gr.ds0 != nullptr;
    if (p.cut) {
        if ((e = launch_ssm_walk_tc(sh, in.step, in.g, jobs, 2, p.unit, 1, 0, exact, s, wait_ns)) != cudaSuccess) return e;
        const ChainJob chains[2] = {{in.s0, nullptr, f(p.states), f(p.decay), 0}, {gr.ds1, gr.ds0, f(p.states_b), f(p.decay_b), 1}};
        if ((e = launch_ssm_chain(sh, p.unit, chains, 2, s)) != cudaSuccess) return e;
        WalkJob again[2] = {jobs[0], jobs[1]};
        again[1].last = nullptr;  // the chain has written it
        e = launch_ssm_walk_tc(sh, in.step, in.g, again, 2, p.unit, 0, 1, 0, s, wait_ns);
    } else {
        e = launch_ssm_walk_tc(sh, in.step, in.g, jobs, 2, p.unit, 0, 0, exact, s, wait_ns);
    }
    if (e != cudaSuccess) return e;
    GradMaps maps;
    const long long rows = sh.seqs.rows();
    if (!rows_map(&maps.x, in.x.p, in.x.ld, sh.P, sh.H, rows, kQ) || !rows_map(&maps.dy, gr.dy.p, gr.dy.ld, sh.P, sh.H, rows, kQ) ||
        !rows_map(&maps.b, in.bm.p, in.bm.ld, sh.N, sh.G, rows, kQ) || !rows_map(&maps.c, in.cm.p, in.cm.ld, sh.N, sh.G, rows, kQ) ||
        !rows_map(&maps.dx, gr.dx.p, gr.dx.ld, sh.P, sh.H, rows, kQ))
        return cudaErrorInvalidValue;
    GradTcArgs a{};
    a.seqs = sh.seqs;
    a.H = sh.H; a.G = sh.G; a.P = sh.P; a.N = sh.N;
    a.heads = p.heads;
    a.splits = p.splits;
    a.rows = rows;
    using BF = __nv_bfloat16;
    a.step = static_cast<const BF*>(in.step);
    a.g = static_cast<const BF*>(in.g);
    a.d = in.d;
    a.h0 = ws + p.h0;
    a.dh = ws + p.dh;
    a.dx = static_cast<BF*>(gr.dx.p);
    a.db = static_cast<BF*>(gr.dbm.p);
    a.dc = static_cast<BF*>(gr.dcm.p);
    a.dstep = static_cast<BF*>(gr.dstep);
    a.dg = static_cast<BF*>(gr.dg);
    a.ld_dx = gr.dx.ld;
    a.ld_db = gr.dbm.ld;
    a.ld_dc = gr.dcm.ld;
    a.part = f(p.part);
    a.dd_part = gr.dd ? f(p.dd) : nullptr;
    a.wait_ns = wait_ns;
    if ((e = cudaFuncSetAttribute(grad_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448)) != cudaSuccess) return e;
    g_launched.store(true, std::memory_order_relaxed);
    // groups' shares of one chunk next to each other: B, C and the gates stay in L2
    grad_tc_kernel<<<dim3(sh.G * p.splits, static_cast<unsigned>(sh.seqs.units(kQ))), kGradTc, 232448, s>>>(maps, a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_ssm_grad_sums(sh, gr, a.part, p.splits, a.dd_part, static_cast<int>(sh.seqs.units(kQ)), s);
}

int ssm_tc_grad_read_clear_status(cudaStream_t s) { return read_clear_status(s); }

}  // namespace gdn2
