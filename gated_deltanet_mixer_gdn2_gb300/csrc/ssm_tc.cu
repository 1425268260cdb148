// ssm_tc.cu -- the selective state-space scan on the tensor cores (bf16, P a multiple of 64, N 64 or 128).
//
// Chunks of 128 tokens. With L_i the inclusive sum of g within the chunk, s_j the steps, D the skip:
//     M_ij = (C_i . B_j) e^{L_i - L_j} s_j  (i >= j),        Y = M X + e^{L} (C H) + D X
//     H'   = e^{L_end} H + B^T X~,                           X~_j = s_j e^{L_end - L_j} x_j
// One block walks over the chunks of its unit for 64 value columns of one head; all five products run on
// tcgen05 with their accumulators in tensor memory, and the state stays in registers in fp32. Only the
// update of the state is serial from chunk to chunk (64 multiply-adds per thread), so the block is a
// pipeline of warp roles over different chunks: products (warp 0: rows 0-31 of M are
// the least work, so its scheduler is the least loaded), copies (warp 1), gates (warps 2 and 3), M (warps 4-7),
// Y (warps 8-15), X~ and state (warps 16-23).
// Roundings to bf16: M, X~ and the state as operands of Y, once each; sums, states and decays are fp32.
// 4 x 2048 tokens, 32 heads of 64 values, N = 128: 32 us, 2 us per chunk and block (CUDA cores: 836 us; even 16 tokens
// of 8 heads take 10 us here and 12 us there); with the state as a result 49 us. The products need 1500 of a chunk's 3150
// cycles. Three things take about as long as the chunk: issuing its 32 products and 8 waits from one warp; the state's way
// round from X~ ready to X~ ready (product, read-out, operand, X~); and X's three stages, each held for its load (2300),
// two chunks and Y's way out. Slower for what they cost the others: two issuing warps (36 us), Y straight to global memory
// (34 us), X~ formed by Y's warps (39 us before the packed arithmetic's 35), pairs of blocks that share B and C by
// multicast loads (42 for 35).
#include "ssm_tc.cuh"

namespace gdn2 {
namespace {

// Shared memory (byte offsets from a 1024-aligned base); tiles are [128 rows][64 bf16], 128-byte swizzle. X has three
// stages: a stage is free only when Y has left through it, the longest way of all. X~ has one buffer per
// part; three of them take the room of C's second stage.
template <int kParts>
struct So {
    static constexpr uint32_t kTile = 16384;
    static constexpr int kXS = 3, kCS = kParts == 1 ? 2 : 1;
    static constexpr uint32_t B = 0;                  // 2 stages x 2 tiles (n 0-63, 64-127)
    static constexpr uint32_t C = B + 4 * kTile;      // kCS x 2
    static constexpr uint32_t X = C + 2 * kCS * kTile;  // kXS; Y replaces X for its store
    static constexpr uint32_t XW = X + kXS * kTile;   // parts of X~
    static constexpr uint32_t HB = XW + kParts * kTile;  // the state as a bf16 operand
    static constexpr uint32_t kGateStage = 4 * 512;   // {L, col, wend, step} [128] fp32, a stage per stage of X
    static constexpr uint32_t GATE = HB + kTile;
    static constexpr uint32_t BAR = GATE + kXS * kGateStage;
    static constexpr uint32_t TOTAL = BAR + 320;
    static_assert(TOTAL + 1024 <= 232448, "scan kernel shared memory");
};

enum Bar {
    kFullB = 0, kFullC = 2, kFullX = 4, kReady = 7, kXEmpty = 10, kSFull = 13, kDFull = 15, kXwReady = 17, kMReady, kYFull = kMReady + 2, kYEmpty,
    kCFree, kYOut = kCFree + 2, kDrain = kYOut + 4, kBars
};
constexpr uint32_t kBarBytes = 8 * kBars + 16;
static_assert(kBarBytes <= 320, "barrier room");
constexpr int kScanThreads = 768;

// tensor-memory columns: scores of two chunks, each half replaced by M (8 packed columns at the start of every
// 16); Y's sum over the chunk, its readouts of the state of two chunks, the state's increment
constexpr uint32_t kTS = 0, kTYi = 256, kTYx = 320, kTD = 448;

struct ScanMaps {
    CUtensorMap x, b, c, y;
};

struct ScanTcArgs {
    Seqs seqs;
    int unit;                        // tokens per block, a multiple of 128 (or at least the longest sequence)
    const __nv_bfloat16 *step, *g;
    const float *d, *s0;
    float* s1;
    __nv_bfloat16* y;
    float* states;                   // [units][H][N][P] when `cut`: the states before the units
    int cut, H, G, P, N;
    long long wait_ns;
};

// Gate arrays of one chunk, by one warp, four tokens per lane: L and the decay sums in units of log 2.
// The decay to the chunk's end is a suffix sum of its own: as a difference of prefix sums it would lose
// the small values' digits behind a strong decay, and the state is held to fp32.
__device__ __forceinline__ void gate_arrays(float* arr, int lane, const float (&gv)[4], const float (&sv)[4]) {
    float p[4], q[4];
    p[0] = gv[0]; p[1] = p[0] + gv[1]; p[2] = p[1] + gv[2]; p[3] = p[2] + gv[3];
    q[3] = 0.f; q[2] = gv[3]; q[1] = q[2] + gv[2]; q[0] = q[1] + gv[1];
    float pre = p[3], suf = p[3];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const float a = __shfl_up_sync(0xffffffffu, pre, d), b = __shfl_down_sync(0xffffffffu, suf, d);
        if (lane >= d) pre += a;
        if (lane + d < 32) suf += b;
    }
    const float before = __shfl_up_sync(0xffffffffu, pre, 1), after = __shfl_down_sync(0xffffffffu, suf, 1);
    const float lo = lane ? before : 0.f, hi = lane < 31 ? after : 0.f;
    const float end = __shfl_sync(0xffffffffu, pre, lane | 7);  // L at the end of the 32-token block
    const float4 L = make_float4(lo + p[0], lo + p[1], lo + p[2], lo + p[3]);
    const float4 s = make_float4(sv[0], sv[1], sv[2], sv[3]);
    float4 col = exp2_4(make_float4(end - L.x, end - L.y, end - L.z, end - L.w));
    col.x *= s.x; col.y *= s.y; col.z *= s.z; col.w *= s.w;
    float4 we = exp2_4(make_float4(hi + q[0], hi + q[1], hi + q[2], hi + q[3]));
    we.x *= s.x; we.y *= s.y; we.z *= s.z; we.w *= s.w;
    reinterpret_cast<float4*>(arr)[lane] = L;
    reinterpret_cast<float4*>(arr + 128)[lane] = col;
    reinterpret_cast<float4*>(arr + 256)[lane] = we;
    reinterpret_cast<float4*>(arr + 384)[lane] = s;
}

// kParts bf16 parts of X~ enter the state's product: one where the state only feeds bf16 results, three
// (2^-24 of every term) where it is returned in fp32 (4 x 2048 tokens of 32 heads: 32 and 49 us).
template <int kParts>
__global__ void __launch_bounds__(kScanThreads, 1) scan_tc_kernel(const __grid_constant__ ScanMaps maps, const ScanTcArgs a) {
    using so = So<kParts>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + so::BAR);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + so::BAR + kBars * 8);
    volatile int* err = reinterpret_cast<volatile int*>(sm + so::BAR + kBars * 8 + 8);
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    const int pb = a.P / kCols, h = blockIdx.x / pb, p0 = (blockIdx.x - h * pb) * kCols, grp = h / (a.H / a.G);
    Unit u;
    if (!find_unit(a.seqs, a.unit, blockIdx.y, u)) return;
    u.len = uniform(u.len);
    u.row = uniform(u.row);
    const int NC = (u.len + kQ - 1) / kQ;
    const long long lim = a.wait_ns;

    if (tid == 0) {
        for (int i = 0; i < kBars; ++i) {
            const bool four = (i >= kXEmpty && i < kXEmpty + 3) || i == kMReady || i == kMReady + 1;
            const bool eight = i == kXwReady || i == kYEmpty;
            mbar_init(bars + i, four ? 4 : eight ? 8 : i >= kYOut && i < kDrain ? 2 : 1);
        }
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
    constexpr uint32_t tmem = 0;  // all 512 columns: the allocation starts at column 0
    const int ks = a.N / 16;  // K steps over the state size
    const size_t plane = static_cast<size_t>(a.N) * a.P;

    if (warp == 1) {
        if (lane == 0) {
            // ---- copies, in the order in which their stages come free: C after the state's readout, B after its increment,
            // X when the chunk before has left through it.
            const int halves = a.N / 64;
            prefetch_tensormap(&maps.b);
            prefetch_tensormap(&maps.c);
            prefetch_tensormap(&maps.x);
            int nb = 0, nc = 0, nx = 0;
            auto load_b = [&]() {
                const int st = nb & 1;
                mbar_arrive_expect_tx(bars + kFullB + st, so::kTile * halves);
                for (int k = 0; k < halves; ++k)
                    tma_load_3d(sm + so::B + (2 * st + k) * so::kTile, &maps.b, 64 * k, grp, u.row + nb * kQ, bars + kFullB + st);
                ++nb;
            };
            auto load_c = [&]() {
                const int st = nc % so::kCS;
                mbar_arrive_expect_tx(bars + kFullC + st, so::kTile * halves);
                for (int k = 0; k < halves; ++k)
                    tma_load_3d(sm + so::C + (2 * st + k) * so::kTile, &maps.c, 64 * k, grp, u.row + nc * kQ, bars + kFullC + st);
                ++nc;
            };
            auto load_x = [&]() {
                const int st = nx % so::kXS;
                mbar_arrive_expect_tx(bars + kFullX + st, so::kTile);
                tma_load_3d(sm + so::X + st * so::kTile, &maps.x, p0, h, u.row + nx * kQ, bars + kFullX + st);
                ++nx;
            };
            auto free_of = [&](int bar, uint32_t parity) { return mbar_wait_or_abort(bars + bar, parity, lim, err); };
            bool ok = true;
            for (int k = 0; k < 2 && k < NC; ++k) {
                if (k < so::kCS) load_c();
                load_b();
                load_x();
            }
            if (nx < NC) load_x();
            for (int c = 0; ok && (nc < NC || nb < NC || nx < NC); ++c) {
                if (nc < NC && (ok = free_of(kCFree + (c & 1), (c >> 1) & 1))) load_c();
                if (ok && nb < NC && (ok = free_of(kDFull + (c & 1), (c >> 1) & 1))) load_b();
                if (ok && c >= 1 && nx < NC && (ok = free_of(kXEmpty + (c - 1) % so::kXS, ((c - 1) / so::kXS) & 1))) load_x();
            }
            if (!ok) note_failure(err);
            auto drain = [&](int issued, int full, int stages) {  // nothing in flight when the block ends
                for (int c = issued > stages ? issued - stages : 0; c < issued; ++c)
                    mbar_wait(bars + full + c % stages, (c / stages) & 1, kDefaultWaitNs);
            };
            drain(nb, kFullB, 2);
            drain(nc, kFullC, so::kCS);
            drain(nx, kFullX, so::kXS);
        }
    } else if (warp == 0) {
        const uint32_t id_s = idesc_bf16(128, 128, false, false), id_d = idesc_bf16(128, 64, true, true),
                       id_x = idesc_bf16(128, 64, false, true);
        const uint32_t lead = elect_one();
        // K-major tiles: 16 channels are 32 bytes of a row, the next 64 the next tile. MN-major: 16 tokens (or
        // state rows) are 16 rows of 128 bytes.
        const uint32_t dk = desc_lo(sb, 16), dm = desc_lo(sb, so::kTile);
        auto wait = [&](int bar, uint32_t parity) { return wait_bar(bars + bar, parity, lim, err); };
        // Two stretches of products per chunk, each behind one set of waits and one tensor-memory fence, which lets the
        // tensor core run dry. Each wait stands for all it can: X~ ready implies the state ready, X loaded, a short
        // chunk's rows cleared and the increment before it taken; Y's sums taken, that chunk's products done; the
        // increment's commit frees B, C and the state's operand.
        bool ok = true;
        for (int c = -1; c < NC && NC > 0; ++c) {
            const uint32_t ph1 = c & 1;  // phase of the barriers used once per chunk
            const int n = c + 1, st = n & 1;
            if (c >= 0) {
                if (!(ok = wait(kXwReady, ph1))) break;
                tc_fence_after();
                // readout of the state, then its increment
                mma_steps<false, kStepK, kStepMn, kJumpK, 0>(lead, kTYx + 64 * (c & 1), dk + ((so::C + 2 * (c % so::kCS) * so::kTile) >> 4),
                                                             dm + (so::HB >> 4), id_x, 0, ks);
                commit_by(lead, bars + kCFree + (c & 1));
#pragma unroll 1
                for (int k = 0; k < kParts; ++k)
                    mma_steps<false, kStepMn, kStepMn, 0, 0>(lead, kTD, dm + ((so::B + 2 * (c & 1) * so::kTile) >> 4),
                                                             dm + ((so::XW + k * so::kTile) >> 4), id_d, k > 0, 8);
                commit_by(lead, bars + kDFull + (c & 1));
            }
            if (c >= 1 && !(ok = wait(kYEmpty, ph1 ^ 1))) break;
            if (n < NC) {
                // the next chunk's scores: M of the next chunk is formed while this one's is used
                if (!(ok = wait(kFullB + st, (n >> 1) & 1) && wait(kFullC + n % so::kCS, (n / so::kCS) & 1))) break;
                // a short chunk's rows of B are cleared first
                if (u.len - n * kQ < kQ && !(ok = wait(kReady + n % so::kXS, (n / so::kXS) & 1))) break;
                mma_steps<false, kStepK, kStepK, kJumpK, kJumpK>(lead, kTS + 128 * st, dk + ((so::C + 2 * (n % so::kCS) * so::kTile) >> 4),
                                                                 dk + ((so::B + 2 * st * so::kTile) >> 4), id_s, 0, ks);
                commit_by(lead, bars + kSFull + st);
            }
            // within the chunk
            if (c >= 0) {
                // two barriers: M of the next chunk may be ready before this is looked at
                if (!(ok = wait(kMReady + (c & 1), (c >> 1) & 1))) break;
                tc_fence_after();
                mma_steps<true, 16, kStepMn, 0, 0>(lead, kTYi, kTS + 128 * (c & 1), dm + ((so::X + (c % so::kXS) * so::kTile) >> 4), id_x, 0, 8);
                commit_by(lead, bars + kYFull);
            }
        }
        commit_by(lead, bars + kDrain);
        mbar_wait(bars + kDrain, 0, kDefaultWaitNs);
    } else if (warp < 4) {
        // ---- gates. A head's values lie 2 H bytes apart and take up to 3500 cycles to arrive, about two chunks: two warps
        // take the chunks in turn, each with its next chunk's values in flight.
        float gn[4], sn[4];
        auto fetch = [&](int c) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = c * kQ + 4 * lane + e;
                const size_t at = static_cast<size_t>(u.row + t) * a.H + h;
                gn[e] = t < u.len ? ssm_gate(__bfloat162float(a.g[at])) * kLog2e : 0.f;
                sn[e] = t < u.len ? __bfloat162float(a.step[at]) : 0.f;
            }
        };
        if (warp - 2 < NC) fetch(warp - 2);
        for (int c = warp - 2; c < NC; c += 2) {
            const int st = c & 1, xs = c % so::kXS;
            // the arrays of the stage have been read: Y, the last reader, frees them with X
            if (c >= so::kXS && !wait_bar(bars + kXEmpty + xs, ((c / so::kXS) & 1) ^ 1, lim, err)) break;
            gate_arrays(reinterpret_cast<float*>(sm + so::GATE + xs * so::kGateStage), lane, gn, sn);
            const int n = u.len - c * kQ;
            if (n < kQ) {
                if (!wait_bar(bars + kFullB + st, (c >> 1) & 1, lim, err) || !wait_bar(bars + kFullX + xs, (c / so::kXS) & 1, lim, err)) break;
                // the rows past the sequence hold other tokens: zeros, so that not even their NaN enters a sum
                const uint4 z = make_uint4(0, 0, 0, 0);
                for (int i = n * 8 + lane; i < kQ * 8; i += 32) {
                    reinterpret_cast<uint4*>(sm + so::B + 2 * st * so::kTile)[i] = z;
                    reinterpret_cast<uint4*>(sm + so::B + (2 * st + 1) * so::kTile)[i] = z;
                    reinterpret_cast<uint4*>(sm + so::X + xs * so::kTile)[i] = z;
                }
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive1(bars + kReady + xs);
            if (c + 2 < NC) fetch(c + 2);
        }
    } else if (warp >= 4 && warp < 8) {
        // ---- M: row i of the chunk per thread, in place of the scores; blocks of 32 columns. Below the diagonal
        // block the decay factors through the end of the column's block (both factors <= 1), one
        // exponential per row and block; on it, one per entry; above it, zeros. The loops of all roles stay
        // rolled: unrolled, the roles' bodies together overran the instruction cache and fetching them was
        // the longest stall (a chunk took 9400 cycles).
        const int q = warp & 3, i = 32 * q + lane;
        const uint32_t lane_base = static_cast<uint32_t>(32 * q) << 16;
        for (int c = 0; c < NC; ++c) {
            const int st = c & 1;
            const uint32_t ph = (c >> 1) & 1;
            const int xs = c % so::kXS;
            if (!wait_bar(bars + kReady + xs, (c / so::kXS) & 1, lim, err)) break;
            if (!wait_bar(bars + kSFull + st, ph, lim, err)) break;
            tc_fence_after();
            const float* arr = reinterpret_cast<const float*>(sm + so::GATE + xs * so::kGateStage);
            const float Li = arr[i];
            const uint32_t at = tmem + lane_base + kTS + 128 * st;
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {
                uint32_t m[16];
                if (b > q) {
#pragma unroll
                    for (int k = 0; k < 16; ++k) m[k] = 0;
                } else {
                    float x[32];
                    tmem_ld_cols<2>(at + 32 * b, x);
                    if (b == q) {
#pragma unroll
                        for (int j4 = 0; j4 < 8; ++j4) {
                            const float4 L = *reinterpret_cast<const float4*>(arr + 32 * b + 4 * j4);
                            const float4 s = *reinterpret_cast<const float4*>(arr + 384 + 32 * b + 4 * j4);
                            const uint64_t l2[2] = {f32x2(L.x, L.y), f32x2(L.z, L.w)}, s2[2] = {f32x2(s.x, s.y), f32x2(s.z, s.w)};
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int j = 4 * j4 + 2 * e;
                                float d0, d1, v0, v1;
                                f32x2_split(sub_f32x2(f32x2(Li, Li), l2[e]), d0, d1);
                                f32x2_split(mul_f32x2(mul_f32x2(f32x2(x[j], x[j + 1]), s2[e]), f32x2(ex2_approx(d0), ex2_approx(d1))), v0, v1);
                                m[2 * j4 + e] = pack_bf16x2(j <= lane ? v0 : 0.f, j + 1 <= lane ? v1 : 0.f);
                            }
                        }
                    } else {
                        const float rf = ex2_approx(Li - arr[32 * b + 31]);
                        const uint64_t rf2 = f32x2(rf, rf);
#pragma unroll
                        for (int j4 = 0; j4 < 8; ++j4) {
                            const float4 cf = *reinterpret_cast<const float4*>(arr + 128 + 32 * b + 4 * j4);
                            const uint64_t v0 = mul_f32x2(mul_f32x2(f32x2(x[4 * j4], x[4 * j4 + 1]), rf2), f32x2(cf.x, cf.y));
                            const uint64_t v1 = mul_f32x2(mul_f32x2(f32x2(x[4 * j4 + 2], x[4 * j4 + 3]), rf2), f32x2(cf.z, cf.w));
                            m[2 * j4] = bf16x2_narrow(v0);
                            m[2 * j4 + 1] = bf16x2_narrow(v1);
                        }
                    }
                }
                const uint32_t m0[8] = {m[0], m[1], m[2], m[3], m[4], m[5], m[6], m[7]}, m1[8] = {m[8], m[9], m[10], m[11], m[12], m[13], m[14], m[15]};
                tmem_st8(at + 32 * b, m0);
                tmem_st8(at + 32 * b + 16, m1);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive1(bars + kMReady + (c & 1));
        }
    } else if (warp >= 8 && warp < 16) {
        // ---- Y: row i of the chunk and half of the 64 columns per thread; replaces that part of X, and the two warps of
        // 32 rows leave by one bulk store. Both sums are taken out of tensor memory before anything else, for the next
        // chunk's products wait for their room.
        const int q = warp & 3, half = warp >= 12, i = 32 * q + lane;
        const uint32_t lane_base = (static_cast<uint32_t>(32 * q) << 16) + 32 * half;
        const float dk = a.d ? a.d[h] : 0.f;
        for (int c = 0; c < NC; ++c) {
            const int xs = c % so::kXS;
            const uint32_t xph = (c / so::kXS) & 1;
            if (!wait_bar(bars + kFullX + xs, xph, lim, err) || !wait_bar(bars + kReady + xs, xph, lim, err)) break;
            const float eL = ex2_approx(reinterpret_cast<const float*>(sm + so::GATE + xs * so::kGateStage)[i]);
            uint8_t* xt = sm + so::X + xs * so::kTile;
            const int n = u.len - c * kQ;
            if (!wait_bar(bars + kYFull, c & 1, lim, err)) break;
            tc_fence_after();
            uint32_t yi[2][16], yx[2][16];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                tmem_ld16(lane_base + kTYi + 16 * k, yi[k]);
                tmem_ld16(lane_base + kTYx + 64 * (c & 1) + 16 * k, yx[k]);
            }
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive1(bars + kYEmpty);
            uint4* yrow = reinterpret_cast<uint4*>(a.y + (static_cast<size_t>(u.row + c * kQ + i) * a.H + h) * a.P + p0 + 32 * half);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint4* cell = reinterpret_cast<uint4*>(xt + i * 128 + (((4 * half + k) ^ (i & 7)) << 4));
                const uint4 xv = *cell;
                const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
                uint32_t ow[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int at = 8 * (k & 1) + 2 * e;
                    const uint64_t yxe = f32x2(__uint_as_float(yx[k >> 1][at]), __uint_as_float(yx[k >> 1][at + 1]));
                    const uint64_t yie = f32x2(__uint_as_float(yi[k >> 1][at]), __uint_as_float(yi[k >> 1][at + 1]));
                    ow[e] = bf16x2_narrow(fma_f32x2(f32x2(dk, dk), bf16x2_widen(xw[e]), fma_f32x2(f32x2(eL, eL), yxe, yie)));
                }
                const uint4 o = make_uint4(ow[0], ow[1], ow[2], ow[3]);
                if (n >= kQ) *cell = o;
                else if (i < n) yrow[k] = o;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive1(bars + kYOut + q);
            if (half == 0) {
                if (!wait_bar(bars + kYOut + q, c & 1, lim, err)) break;
                if (lane == 0) {
                    if (n >= kQ) {
                        tma_store_3d(&maps.y, xt + 4096 * q, p0, h, u.row + c * kQ + 32 * q);
                        bulk_commit();
                        bulk_wait_read_all();
                    }
                    mbar_arrive1(bars + kXEmpty + xs);
                }
                __syncwarp();
            }
        }
        if (lane == 0) bulk_wait_all();
    } else {
        // ---- X~ of the next chunk, then the state over this one: row n of the state (token of X~) per thread, half
        // of the 64 columns per group of four warps
        const int q = warp & 3, half = warp >= 20, r = 32 * q + lane;
        const uint32_t lane_base = static_cast<uint32_t>(32 * q) << 16;
        const bool real = r < a.N;
        const size_t at = static_cast<size_t>(real ? r : 0) * a.P + p0 + 32 * half;
        float hx[32];
        {
            const float* from = a.cut ? a.states + (static_cast<size_t>(blockIdx.y) * a.H + h) * plane
                                      : (a.s0 ? a.s0 + (static_cast<size_t>(u.seq) * a.H + h) * plane : nullptr);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float4 f = from && real ? reinterpret_cast<const float4*>(from + at)[k] : make_float4(0.f, 0.f, 0.f, 0.f);
                hx[4 * k] = f.x; hx[4 * k + 1] = f.y; hx[4 * k + 2] = f.z; hx[4 * k + 3] = f.w;
            }
        }
        float2 decay = make_float2(1.f, 0.f);
        bool ok = true;
        for (int c = -1; c < NC; ++c) {
            const int n = c + 1;
            if (c >= 0) {
                if (!(ok = wait_bar(bars + kDFull + (c & 1), (c >> 1) & 1, lim, err))) break;
                tc_fence_after();
                float x[32];
                tmem_ld_cols<2>(tmem + lane_base + kTD + 32 * half, x);
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const uint64_t h2 = f32x2(hx[2 * k], hx[2 * k + 1]), d2 = f32x2(x[2 * k], x[2 * k + 1]);
                    f32x2_split(fma_f32x2(f32x2(decay.x, decay.x), h2, kParts == 1 ? d2 : fma_f32x2(f32x2(decay.y, decay.y), h2, d2)), hx[2 * k], hx[2 * k + 1]);
                }
                tc_fence_before();
            }
            if (n < NC) {
                st_row_bf16x32(sm + so::HB, r, 4 * half, hx);
                // X~ of chunk n, row r, once the increment before it has been formed from the last: each part is the bf16
                // rounding of what the parts before it leave
                const int xs = n % so::kXS;
                if (!(ok = wait_bar(bars + kFullX + xs, (n / so::kXS) & 1, lim, err) && wait_bar(bars + kReady + xs, (n / so::kXS) & 1, lim, err))) break;
                const float* arr = reinterpret_cast<const float*>(sm + so::GATE + xs * so::kGateStage);
                const float w = arr[256 + r];
                decay = kParts == 1 ? make_float2(ex2_approx(arr[127]), 0.f) : ssm_decay(kLn2 * arr[127]);
                const uint8_t* xt = sm + so::X + xs * so::kTile + r * 128;
                uint8_t* to = sm + so::XW + r * 128;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int cell = ((4 * half + k) ^ (r & 7)) << 4;
                    const uint4 xv = *reinterpret_cast<const uint4*>(xt + cell);
                    uint64_t v[4] = {bf16x2_widen(xv.x), bf16x2_widen(xv.y), bf16x2_widen(xv.z), bf16x2_widen(xv.w)};
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = mul_f32x2(v[e], f32x2(w, w));
#pragma unroll
                    for (int part = 0; part < kParts; ++part) {
                        const uint4 o = make_uint4(bf16x2_narrow(v[0]), bf16x2_narrow(v[1]), bf16x2_narrow(v[2]), bf16x2_narrow(v[3]));
                        *reinterpret_cast<uint4*>(to + part * so::kTile + cell) = o;
                        if (part + 1 < kParts) {
                            v[0] = sub_f32x2(v[0], bf16x2_widen(o.x));
                            v[1] = sub_f32x2(v[1], bf16x2_widen(o.y));
                            v[2] = sub_f32x2(v[2], bf16x2_widen(o.z));
                            v[3] = sub_f32x2(v[3], bf16x2_widen(o.w));
                        }
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive1(bars + kXwReady);
            }
        }
        if (ok && a.s1 && u.k == u.count - 1 && real) {
            float* to = a.s1 + (static_cast<size_t>(u.seq) * a.H + h) * plane + at;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                reinterpret_cast<float4*>(to)[k] = make_float4(hx[4 * k], hx[4 * k + 1], hx[4 * k + 2], hx[4 * k + 3]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(*tmem_slot, 512);
}

template <int kParts>
cudaError_t launch_scan(const ScanMaps& maps, const ScanTcArgs& a, dim3 grid, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(scan_tc_kernel<kParts>, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
    if (e != cudaSuccess) return e;
    g_launched.store(true, std::memory_order_relaxed);
    // the whole shared memory: one block per SM, and no operand descriptor reaches past the block's own
    scan_tc_kernel<kParts><<<grid, kScanThreads, 232448, s>>>(maps, a);
    return cudaGetLastError();
}

}  // namespace

bool ssm_tc_shape(const ScanShape& sh) {
    return sh.dt == GDN2_BF16 && sh.P % 64 == 0 && (sh.N == 64 || sh.N == 128) && sh.seqs.units(kQ) <= 65535;
}

namespace {
// Tokens per block: whole sequences while their chains fill four fifths of the SMs, else units whose starting states come
// from a pass over their increments (2 x 32768 tokens, 32 heads, with the last state: 386 us cut, 607 whole; 1 x 8192, 8 heads: 43
// and 96; a packed batch of 8 with enough chains: 138 cut, 95 whole). The rule sees the number of sequences, not their lengths:
// one of 30000 tokens among seven of a few takes 348 us, 197 alone.
int fwd_unit(const ScanShape& sh) {
    int dev = 0, sms = 152;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) sms = 152;
    const int whole = (sh.seqs.T + kQ - 1) / kQ * kQ;
    const long long chains = static_cast<long long>(sh.H) * (sh.P / kCols), chunks = (sh.seqs.rows() + kQ - 1) / kQ;
    if (10 * chains * sh.seqs.B >= 8 * sms) return whole;
    // about six blocks per SM, of 1024 tokens or more
    long long len = (chains * chunks + 6LL * sms - 1) / (6LL * sms) * kQ;
    if (len < 1024) len = 1024;
    return 2 * len > whole ? whole : static_cast<int>(len);
}
}  // namespace

// States and decays of the units, when sequences are cut.
size_t ssm_tc_fwd_workspace(const ScanShape& sh) {
    const int unit = fwd_unit(sh);
    if (unit >= sh.seqs.T) return 0;
    return align_up(sizeof(float) * static_cast<size_t>(sh.seqs.units(unit)) * sh.H * (static_cast<size_t>(sh.N) * sh.P + 4), 256);
}

cudaError_t launch_ssm_tc_fwd(const ScanShape& sh, const ScanIn& in, void* y, float* s1, void* ws, cudaStream_t s, long long wait_ns) {
    ScanMaps maps;
    const long long rows = sh.seqs.rows();
    if (!rows_map(&maps.x, in.x.p, in.x.ld, sh.P, sh.H, rows, kQ) || !rows_map(&maps.b, in.bm.p, in.bm.ld, sh.N, sh.G, rows, kQ) ||
        !rows_map(&maps.c, in.cm.p, in.cm.ld, sh.N, sh.G, rows, kQ) || !rows_map(&maps.y, y, (long long)sh.H * sh.P, sh.P, sh.H, rows, 32))
        return cudaErrorInvalidValue;
    ScanTcArgs a{};
    a.seqs = sh.seqs;
    a.unit = fwd_unit(sh);
    a.cut = a.unit < sh.seqs.T;
    a.step = static_cast<const __nv_bfloat16*>(in.step);
    a.g = static_cast<const __nv_bfloat16*>(in.g);
    a.d = in.d;
    a.s0 = in.s0;
    a.s1 = a.cut ? nullptr : s1;
    a.y = static_cast<__nv_bfloat16*>(y);
    a.H = sh.H; a.G = sh.G; a.P = sh.P; a.N = sh.N;
    a.wait_ns = wait_ns;
    const dim3 grid(sh.H * (sh.P / kCols), static_cast<unsigned>(sh.seqs.units(a.unit)));
    if (a.cut) {
        // the units' increments, exact where the last state is a result, and their starting states
        a.states = static_cast<float*>(ws);
        float* decay = a.states + static_cast<size_t>(sh.seqs.units(a.unit)) * sh.H * sh.N * sh.P;
        const WalkJob job{in.bm, in.x, in.s0, nullptr, a.states, decay, nullptr, 0};
        cudaError_t e = launch_ssm_walk_tc(sh, in.step, in.g, &job, 1, a.unit, 1, 0, s1 != nullptr, s, wait_ns);
        if (e != cudaSuccess) return e;
        const ChainJob chain{in.s0, s1, a.states, decay, 0};
        if ((e = launch_ssm_chain(sh, a.unit, &chain, 1, s)) != cudaSuccess) return e;
    }
    return a.s1 ? launch_scan<3>(maps, a, grid, s) : launch_scan<1>(maps, a, grid, s);
}

int ssm_tc_read_clear_status(cudaStream_t s) { return read_clear_status(s); }

}  // namespace gdn2
