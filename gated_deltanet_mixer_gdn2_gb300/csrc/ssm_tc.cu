// ssm_tc.cu -- the selective state-space scan on the tensor cores (bf16, P a multiple of 64, N 64 or 128).
//
// Chunks of 128 tokens. With L_i the inclusive sum of g within the chunk, s_j the steps, D the skip:
//     M_ij = (C_i . B_j) e^{L_i - L_j} s_j  (i >= j),        Y = M X + e^{L} (C H) + D X
//     H'   = e^{L_end} H + B^T X~,                           X~_j = s_j e^{L_end - L_j} x_j
// One block walks over the chunks of its unit for 64 value columns of one head; all five products run on
// tcgen05 with their accumulators in tensor memory, and the state stays in registers in fp32. Only the
// update of the state is serial from chunk to chunk (64 multiply-adds per thread), so the block is a
// pipeline of warp roles over different chunks: copies (warps 0 and 3), products (warp 1), gates
// (warp 2), M (warps 4-7), Y (warps 8-11), X~ and state (warps 12-15).
#include "ssm_common.cuh"
#include "tc_common.cuh"

namespace gdn2 {
namespace {

constexpr int kQ = 128;   // tokens per chunk
constexpr int kCols = 64; // value columns per block

// shared memory (byte offsets from a 1024-aligned base); tiles are [128 rows][64 bf16], 128-byte swizzle
namespace so {
constexpr uint32_t kTile = 16384;
constexpr uint32_t B = 0;                    // 2 stages x 2 tiles (n 0-63, 64-127)
constexpr uint32_t C = B + 4 * kTile;        // 2 x 2
constexpr uint32_t X = C + 4 * kTile;        // 2; Y replaces X for its store
constexpr uint32_t XW = X + 2 * kTile;       // 2 buffers of X~ parts
constexpr uint32_t HB = XW + 2 * kTile;      // the state as a bf16 operand
constexpr uint32_t GATE = HB + kTile;        // 2 stages x {L, col, wend, step} [128] fp32
constexpr uint32_t kGateStage = 4 * 512;
constexpr uint32_t BAR = GATE + 2 * kGateStage;
constexpr uint32_t TOTAL = BAR + 256;
}  // namespace so
static_assert(so::TOTAL + 1024 <= 232448, "scan kernel shared memory");

enum Bar {
    kFull = 0, kFullX = 2, kReady = 4, kBcEmpty = 6, kXEmpty = 8, kSFull = 10, kSEmpty = 12, kXwReady = 14, kXwFree = 16,
    kMReady = 18, kYFull, kYEmpty, kDFull, kDEmpty, kHReady, kHFree, kDrain, kBars
};
static_assert(kBars * 8 + 16 <= 256, "barrier room");

// tensor-memory columns
constexpr uint32_t kTS = 0, kTM = 256, kTYi = 320, kTYx = 384, kTD = 448;

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
    float* states;                   // [units][H][N][P]: read by the full form when `cut`, written by the state form
    float* decay;                    // [units][H] log: written by the state form
    __nv_bfloat16* save;             // state form: the state before every chunk, or null
    int cut, H, G, P, N;
    long long wait_ns;
};

__device__ __forceinline__ float4 exp2_4(float4 v) {
    return make_float4(ex2_approx(v.x), ex2_approx(v.y), ex2_approx(v.z), ex2_approx(v.w));
}

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
// (2^-24 of every term) where it is returned in fp32.
template <int kParts>
__global__ void __launch_bounds__(512, 1) scan_tc_kernel(const __grid_constant__ ScanMaps maps, const ScanTcArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + so::BAR);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + so::BAR + kBars * 8);
    volatile int* err = reinterpret_cast<volatile int*>(sm + so::BAR + kBars * 8 + 8);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int pb = a.P / kCols, h = blockIdx.x / pb, p0 = (blockIdx.x - h * pb) * kCols, grp = h / (a.H / a.G);
    Unit u;
    if (!find_unit(a.seqs, a.unit, blockIdx.y, u)) return;
    const int NC = (u.len + kQ - 1) / kQ;
    const long long lim = a.wait_ns;

    if (tid == 0) {
        const int counts[kBars] = {1, 1, 1, 1, 1, 1, 1, 1, 4, 4, 1, 1, 4, 4, 4, 4, 1, 1, 4, 1, 4, 1, 4, 4, 1, 1};
        for (int i = 0; i < kBars; ++i) mbar_init(bars + i, counts[i]);
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
    const uint32_t tmem = *tmem_slot;
    const int ks = a.N / 16;  // K steps over the state size
    const size_t plane = static_cast<size_t>(a.N) * a.P;

    if (warp == 0 || warp == 3) {
        // copies: B and C (warp 0) are free again earlier than X, whose room Y leaves through (warp 3)
        if (lane == 0) {
            const bool bc = warp == 0;
            const int full = bc ? kFull : kFullX, empty = bc ? kBcEmpty : kXEmpty, halves = a.N / 64;
            prefetch_tensormap(bc ? &maps.b : &maps.x);
            if (bc) prefetch_tensormap(&maps.c);
            int issued = 0;
            for (int c = 0; c < NC; ++c) {
                const int st = c & 1;
                if (c >= 2 && !mbar_wait_or_abort(bars + empty + st, ((c >> 1) & 1) ^ 1, lim, err)) {
                    note_failure(err);
                    break;
                }
                const int row = u.row + c * kQ;
                uint64_t* bar = bars + full + st;
                if (bc) {
                    mbar_arrive_expect_tx(bar, so::kTile * 2 * halves);
                    for (int k = 0; k < halves; ++k) {
                        tma_load_3d(sm + so::B + (2 * st + k) * so::kTile, &maps.b, 64 * k, grp, row, bar);
                        tma_load_3d(sm + so::C + (2 * st + k) * so::kTile, &maps.c, 64 * k, grp, row, bar);
                    }
                } else {
                    mbar_arrive_expect_tx(bar, so::kTile);
                    tma_load_3d(sm + so::X + st * so::kTile, &maps.x, p0, h, row, bar);
                }
                issued = c + 1;
            }
            for (int c = issued > 2 ? issued - 2 : 0; c < issued; ++c)  // nothing in flight when the block ends
                mbar_wait(bars + full + (c & 1), (c >> 1) & 1, kDefaultWaitNs);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t id_s = idesc_bf16(128, 128, false, false), id_d = idesc_bf16(128, 64, true, true),
                           id_x = idesc_bf16(128, 64, false, true), id_i = idesc_bf16(128, 64, false, true);
            bool ok = true;
            auto wait = [&](int bar, uint32_t parity) {
                if (!mbar_wait_or_abort(bars + bar, parity, lim, err)) {
                    note_failure(err);
                    return false;
                }
                tc_fence_after();
                return true;
            };
            auto scores = [&](int c) {
                const int st = c & 1;
                const uint32_t ph = (c >> 1) & 1;
                if (!wait(kFull + st, ph)) return false;
                if (u.len - c * kQ < kQ && !wait(kReady + st, ph)) return false;  // a short chunk's rows of B are cleared first
                if (c >= 2 && !wait(kSEmpty + st, ph ^ 1)) return false;
                const uint32_t ca = sb + so::C + 2 * st * so::kTile, ba = sb + so::B + 2 * st * so::kTile;
                for (int s = 0; s < ks; ++s) {
                    const uint32_t off = (s >> 2) * so::kTile + (s & 3) * 32;
                    mma_bf16(tmem + kTS + 128 * st, smem_desc(ca + off, 16, 1024, kSwizzle128B),
                             smem_desc(ba + off, 16, 1024, kSwizzle128B), id_s, s > 0);
                }
                mma_commit(bars + kSFull + st);
                return true;
            };
            ok = NC > 0 && scores(0);
            for (int c = 0; ok && c < NC; ++c) {
                const int st = c & 1;
                const uint32_t ph1 = c & 1;  // phase of the barriers used once per chunk
                if (c + 1 < NC && !(ok = scores(c + 1))) break;
                // state increment
                if (c >= 1 && !(ok = wait(kDEmpty, ph1 ^ 1))) break;
                for (int k = 0; ok && k < kParts; ++k) {
                    const int seq = c * kParts + k, buf = seq & 1;
                    if (!(ok = wait(kXwReady + buf, (seq >> 1) & 1))) break;
                    const uint32_t ba = sb + so::B + 2 * st * so::kTile, xa = sb + so::XW + buf * so::kTile;
                    for (int s = 0; s < 8; ++s)
                        mma_bf16(tmem + kTD, smem_desc(ba + s * 2048, so::kTile, 1024, kSwizzle128B),
                                 smem_desc(xa + s * 2048, so::kTile, 1024, kSwizzle128B), id_d, k > 0 || s > 0);
                    mma_commit(bars + kXwFree + buf);
                }
                if (!ok) break;
                mma_commit(bars + kDFull);
                // readout of the state
                if (!(ok = wait(kHReady, ph1))) break;
                if (c >= 1 && !(ok = wait(kYEmpty, ph1 ^ 1))) break;
                for (int s = 0; s < ks; ++s)
                    mma_bf16(tmem + kTYx, smem_desc(sb + so::C + 2 * st * so::kTile + (s >> 2) * so::kTile + (s & 3) * 32, 16, 1024, kSwizzle128B),
                             smem_desc(sb + so::HB + s * 2048, so::kTile, 1024, kSwizzle128B), id_x, s > 0);
                mma_commit(bars + kBcEmpty + st);
                mma_commit(bars + kHFree);
                // within the chunk
                if (!(ok = wait(kFullX + st, (c >> 1) & 1) && wait(kReady + st, (c >> 1) & 1) && wait(kMReady, ph1))) break;
                for (int s = 0; s < 8; ++s)
                    mma_bf16_ts(tmem + kTYi, tmem + kTM + 8 * s, smem_desc(sb + so::X + st * so::kTile + s * 2048, so::kTile, 1024, kSwizzle128B),
                                id_i, s > 0);
                mma_commit(bars + kYFull);
            }
            mma_commit(bars + kDrain);
            mbar_wait(bars + kDrain, 0, kDefaultWaitNs);
        }
    } else if (warp == 2) {
        // gates of the next chunk are in registers before this chunk's are due
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
        if (NC > 0) fetch(0);
        for (int c = 0; c < NC; ++c) {
            const int st = c & 1;
            if (!warp_wait(bars + kFull + st, (c >> 1) & 1, lim, err)) break;
            // the tail's rows of X are cleared here too; and X's arrival says that the arrays' readers are done
            if (!warp_wait(bars + kFullX + st, (c >> 1) & 1, lim, err)) break;
            gate_arrays(reinterpret_cast<float*>(sm + so::GATE + st * so::kGateStage), lane, gn, sn);
            const int n = u.len - c * kQ;
            if (n < kQ) {
                // the rows past the sequence hold other tokens: zeros, so that not even their NaN enters a sum
                const uint4 z = make_uint4(0, 0, 0, 0);
                for (int i = n * 8 + lane; i < kQ * 8; i += 32) {
                    reinterpret_cast<uint4*>(sm + so::B + 2 * st * so::kTile)[i] = z;
                    reinterpret_cast<uint4*>(sm + so::B + (2 * st + 1) * so::kTile)[i] = z;
                    reinterpret_cast<uint4*>(sm + so::X + st * so::kTile)[i] = z;
                }
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive1(bars + kReady + st);
            if (c + 1 < NC) fetch(c + 1);
        }
    } else if (warp >= 4 && warp < 8) {
        // ---- M: row i of the chunk per thread; blocks of 32 columns. Below the diagonal block the decay
        // factors through the end of the column's block (both factors <= 1), one exponential per row and
        // block; on it, one per entry. Blocks above stay the zeros written here.
        const int q = warp & 3, i = 32 * q + lane;
        const uint32_t lane_base = static_cast<uint32_t>(32 * q) << 16;
        {
            const uint32_t z[16] = {};
            for (int b = q + 1; b < 4; ++b) tmem_st16(tmem + lane_base + kTM + 16 * b, z);
            tmem_st_wait();
        }
        for (int c = 0; c < NC; ++c) {
            const int st = c & 1;
            const uint32_t ph = (c >> 1) & 1;
            if (!warp_wait(bars + kReady + st, ph, lim, err)) break;
            if (!warp_wait(bars + kSFull + st, ph, lim, err)) break;
            tc_fence_after();
            const float* arr = reinterpret_cast<const float*>(sm + so::GATE + st * so::kGateStage);
            const float Li = arr[i];
            uint32_t m[4][16];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                if (b > q) continue;
                float x[32];
                tmem_ld_cols<2>(tmem + lane_base + kTS + 128 * st + 32 * b, x);
                if (b == q) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive1(bars + kSEmpty + st);
#pragma unroll
                    for (int j4 = 0; j4 < 8; ++j4) {
                        const float4 L = *reinterpret_cast<const float4*>(arr + 32 * b + 4 * j4);
                        const float4 s = *reinterpret_cast<const float4*>(arr + 384 + 32 * b + 4 * j4);
                        const float l4[4] = {L.x, L.y, L.z, L.w}, s4[4] = {s.x, s.y, s.z, s.w};
                        float v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float w = ex2_approx(Li - l4[e]) * s4[e];
                            v[e] = 4 * j4 + e <= lane ? x[4 * j4 + e] * w : 0.f;
                        }
                        m[b][2 * j4] = pack_bf16x2(v[0], v[1]);
                        m[b][2 * j4 + 1] = pack_bf16x2(v[2], v[3]);
                    }
                } else {
                    const float rf = ex2_approx(Li - arr[32 * b + 31]);
                    const uint64_t rf2 = f32x2(rf, rf);
#pragma unroll
                    for (int j4 = 0; j4 < 8; ++j4) {
                        const float4 cf = *reinterpret_cast<const float4*>(arr + 128 + 32 * b + 4 * j4);
                        const uint64_t v0 = mul_f32x2(mul_f32x2(f32x2(x[4 * j4], x[4 * j4 + 1]), rf2), f32x2(cf.x, cf.y));
                        const uint64_t v1 = mul_f32x2(mul_f32x2(f32x2(x[4 * j4 + 2], x[4 * j4 + 3]), rf2), f32x2(cf.z, cf.w));
                        m[b][2 * j4] = bf16x2_narrow(v0);
                        m[b][2 * j4 + 1] = bf16x2_narrow(v1);
                    }
                }
            }
            if (c >= 1 && !warp_wait(bars + kYFull, (c - 1) & 1, lim, err)) break;  // the previous M has been used
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (b <= q) tmem_st16(tmem + lane_base + kTM + 16 * b, m[b]);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive1(bars + kMReady);
        }
    } else if (warp >= 8 && warp < 12) {
        // ---- Y: row i of the chunk per thread, all 64 columns; replaces the row of X and leaves by a bulk store
        const int q = warp & 3, i = 32 * q + lane;
        const uint32_t lane_base = static_cast<uint32_t>(32 * q) << 16;
        const float dk = a.d ? a.d[h] : 0.f;
        for (int c = 0; c < NC; ++c) {
            const int st = c & 1;
            if (!warp_wait(bars + kFullX + st, (c >> 1) & 1, lim, err)) break;
            if (!warp_wait(bars + kReady + st, (c >> 1) & 1, lim, err)) break;
            if (!warp_wait(bars + kYFull, c & 1, lim, err)) break;
            tc_fence_after();
            const float eL = ex2_approx(reinterpret_cast<const float*>(sm + so::GATE + st * so::kGateStage)[i]);
            uint8_t* xt = sm + so::X + st * so::kTile;
            const int n = u.len - c * kQ;
            __nv_bfloat16* yrow = a.y + (static_cast<size_t>(u.row + c * kQ + i) * a.H + h) * a.P + p0;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float yi[32], yx[32];
                tmem_ld_cols<2>(tmem + lane_base + kTYi + 32 * half, yi);
                tmem_ld_cols<2>(tmem + lane_base + kTYx + 32 * half, yx);
                if (half) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive1(bars + kYEmpty);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint4* cell = reinterpret_cast<uint4*>(xt + i * 128 + (((4 * half + k) ^ (i & 7)) << 4));
                    float xv[8], out[8];
                    unpack8(*cell, xv);
#pragma unroll
                    for (int e = 0; e < 8; ++e) out[e] = fmaf(dk, xv[e], fmaf(eL, yx[8 * k + e], yi[8 * k + e]));
                    const uint4 o = pack8(out);
                    if (n >= kQ) *cell = o;
                    else if (i < n) reinterpret_cast<uint4*>(yrow)[4 * half + k] = o;
                }
            }
            if (n >= kQ) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_3d(&maps.y, xt + 4096 * q, p0, h, u.row + c * kQ + 32 * q);
                    bulk_commit();
                    bulk_wait_read_all();
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive1(bars + kXEmpty + st);
        }
        if (lane == 0) bulk_wait_all();
    } else if (warp >= 12) {
        // ---- X~ of the next chunk, then the state over this one: row n of the state per thread, 64 columns
        const int q = warp & 3, r = 32 * q + lane;
        const uint32_t lane_base = static_cast<uint32_t>(32 * q) << 16;
        const bool real = r < a.N;
        const size_t at = static_cast<size_t>(real ? r : 0) * a.P + p0;
        float hx[64];
        {
            const float* from = a.cut ? a.states + (static_cast<size_t>(blockIdx.y) * a.H + h) * plane
                                      : (a.s0 ? a.s0 + (static_cast<size_t>(u.seq) * a.H + h) * plane : nullptr);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const float4 f = from && real ? reinterpret_cast<const float4*>(from + at)[k] : make_float4(0.f, 0.f, 0.f, 0.f);
                hx[4 * k] = f.x; hx[4 * k + 1] = f.y; hx[4 * k + 2] = f.z; hx[4 * k + 3] = f.w;
            }
        }
        uint8_t* hb = sm + so::HB;
        auto put_state = [&]() {
            st_row_bf16x32(hb, r, 0, hx);
            st_row_bf16x32(hb, r, 4, hx + 32);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive1(bars + kHReady);
        };
        float decay_next = 1.f;
        // X~ of chunk c, token row r: parts [first, first + 2) or the one at `first`, each the bf16 rounding of
        // what the parts before it leave
        auto weigh = [&](int c, int first, int count) -> bool {
            const int st = c & 1;
            if (!warp_wait(bars + kFullX + st, (c >> 1) & 1, lim, err)) return false;
            if (!warp_wait(bars + kReady + st, (c >> 1) & 1, lim, err)) return false;
            const float* arr = reinterpret_cast<const float*>(sm + so::GATE + st * so::kGateStage);
            const float w = arr[256 + r];
            decay_next = ex2_approx(arr[127]);
            for (int k = 0; k < count; ++k) {
                const int seq = c * kParts + first + k;
                if (seq >= 2 && !warp_wait(bars + kXwFree + (seq & 1), ((seq >> 1) & 1) ^ 1, lim, err)) return false;
            }
            const uint8_t* xt = sm + so::X + st * so::kTile + r * 128;
            uint8_t* to = sm + so::XW + r * 128;
            const int buf = (c * kParts + first) & 1;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int cell = (k ^ (r & 7)) << 4;
                float v[8], hi[8];
                unpack8(*reinterpret_cast<const uint4*>(xt + cell), v);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= w;
                uint4 o = pack8(v);
                if (kParts == 3) {
                    if (first == 0) *reinterpret_cast<uint4*>(to + buf * so::kTile + cell) = o;
                    unpack8(o, hi);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] -= hi[e];
                    o = pack8(v);
                    if (first == 0) {
                        *reinterpret_cast<uint4*>(to + (buf ^ 1) * so::kTile + cell) = o;
                    } else {
                        unpack8(o, hi);
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] -= hi[e];
                        *reinterpret_cast<uint4*>(to + buf * so::kTile + cell) = pack8(v);
                    }
                } else {
                    *reinterpret_cast<uint4*>(to + buf * so::kTile + cell) = o;
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                for (int k = 0; k < count; ++k) mbar_arrive1(bars + kXwReady + (buf ^ k));
            return true;
        };
        // Three parts share two buffers, so the third waits for the first one's product, and that product
        // for the previous increment to be read: with three parts X~ is formed after the state's update.
        auto weigh_all = [&](int c) { return kParts == 1 ? weigh(c, 0, 1) : weigh(c, 0, 2) && weigh(c, 2, 1); };
        bool ok = NC > 0;
        if (ok) {
            put_state();
            ok = weigh_all(0);
        }
        for (int c = 0; ok && c < NC; ++c) {
            const float decay = decay_next;
            if (kParts == 1 && c + 1 < NC && !(ok = weigh_all(c + 1))) break;
            if (!(ok = warp_wait(bars + kDFull, c & 1, lim, err))) break;
            tc_fence_after();
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float x[32];
                tmem_ld_cols<2>(tmem + lane_base + kTD + 32 * half, x);
#pragma unroll
                for (int k = 0; k < 32; ++k) hx[32 * half + k] = fmaf(decay, hx[32 * half + k], x[k]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive1(bars + kDEmpty);
            if (c + 1 < NC) {
                if (!(ok = warp_wait(bars + kHFree, c & 1, lim, err))) break;
                put_state();
                if (kParts > 1) ok = weigh_all(c + 1);
            }
        }
        if ((ok || NC == 0) && a.s1 && u.k == u.count - 1 && real) {
            float* to = a.s1 + (static_cast<size_t>(u.seq) * a.H + h) * plane + at;
#pragma unroll
            for (int k = 0; k < 16; ++k)
                reinterpret_cast<float4*>(to)[k] = make_float4(hx[4 * k], hx[4 * k + 1], hx[4 * k + 2], hx[4 * k + 3]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// [rows, heads, width] bf16 with a row stride, as (width, heads, rows); box (64, 1, box_rows)
bool rows_map(CUtensorMap* m, const void* p, long long ld, int width, int heads, long long rows, int box_rows) {
    const uint64_t dims[3] = {(uint64_t)width, (uint64_t)heads, (uint64_t)rows};
    const uint64_t st[2] = {(uint64_t)width * 2, (uint64_t)ld * 2};
    const uint32_t box[3] = {64, 1, (uint32_t)box_rows};
    return make_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p, dims, st, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int kParts>
cudaError_t launch_scan(const ScanMaps& maps, const ScanTcArgs& a, dim3 grid, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(scan_tc_kernel<kParts>, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
    if (e != cudaSuccess) return e;
    // the whole shared memory: one block per SM, and no operand descriptor reaches past the block's own
    scan_tc_kernel<kParts><<<grid, 512, 232448, s>>>(maps, a);
    return cudaGetLastError();
}

}  // namespace

bool ssm_tc_shape(const ScanShape& sh) {
    return sh.dt == GDN2_BF16 && sh.P % 64 == 0 && (sh.N == 64 || sh.N == 128) && sh.seqs.units(kQ) <= 65535;
}

size_t ssm_tc_fwd_workspace(const ScanShape&) { return 0; }

cudaError_t launch_ssm_tc_fwd(const ScanShape& sh, const ScanIn& in, void* y, float* s1, void*, cudaStream_t s, long long wait_ns) {
    ScanMaps maps;
    const long long rows = sh.seqs.rows();
    if (!rows_map(&maps.x, in.x.p, in.x.ld, sh.P, sh.H, rows, kQ) || !rows_map(&maps.b, in.bm.p, in.bm.ld, sh.N, sh.G, rows, kQ) ||
        !rows_map(&maps.c, in.cm.p, in.cm.ld, sh.N, sh.G, rows, kQ) || !rows_map(&maps.y, y, (long long)sh.H * sh.P, sh.P, sh.H, rows, 32))
        return cudaErrorInvalidValue;
    ScanTcArgs a{};
    a.seqs = sh.seqs;
    a.unit = (sh.seqs.T + kQ - 1) / kQ * kQ;
    a.step = static_cast<const __nv_bfloat16*>(in.step);
    a.g = static_cast<const __nv_bfloat16*>(in.g);
    a.d = in.d;
    a.s0 = in.s0;
    a.s1 = s1;
    a.y = static_cast<__nv_bfloat16*>(y);
    a.H = sh.H; a.G = sh.G; a.P = sh.P; a.N = sh.N;
    a.wait_ns = wait_ns;
    const dim3 grid(sh.H * (sh.P / kCols), static_cast<unsigned>(sh.seqs.units(a.unit)));
    return s1 ? launch_scan<3>(maps, a, grid, s) : launch_scan<1>(maps, a, grid, s);
}

int ssm_tc_read_clear_status(cudaStream_t s) {
    int v = 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_status_tc, sizeof(int), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess) return -1;
    if (cudaStreamSynchronize(s) != cudaSuccess) return -1;
    const int zero = 0;
    if (v && cudaMemcpyToSymbolAsync(g_status_tc, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s) != cudaSuccess) return -1;
    cudaStreamSynchronize(s);
    return v;
}

}  // namespace gdn2
