// ssm_tc_walk.cu -- the states of the selective state-space scan over chunks of 128 tokens, without outputs, on
// the tensor cores: what the gradients start from (the state before every chunk, and backwards the adjoint
// after it), and the increments that let a long sequence be cut into units.
//     forward   H' = e^{L_end} H + B^T X~,    X~_j = s_j e^{L_end - L_j} x_j
//     backward  A  = e^{L_end} A' + C^T Y~,   Y~_i = e^{L_i} dy_i
// One block per unit and 64 value columns of a head; both directions of a call run in one launch. Per chunk it
// reads the keys (from L2, shared by a group's heads) and the values once and writes nothing but the saved
// state. Both directions of 4 x 2048 tokens, 32 heads of 64 values, N = 128: 41 us for 134 MB of saved states and 290 MB
// of tiles from L2, 2.6 us per chunk and block: the latency of a chunk's tiles and its two handshakes, which two blocks per
// SM hide in part. Saved states are bf16, operands of products whose results are bf16.
#include "ssm_tc.cuh"

namespace gdn2 {
namespace {

// Stages of keys and values; X~ replaces its values in place, with three parts the other two have two sets of buffers.
// With one part two stages let two blocks share an SM and hide each other's waits; a tile takes 2300 cycles from its
// request, so the one block that three parts leave room for has three (two: 197 us instead of 160 us, now 157, for
// 2 x 32768 tokens, 32 heads).
template <int kParts>
struct Sw {
    static constexpr int kStages = kParts == 1 ? 2 : 3;
    static constexpr uint32_t K = 0;                                    // kStages x 2 tiles
    static constexpr uint32_t X = K + 2 * kStages * kTileBytes;         // kStages
    static constexpr uint32_t XW = X + kStages * kTileBytes;            // 2 sets x (kParts - 1)
    static constexpr uint32_t GATE = XW + 2 * (kParts - 1) * kTileBytes;  // {weight [128], decay} per stage
    static constexpr uint32_t kGateStage = 512 + 16;
    static constexpr uint32_t BAR = GATE + kStages * kGateStage;
    static constexpr uint32_t TOTAL = BAR + 160;
    static constexpr uint32_t kAlloc = TOTAL + 1024;
    static constexpr int kPerSm = kParts == 1 ? 2 : 1;
    static_assert(kPerSm * (kAlloc + 1024 + 16) <= 228 * 1024 && BAR % 8 == 0, "walk kernel shared memory");
};
enum WalkBar { wFull = 0, wReady = 3, wEmpty = 6, wXwReady = 9, wDFull = 12, wDEmpty = 14, wDrain = 16, wBars };
static_assert(wBars * 8 + 16 <= 160, "barrier room");
constexpr int kWalkThreadsTc = 384;

struct WalkMaps {
    CUtensorMap k[2], x[2];
};
struct WalkTcArgs {
    Seqs seqs;
    int unit, increments, cut, H, G, P, N;
    const __nv_bfloat16 *step, *g;
    WalkJob job[2];
    long long wait_ns;
};

template <int kParts>
__global__ void __launch_bounds__(kWalkThreadsTc, Sw<kParts>::kPerSm) walk_tc_kernel(const __grid_constant__ WalkMaps maps, const __grid_constant__ WalkTcArgs a) {
    using sw = Sw<kParts>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + sw::BAR);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + sw::BAR + wBars * 8);
    volatile int* err = reinterpret_cast<volatile int*>(sm + sw::BAR + wBars * 8 + 8);
    __shared__ float totals[2];
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    const WalkJob& job = a.job[blockIdx.z];
    const bool back = job.back != 0;
    const int pb = a.P / kCols, h = blockIdx.x / pb, pi = blockIdx.x - h * pb, p0 = pi * kCols, grp = h / (a.H / a.G);
    Unit u;
    if (!find_unit(a.seqs, a.unit, blockIdx.y, u)) return;
    u.len = uniform(u.len);
    u.row = uniform(u.row);
    const int NC = (u.len + kQ - 1) / kQ;
    const long long lim = a.wait_ns;

    if (tid == 0) {
        for (int i = 0; i < wBars; ++i)
            mbar_init(bars + i, (i >= wXwReady && i < wDFull) || (i >= wDEmpty && i < wDrain) ? 8 : 1);
        *err = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(tmem_slot, 128);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(*tmem_slot);
    const size_t plane = static_cast<size_t>(a.N) * a.P;
    auto chunk_at = [&](int c) { return back ? NC - 1 - c : c; };  // the c-th chunk walked over

    if (warp == 0) {
        if (lane == 0) {
            const int halves = a.N / 64;
            const CUtensorMap *mk = &maps.k[blockIdx.z], *mx = &maps.x[blockIdx.z];
            prefetch_tensormap(mk);
            prefetch_tensormap(mx);
            int n = 0;
            for (; n < NC; ++n) {
                const int st = n % sw::kStages, row = u.row + chunk_at(n) * kQ;
                if (n >= sw::kStages && !mbar_wait_or_abort(bars + wEmpty + st, ((n / sw::kStages) & 1) ^ 1, lim, err)) {
                    note_failure(err);
                    break;
                }
                mbar_arrive_expect_tx(bars + wFull + st, kTileBytes * (1 + halves));
                for (int k = 0; k < halves; ++k) tma_load_3d(sm + sw::K + (2 * st + k) * kTileBytes, mk, 64 * k, grp, row, bars + wFull + st);
                tma_load_3d(sm + sw::X + st * kTileBytes, mx, p0, h, row, bars + wFull + st);
            }
            for (int c = n > sw::kStages ? n - sw::kStages : 0; c < n; ++c)  // nothing in flight when the block ends
                mbar_wait(bars + wFull + c % sw::kStages, (c / sw::kStages) & 1, kDefaultWaitNs);
        }
    } else if (warp == 1) {
        const uint32_t id_d = idesc_bf16(128, 64, true, true), lead = elect_one();
        const uint32_t dm = desc_lo(sb, kTileBytes);
        bool ok = true;
        for (int c = 0; c < NC; ++c) {
            const int st = c % sw::kStages, set = c & 1;
            if (!(ok = wait_bar(bars + wXwReady + st, (c / sw::kStages) & 1, lim, err))) break;  // after the tiles' arrival
            if (c >= 2 && !(ok = wait_bar(bars + wDEmpty + set, ((c >> 1) & 1) ^ 1, lim, err))) break;
            tc_fence_after();
            const uint32_t km = dm + ((sw::K + 2 * st * kTileBytes) >> 4);
#pragma unroll 1
            for (int k = 0; k < kParts; ++k) {
                const uint32_t xa = dm + ((k ? sw::XW + (set * (kParts - 1) + k - 1) * kTileBytes : sw::X + st * kTileBytes) >> 4);
                mma_steps<false, kStepMn, kStepMn, 0, 0>(lead, tmem + 64 * set, km, xa, id_d, k > 0, 8);
            }
            commit_by(lead, bars + wDFull + set);
            commit_by(lead, bars + wEmpty + st);
        }
        commit_by(lead, bars + wDrain);
        mbar_wait(bars + wDrain, 0, kDefaultWaitNs);
    } else if (warp < 4) {
        // ---- gates, four tokens per lane. A head's values lie 2 H bytes apart and take 3500 cycles to arrive, about two
        // chunks: two warps take the chunks in turn, each with its next chunk's values in flight.
        float gn[4], sn[4], total = 0.f;
        auto fetch = [&](int c) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = chunk_at(c) * kQ + 4 * lane + e;
                const size_t at = static_cast<size_t>(u.row + t) * a.H + h;
                gn[e] = t < u.len ? ssm_gate(__bfloat162float(a.g[at])) * kLog2e : 0.f;
                sn[e] = back ? 1.f : t < u.len ? __bfloat162float(a.step[at]) : 0.f;
            }
        };
        if (warp - 2 < NC) fetch(warp - 2);
        for (int c = warp - 2; c < NC; c += 2) {
            const int st = c % sw::kStages;
            if (!wait_bar(bars + wFull + st, (c / sw::kStages) & 1, lim, err)) break;
            // forward: the decay behind the token up to the chunk's end; backward: up to and with the token.
            // Sums from the nearer side, so that small values keep their digits behind strong decays.
            float p[4], acc;
            if (back) {
                p[0] = gn[0]; p[1] = p[0] + gn[1]; p[2] = p[1] + gn[2]; p[3] = p[2] + gn[3];
                acc = p[3];
            } else {
                p[3] = 0.f; p[2] = gn[3]; p[1] = p[2] + gn[2]; p[0] = p[1] + gn[1];
                acc = p[0] + gn[0];
            }
            float incl = acc;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const float up = __shfl_up_sync(0xffffffffu, incl, d), dn = __shfl_down_sync(0xffffffffu, incl, d);
                if (back ? lane >= d : lane + d < 32) incl += back ? up : dn;
            }
            const float up = __shfl_up_sync(0xffffffffu, incl, 1), dn = __shfl_down_sync(0xffffffffu, incl, 1);
            const float base = back ? (lane ? up : 0.f) : (lane < 31 ? dn : 0.f);
            const float end = __shfl_sync(0xffffffffu, incl, back ? 31 : 0);
            total += end;
            float4 w = exp2_4(make_float4(base + p[0], base + p[1], base + p[2], base + p[3]));
            w.x *= sn[0]; w.y *= sn[1]; w.z *= sn[2]; w.w *= sn[3];
            uint8_t* arr = sm + sw::GATE + st * sw::kGateStage;
            reinterpret_cast<float4*>(arr)[lane] = w;
            if (lane == 0) *reinterpret_cast<float2*>(arr + 512) = kParts == 1 ? make_float2(ex2_approx(end), 0.f) : ssm_decay(kLn2 * end);
            const int n = u.len - chunk_at(c) * kQ;
            if (n < kQ) {  // the rows past the sequence hold other tokens: zeros, so that not even their NaN enters a sum
                const uint4 z = make_uint4(0, 0, 0, 0);
                for (int i = n * 8 + lane; i < kQ * 8; i += 32) {
                    reinterpret_cast<uint4*>(sm + sw::K + 2 * st * kTileBytes)[i] = z;
                    reinterpret_cast<uint4*>(sm + sw::K + (2 * st + 1) * kTileBytes)[i] = z;
                    reinterpret_cast<uint4*>(sm + sw::X + st * kTileBytes)[i] = z;
                }
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive1(bars + wReady + st);
            if (c + 2 < NC) fetch(c + 2);
        }
        if (lane == 0) totals[warp - 2] = total;
    } else if (warp >= 4) {
        // X~ of the next chunk, then the state over this one: row r per thread, half of the 64 columns per four warps
        const int q = warp & 3, half = warp >= 8, r = 32 * q + lane;
        const uint32_t lane_base = static_cast<uint32_t>(32 * q) << 16;
        const bool real = r < a.N;
        const size_t at = static_cast<size_t>(real ? r : 0) * a.P + p0 + 32 * half;
        const size_t unit_plane = (static_cast<size_t>(blockIdx.y) * a.H + h) * plane, seq_plane = (static_cast<size_t>(u.seq) * a.H + h) * plane;
        float hx[32];
        {
            const float* from = a.increments ? nullptr : a.cut ? job.states + unit_plane : (job.first ? job.first + seq_plane : nullptr);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float4 f = from && real ? reinterpret_cast<const float4*>(from + at)[k] : make_float4(0.f, 0.f, 0.f, 0.f);
                hx[4 * k] = f.x; hx[4 * k + 1] = f.y; hx[4 * k + 2] = f.z; hx[4 * k + 3] = f.w;
            }
        }
        const uint32_t tile = a.N * 128;  // bytes of a saved state
        uint8_t* save = nullptr;
        if (job.save && !a.increments) {
            const long long first_chunk = units_before(a.seqs, kQ, u.seq) + static_cast<long long>(u.k) * (a.unit / kQ);
            if (Seqs::held(first_chunk, NC, static_cast<int>(a.seqs.units(kQ))) == NC)
                save = static_cast<uint8_t*>(job.save) + ((static_cast<size_t>(first_chunk) * a.H + h) * pb + pi) * tile;
        }
        const size_t save_step = static_cast<size_t>(a.H) * pb * tile;
        float2 decay = make_float2(1.f, 0.f);
        bool ok = true;
        for (int c = -1; c < NC; ++c) {
            const int n = c + 1;
            const float2 decay_c = decay;
            if (n < NC) {
                const int st = n % sw::kStages;
                const uint32_t ph = (n / sw::kStages) & 1;
                if (!(ok = wait_bar(bars + wFull + st, ph, lim, err) && wait_bar(bars + wReady + st, ph, lim, err))) break;
                const float* arr = reinterpret_cast<const float*>(sm + sw::GATE + st * sw::kGateStage);
                const float w = arr[r];
                decay = *reinterpret_cast<const float2*>(arr + 128);
                uint8_t* xt = sm + sw::X + st * kTileBytes + r * 128;
                uint8_t* more = sm + sw::XW + (n & 1) * (kParts - 1) * kTileBytes + r * 128;  // of two chunks before: taken with its increment
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
                        *reinterpret_cast<uint4*>((part ? more + (part - 1) * kTileBytes : xt) + cell) = o;
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
                if (lane == 0) mbar_arrive1(bars + wXwReady + st);
            }
            if (c >= 0) {
                const int set = c & 1;
                if (!(ok = wait_bar(bars + wDFull + set, (c >> 1) & 1, lim, err))) break;
                tc_fence_after();
                float x[32];
                tmem_ld_cols<2>(tmem + lane_base + 64 * set + 32 * half, x);
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const uint64_t h2 = f32x2(hx[2 * k], hx[2 * k + 1]), d2 = f32x2(x[2 * k], x[2 * k + 1]);
                    f32x2_split(fma_f32x2(f32x2(decay_c.x, decay_c.x), h2, kParts == 1 ? d2 : fma_f32x2(f32x2(decay_c.y, decay_c.y), h2, d2)),
                                hx[2 * k], hx[2 * k + 1]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive1(bars + wDEmpty + set);
            }
            if (save && n < NC && real)  // the 32-byte sectors of the operand layout are whole
                st_row_bf16x32(save + static_cast<size_t>(chunk_at(n)) * save_step, r, 4 * half, hx);
        }
        float* to = nullptr;
        if (ok && a.increments) to = job.states + unit_plane;
        else if (ok && job.last && u.k == (back ? 0 : u.count - 1)) to = job.last + seq_plane;
        if (to && real) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                reinterpret_cast<float4*>(to + at)[k] = make_float4(hx[4 * k], hx[4 * k + 1], hx[4 * k + 2], hx[4 * k + 3]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (a.increments && tid == 0 && pi == 0) job.decay[static_cast<size_t>(blockIdx.y) * a.H + h] = (totals[0] + totals[1]) * kLn2;
    if (warp == 0) tmem_dealloc(*tmem_slot, 128);
}

}  // namespace

cudaError_t launch_ssm_walk_tc(const ScanShape& sh, const void* step, const void* g, const WalkJob* jobs, int n_jobs, int unit,
                               int increments, int cut, int exact, cudaStream_t s, long long wait_ns) {
    WalkMaps maps;
    WalkTcArgs a{};
    const long long rows = sh.seqs.rows();
    for (int i = 0; i < n_jobs; ++i) {
        a.job[i] = jobs[i];
        if (!rows_map(&maps.k[i], jobs[i].keys.p, jobs[i].keys.ld, sh.N, sh.G, rows, kQ) ||
            !rows_map(&maps.x[i], jobs[i].values.p, jobs[i].values.ld, sh.P, sh.H, rows, kQ))
            return cudaErrorInvalidValue;
    }
    a.seqs = sh.seqs;
    a.unit = unit;
    a.increments = increments;
    a.cut = cut;
    a.H = sh.H; a.G = sh.G; a.P = sh.P; a.N = sh.N;
    a.step = static_cast<const __nv_bfloat16*>(step);
    a.g = static_cast<const __nv_bfloat16*>(g);
    a.wait_ns = wait_ns;
    auto* kernel = exact ? walk_tc_kernel<3> : walk_tc_kernel<1>;
    const uint32_t smem = exact ? Sw<3>::kAlloc : Sw<1>::kAlloc;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    g_launched.store(true, std::memory_order_relaxed);
    kernel<<<dim3(sh.H * (sh.P / kCols), static_cast<unsigned>(sh.seqs.units(unit)), n_jobs), kWalkThreadsTc, smem, s>>>(maps, a);
    return cudaGetLastError();
}

int ssm_tc_walk_read_clear_status(cudaStream_t s) { return read_clear_status(s); }

}  // namespace gdn2
