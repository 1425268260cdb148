// attn_decode_tc.cuh -- part of attn_decode.cu: units of up to 32 query rows over bf16 caches, both products in tensor memory.
//
// 128 keys a step. The keys are the 128 rows of the product, the query rows its columns: S^T = K Q^T [128 keys][32 rows], then
// O^T += V^T [weights, their rest] [D][32 + 32], so that neither product has rows to spare, and K and V are used as they lie: K with its
// width along the depth, V with its keys along it. Weights enter as two bf16 parts (2^-17) side by side, which one pass over V takes.
// Three warps copy (a ring of K and V tiles), one issues the products, four make weights of scores: a thread has one key and all rows of the
// scores, one column of the output and all rows of it. (A ninth warp would leave each thread 168 registers, and these need more.) The maximum
// that weights refer to follows the scores only where they pass it by 8, as in the other form.
//
// 16 rows of 7600 to 8192 tokens, 4 tokens of 32/4 heads of 128: 61 us for 38 of copies, of which 5 are the joining launch and some 12 the
// way in and out of a unit, a good part of it code that runs for the first time. In between a step of 64 KB takes 1.5 us, a little more than its share of
// the copy rate, with the copying warps never idle for long; its chain (scores, weights, values) takes 1.3. Copies of 16 bytes a lane instead
// of tensor copies: 75 (what pages that are no multiples of 16 keys get); products issued by a warp that makes weights too: 77; every loop
// over rows unrolled: 69; tensor copies of 64 keys: 62 for 58 with one row of 131072 tokens.
#pragma once

#include "ssm_tc.cuh"

namespace gdn2 {
namespace {

constexpr int kTcRows = 32, kTcKeys = 128, kTcWarps = 8, kTcThreads = 32 * kTcWarps;
constexpr int kPanel = 16384;  // 128 keys by 64 columns, 128 bytes a row, swizzled

template <int D>
struct TcLayout {
    static constexpr int kPanels = D / 64, kTileBytes = kPanels * kPanel;
    static constexpr int kSlots = D == 128 ? 6 : 3;  // tiles in the ring
    static constexpr unsigned kAhead = D == 128 ? 4 : 2;  // tiles on their way behind the one that is waited for; fewer than slots, or none comes free
    static constexpr int kKept = D == 128 ? 256 : 32;
    static constexpr int kQ = kSlots * kTileBytes, kP = kQ + kTcRows * D * 2, kSmall = kP + kPanel;
    static constexpr int kScores = 0, kOut = 64, kColumns = D == 128 ? 128 : 256;  // tensor memory: two sets of scores, then 64 columns per 128 of the width
};

template <int D>
struct TcSmall {
    uint64_t full[TcLayout<D>::kSlots], empty[TcLayout<D>::kSlots], scored[2], weighed, added, asked, drain;
    long long red[kTcWarps], first;
    uint32_t tmem;
    int row, err;
    alignas(16) unsigned short seen[TcLayout<D>::kSlots][8];  // which of a tile's keys were copied
    Limits lim[kTcRows];
    float over[4][kTcRows];  // per warp: maxima, sums
    unsigned hidden[kTcKeys];  // of the step's keys: rows that do not see them
    int2 kept[TcLayout<D>::kKept];
};

// The pools as (width, key of a page, page and head), 64 columns of 16 keys at a time.
struct CacheMaps {
    CUtensorMap k, v;
};

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}
// As tma_load_3d, by the lane that has `lead`; the operands are the warp's, so that they lie in uniform registers (with a lane per panel each copy
// took 170 cycles to issue).
__device__ __forceinline__ void tma_load_by(uint32_t lead, uint32_t to, const void* map, int c0, int c1, int c2, uint64_t* bar) {
    asm volatile(
        "{\n .reg .pred e;\n setp.ne.b32 e, %6, 0;\n"
        " @e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n}\n" ::"r"(to),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar)), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// Lane r leaves with the combination over all lanes of x[r].
template <typename F>
__device__ __forceinline__ float across(float (&x)[32], F f) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 16; h; h >>= 1) {
        const bool up = lane & h;
#pragma unroll
        for (int i = 0; i < h; ++i) {
            const float keep = up ? x[i + h] : x[i], give = up ? x[i] : x[i + h];
            x[i] = f(keep, __shfl_xor_sync(0xffffffffu, give, h));
        }
    }
    return x[0];
}

__device__ __forceinline__ void weights_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool weights_any(bool v) {
    uint32_t r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
                 : "=r"(r)
                 : "r"(static_cast<uint32_t>(v))
                 : "memory");
    return r != 0;
}

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1)
    decode_tc_kernel(const __grid_constant__ DecodeArgs a, const __grid_constant__ CacheMaps maps, const bool maps_used) {
    using Lay = TcLayout<D>;
    using Walk = Cursor<kTcKeys>;
    constexpr int kSlots = Lay::kSlots, kChunks = D / 8, kBlocks = D / 128;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    TcSmall<D>& x = *reinterpret_cast<TcSmall<D>*>(sm + Lay::kSmall);
    const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5), units = a.Hkv * a.tiles;
    volatile int* err = &x.err;
    const long long lim = a.wait_ns;

    auto clear_row = [&](int b) {
        const int n = vectors_of(a.N, a.Hq, a.d, 2);
        uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + static_cast<long long>(b) * a.N * a.Hq * a.d);
        for (int i = lane; i < n; i += 32) o[i] = make_uint4(0, 0, 0, 0);
    };
    auto row_span = [&](int b) { return b < Lay::kKept ? span_of(a, x.kept[b].x, x.kept[b].y) : span_of(a, b); };
    if (!a.whole) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    Walk at;
    if (a.whole) {
        at.b = blockIdx.x / units;
        at.span = span_of(a, at.b);
        at.steps = steps_of<kTcKeys>(at.span);
        at.ht = blockIdx.x - at.b * units;
        at.step = 0;
        at.left = at.steps;
        if (at.steps == 0) {
            if (at.ht == 0 && warp == 0 && at.span.slot >= 0) clear_row(at.b);
            return;
        }
    } else {
        for (int b = tid; b < min(a.B, Lay::kKept); b += kTcThreads) {
            const Span s = span_of(a, b);
            x.kept[b] = make_int2(s.slot, s.hi);
        }
        if (tid == 0) x.row = -1;
        __syncthreads();
        for (int b = blockIdx.x * kTcWarps + warp; b < a.B; b += gridDim.x * kTcWarps) {
            const Span s = row_span(b);
            if (s.slot >= 0 && steps_of<kTcKeys>(s) == 0) clear_row(b);
        }
        if (!begin_stretch<kTcThreads, kTcKeys>(a, row_span, units, x.red, &x.row, &x.first, at)) return;
    }

    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(x.full + i, 3);
            mbar_init(x.empty + i, 5);  // the product, and the four warps that look at the tile
        }
        mbar_init(x.scored, 1);
        mbar_init(x.scored + 1, 1);
        mbar_init(&x.weighed, 4);
        mbar_init(&x.added, 1);
        mbar_init(&x.asked, 4);
        mbar_init(&x.drain, 1);
        x.err = 0;
        fence_mbar_init();
    }
    if (warp == 4) {
        tmem_alloc(&x.tmem, Lay::kColumns);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = x.tmem, sb = smem_u32(sm);

    if (warp >= 5) {
        // ---- copies: of a step's eight groups of 16 keys two or three per warp, K and then V. A group that lies in one page and is all there
        // comes by a tensor copy of each 64 columns (copies of 16 bytes a lane held the loads to 27 bytes a cycle and SM, L2 or not); others
        // come key by key, zeros where there is none.
        const int part = warp - 5, chunks = a.d / 8, panels = (a.d + 63) / 64;
        const unsigned char *kp = static_cast<const unsigned char*>(a.k), *vp = static_cast<const unsigned char*>(a.v);
        const long long row_bytes = 2LL * a.d;
        int head = at.ht / a.tiles;
        // A key of a step: its table entry, asked for a step ahead, and its place in the page; negative where it is not one to read.
        struct Key {
            int entry, in;
        };
        auto look = [&](int key) -> Key {
            const int t = at.span.base() + at.step * kTcKeys + key, u = min(t, at.span.hi - 1);
            int i = __umulhi(u, a.page_inverse), in = u - i * a.cache.page;  // u / page, give or take one
            const int off = in < 0 ? -1 : in >= a.cache.page ? 1 : 0;
            i += off;
            in -= off * a.cache.page;
            return Key{__ldg(a.cache.table + static_cast<long long>(at.span.slot) * a.cache.max_pages + i), t == u && t >= at.span.lo ? in : -1};
        };
        auto is = [&](const Key& k) { return k.in >= 0 && k.entry >= 0 && k.entry < a.cache.n_pages; };
        // group g of the warp's is group part + 3 g of the step; lanes look up one key of its first two, the lower ones one of the third
        const int groups = part < 2 ? 3 : 2;
        const int key0 = (part + 3 * (lane / 16)) * 16 + (lane & 15), key1 = (part + 6) * 16 + (lane & 15);
        constexpr int kRowsPer = 32 / kChunks;  // keys that one copy of all lanes spans
        const int lane_row = lane / kChunks, chunk = lane % kChunks;
        Key next0 = look(key0), next1 = look(key1);
        const uint32_t lead = elect_one();
        int slot = 0;
        unsigned tiles = 0;
        bool ok = true;
        // What came key by key into tile j has landed. With pages that take no tensor copies that is looked at kAhead tiles later; where only the
        // ends of rows come so, at once.
        auto give = [&](unsigned j) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive1(x.full + j % kSlots);
        };
        if (lane < 2 && maps_used) prefetch_tensormap(lane ? &maps.v : &maps.k);
        while (ok && at.left > 0) {
            const Key here0 = next0, here1 = next1;
            const int here_head = head;
            const unsigned there0 = __ballot_sync(0xffffffffu, is(here0)), there1 = __ballot_sync(0xffffffffu, is(here1));
            auto there = [&](int g) { return (g < 2 ? there0 >> 16 * g : there1) & 0xffffu; };
            if (at.next(a, row_span, 1)) head = at.ht / a.tiles;
            if (at.left > 0) {
                next0 = look(key0);
                next1 = look(key1);
            }
            unsigned whole = 0;  // groups that come by tensor copies
            if (maps_used) {
#pragma unroll
                for (int g = 0; g < 3; ++g) whole |= static_cast<unsigned>(g < groups && there(g) == 0xffffu) << g;
            }
            const bool all = whole == (1u << groups) - 1u;
            const unsigned before = tiles;
#pragma unroll 1
            for (int kv = 0; kv < 2; ++kv, ++tiles) {
                if (tiles >= kSlots && !(ok = wait_bar(x.empty + slot, (tiles / kSlots - 1) & 1, lim, err))) break;
                uint64_t* bar = x.full + slot;
                if (lane == 0) {
#pragma unroll
                    for (int g = 0; g < 3; ++g)
                        if (g < groups) x.seen[slot][part + 3 * g] = static_cast<unsigned short>(there(g));
                    if (all) mbar_arrive_expect_tx(bar, groups * panels * 2048);
                    else if (whole) mbar_expect_tx(bar, __popc(whole) * panels * 2048);
                }
                __syncwarp();
                unsigned char* tile = sm + slot * Lay::kTileBytes;
                const unsigned char* src = (kv ? vp : kp) + 16 * chunk;
#pragma unroll
                for (int g = 0; g < 3; ++g) {
                    if (!(whole >> g & 1)) continue;
                    const Key& of = g < 2 ? here0 : here1;
                    const int in = __shfl_sync(0xffffffffu, of.in, (g & 1) * 16), plane = __shfl_sync(0xffffffffu, of.entry, (g & 1) * 16) * a.Hkv + here_head;
                    const uint32_t to = smem_u32(tile) + (part + 3 * g) * 2048;
#pragma unroll
                    for (int p = 0; p < Lay::kPanels; ++p)
                        if (p < panels) tma_load_by(lead, to + p * kPanel, kv ? &maps.v : &maps.k, 64 * p, in, plane, bar);
                }
#pragma unroll 1
                for (int g = 0; g < groups; ++g) {
                    if (!(whole >> g & 1)) {
                        const int from = (g & 1) * 16;
                        const Key of = g < 2 ? here0 : here1;
                        const unsigned some = there(g);
                        // all addresses first: a copy behind each one's shuffle would wait for it
                        long long row[16 / kRowsPer];
                        const long long mine = is(of) ? ((static_cast<long long>(of.entry) * a.Hkv + here_head) * a.cache.page + of.in) * row_bytes : 0;
#pragma unroll
                        for (int i = 0; i < 16 / kRowsPer; ++i) row[i] = __shfl_sync(0xffffffffu, mine, from + i * kRowsPer + lane_row);
                        if (chunk < chunks) {
#pragma unroll
                            for (int i = 0; i < 16 / kRowsPer; ++i) {
                                const int r = i * kRowsPer + lane_row, key = (part + 3 * g) * 16 + r;
                                copy16(smem_u32(tile) + chunk / 8 * kPanel + key * 128 + (((chunk & 7) ^ (key & 7)) << 4), src + row[i], some >> r & 1);
                            }
                        }
                    }
                }
                copies_commit();
                slot = slot == kSlots - 1 ? 0 : slot + 1;
                if (!maps_used && tiles >= Lay::kAhead) {
                    copies_wait<Lay::kAhead>();
                    give(tiles - Lay::kAhead);
                }
            }
            if (maps_used && !all)
                for (unsigned j = before; j < tiles; ++j) {  // K, then V
                    if (j + 1 < tiles) copies_wait<1>();
                    else copies_wait<0>();
                    give(j);
                }
        }
        if (!maps_used)
            for (unsigned j = tiles > Lay::kAhead ? tiles - Lay::kAhead : 0; j < tiles; ++j) {
                if (j + 3 < tiles) copies_wait<3>();
                else if (j + 2 < tiles) copies_wait<2>();
                else if (j + 1 < tiles) copies_wait<1>();
                else copies_wait<0>();
                give(j);
            }
        copies_wait<0>();  // nothing on its way when the block ends
        for (unsigned j = tiles > kSlots ? tiles - kSlots : 0; j < tiles; ++j) mbar_wait(x.full + j % kSlots, (j / kSlots) & 1, kDefaultWaitNs);
    } else if (warp == 4) {
        // ---- products
        const uint32_t lead = elect_one();
        constexpr uint32_t id_s = idesc_bf16(128, kTcRows, false, false), id_o = idesc_bf16(128, 2 * kTcRows, true, true);
        const int depth = a.d / 16;
        int slot = 0, phase = 0, vslot = 1, vphase = 0;  // the next keys, the next values
        unsigned n = 0, unit = 0;
        bool ok = true;
        auto step_slot = [&](int& s, int& p) {
            s = s == kSlots - 1 ? 0 : s + 1;
            if (s == 0) p ^= 1;
        };
        // scores of step m from the tile of keys in slot s, which has landed
        auto score = [&](unsigned m, int s) {
            tc_fence_after();
            const uint32_t ka = desc_lo(sb + s * Lay::kTileBytes, 16), qb = desc_lo(sb + Lay::kQ, 16), to = tmem + Lay::kScores + 32 * (m & 1);
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
                if (i < depth) mma_by(lead, to, ka + i / 4 * (kPanel / 16) + i % 4 * 2, qb + i / 4 * (kTcRows * 128 / 16) + i % 4 * 2, id_s, i > 0);
            commit_by(lead, x.empty + s);
            commit_by(lead, x.scored + (m & 1));
        };
        auto add = [&](int s) {
            tc_fence_after();
            const uint32_t va = desc_lo(sb + s * Lay::kTileBytes, kPanel), pb = desc_lo(sb + Lay::kP, kPanel);
#pragma unroll
            for (int c = 0; c < kBlocks; ++c)
#pragma unroll
                for (int k = 0; k < kTcKeys / 16; ++k) mma_by(lead, tmem + Lay::kOut + 64 * c, va + c * (2 * kPanel / 16) + k * 128, pb + k * 128, id_o, 1);
            commit_by(lead, x.empty + s);
            commit_by(lead, &x.added);
        };
        while (ok && at.left > 0) {
            const int n_steps = static_cast<int>(at.left < at.steps - at.step ? at.left : at.steps - at.step);
            ok = wait_bar(&x.asked, unit++ & 1, lim, err);
            // steps whose scores have been issued, and whose values have; scores run a step ahead if their keys are there
            for (int m = 0, i = 0; ok && i < n_steps;) {
                if (m < n_steps && m <= i + 1) {
                    const bool must = m == i;
                    if (must && !(ok = wait_bar(x.full + slot, phase, lim, err))) break;
                    if (must || __all_sync(0xffffffffu, mbar_test_wait(x.full + slot, phase))) {
                        score(n + m, slot);
                        step_slot(slot, phase);  // the values of step m, and the keys of the next
                        step_slot(slot, phase);
                        ++m;
                        if (must) continue;
                    }
                }
                if (!(ok = wait_bar(&x.weighed, (n + i) & 1, lim, err) && wait_bar(x.full + vslot, vphase, lim, err))) break;
                add(vslot);
                step_slot(vslot, vphase);
                step_slot(vslot, vphase);
                ++i;
            }
            n += n_steps;
            at.next(a, row_span, n_steps);
        }
        if (!ok) {  // no product on its way when the block ends
            commit_by(lead, &x.drain);
            mbar_wait(&x.drain, 0, kDefaultWaitNs);
        }
    } else {
        // ---- weights: this thread's key of a step, and this thread's columns of the output
        const uint32_t mine = tmem + (static_cast<uint32_t>(32 * warp) << 16);
        const int chunks = a.d / 8;
        int slot = 0, phase = 0;
        unsigned n = 0;
        bool failed = false, stop = false;
        float top, ref[kTcRows], l[kTcRows];  // top: row `lane`'s reference maximum, which ref has of all rows
        auto take8 = [&](int column, float (&v)[8]) {
            uint32_t u[8];
            tmem_ld8(mine + Lay::kOut + column, u);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[i]);
        };
        auto put8 = [&](int column, const float (&v)[8]) {
            uint32_t u[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(v[i]);
            tmem_st8(mine + Lay::kOut + column, u);
        };
        auto step_slot = [&]() {
            slot = slot == kSlots - 1 ? 0 : slot + 1;
            if (slot == 0) phase ^= 1;
        };
        while (!stop && at.left > 0) {
            const int unit_row = at.ht % a.tiles * kTcRows, head = at.ht / a.tiles;
            const int n_steps = static_cast<int>(at.left < at.steps - at.step ? at.left : at.steps - at.step);
            const int valid = min(kTcRows, a.N * a.G - unit_row);
            // the unit's queries, zeros for rows that it does not have; the products of the unit before have ended
            uint4 asked[kTcRows * kChunks / 128];
#pragma unroll
            for (int i = 0; i < kTcRows * kChunks / 128; ++i) {
                const int r = (tid + 128 * i) / kChunks, c = tid % kChunks, row = unit_row + r, t = row / a.G;
                const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) + (static_cast<long long>(at.b) * a.N + t) * a.ld_q +
                                           static_cast<long long>(head * a.G + row - t * a.G) * a.d + c * 8;
                asked[i] = r < valid && c < chunks ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < kTcRows * kChunks / 128; ++i) {
                const int r = (tid + 128 * i) / kChunks, c = tid % kChunks;
                *reinterpret_cast<uint4*>(sm + Lay::kQ + c / 8 * (kTcRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = asked[i];
            }
            if (tid < kTcRows) x.lim[tid] = limits_of(a, at.span, unit_row + tid);
            const float zero[8] = {};
#pragma unroll 1
            for (int c = 0; c < 64 * kBlocks; c += 8) put8(c, zero);
            tmem_st_wait();
            tc_fence_before();
            fence_proxy_async_smem();
            top = kNone;
#pragma unroll
            for (int r = 0; r < kTcRows; ++r) {
                ref[r] = kNone;
                l[r] = 0.f;
            }
            const Limits newest = limits_of(a, at.span, unit_row + valid - 1), oldest = limits_of(a, at.span, unit_row);
            __syncwarp();
            if (lane == 0) mbar_arrive1(&x.asked);
            weights_sync();  // limits are there
            for (int i = 0; i < n_steps; ++i, ++n) {
                const int base = at.span.base() + (at.step + i) * kTcKeys, key = base + tid;
                failed |= !wait_bar(x.scored + (n & 1), (n >> 1) & 1, lim, err);
                tc_fence_after();
                float s[kTcRows], z[kTcRows];
                tmem_ld_cols<2>(mine + Lay::kScores + 32 * (n & 1), s);
                failed |= !wait_bar(x.full + slot, phase, lim, err);  // has come to pass: for what lies in `seen`
                const unsigned there = reinterpret_cast<const unsigned*>(x.seen[slot])[warp];
                __syncwarp();
                if (lane == 0) mbar_arrive1(x.empty + slot);
                step_slot();  // to the values
                const bool plain = there == 0xffffffffu && base + 32 * warp >= newest.low && base + 32 * warp + 31 <= oldest.limit;
                unsigned hidden = 0;  // rows that do not see this key
                if (!plain) {
#pragma unroll 2
                    for (int r = 0; r < kTcRows; ++r) hidden |= static_cast<unsigned>(!(there >> lane & 1) || key < x.lim[r].low || key > x.lim[r].limit) << r;
                }
                bool over = failed;
#pragma unroll
                for (int r = 0; r < kTcRows; ++r) {
                    z[r] = fmaf(s[r], a.scale, -ref[r]);  // a row without a reference yet: +inf, or NaN
                    if (hidden >> r & 1) z[r] = kNone;
                    over |= !(z[r] <= 8.f);
                }
                if (weights_any(over)) {
                    // Some score passes its row's reference by 8: such rows' references to their maxima, sums and output with them. The others
                    // stay as they are, so that no row's bits depend on another's scores.
                    if ((stop = weights_any(failed))) break;
                    float v[kTcRows];
#pragma unroll
                    for (int r = 0; r < kTcRows; ++r) v[r] = hidden >> r & 1 ? kNone : s[r] * a.scale;
                    x.over[warp][lane] = across(v, [](float p, float q) { return fmaxf(p, q); });
                    weights_sync();
                    const float most = fmaxf(fmaxf(x.over[0][lane], x.over[1][lane]), fmaxf(x.over[2][lane], x.over[3][lane]));
                    const float now = most > top + 8.f ? most : top;
                    const float f = now == kNone ? 0.f : ex2_approx(top - now);
                    top = now;
#pragma unroll
                    for (int r = 0; r < kTcRows; ++r) {
                        ref[r] = __shfl_sync(0xffffffffu, now, r);
                        l[r] *= __shfl_sync(0xffffffffu, f, r);
                        // Scores of -inf alone: weights of 0. A score that is +inf when scaled makes its row NaN, though its product may be finite: 0 times
                        // such a reference is NaN (by comparison with it: 16 drafts 64 us, so 62).
                        const float by = ref[r] == kNone ? 0.f : fmaf(0.f, ref[r], -ref[r]);
                        z[r] = hidden >> r & 1 ? kNone : fmaf(s[r], a.scale, by);
                    }
                    if (i > 0) {
                        failed |= !wait_bar(&x.added, (n - 1) & 1, lim, err);
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < 64 * kBlocks; c += 8) {
                            float o[8];
                            take8(c, o);
#pragma unroll
                            for (int e = 0; e < 8; ++e) o[e] *= __shfl_sync(0xffffffffu, f, (c & 31) + e);
                            put8(c, o);
                        }
                        tmem_st_wait();
                    }
                }
                uint32_t hi[kTcRows / 2], lo[kTcRows / 2];
#pragma unroll
                for (int r = 0; r < kTcRows; r += 2) {
                    const float p = ex2_approx(z[r]), q = ex2_approx(z[r + 1]);
                    l[r] += p;
                    l[r + 1] += q;
                    const uint32_t u = pack_bf16x2(p, q);
                    hi[r / 2] = u;
                    lo[r / 2] = pack_bf16x2(p - __uint_as_float(u << 16), q - __uint_as_float(u & 0xffff0000u));
                }
                if (n > 0) failed |= !wait_bar(&x.added, (n - 1) & 1, lim, err);  // the last weights have been read
                uint8_t* p = sm + Lay::kP + tid * 128;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    *reinterpret_cast<uint4*>(p + ((c ^ (tid & 7)) << 4)) = make_uint4(hi[4 * c], hi[4 * c + 1], hi[4 * c + 2], hi[4 * c + 3]);
                    *reinterpret_cast<uint4*>(p + (((4 + c) ^ (tid & 7)) << 4)) = make_uint4(lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]);
                }
                // Keys that some of the unit's tokens see and others do not: their values may not be finite, which a weight of 0 does not keep
                // out. Their products are made here, for the rows that see them, and the matrix product takes zeros for them.
                const int begin = max(base, at.span.lo), end = min(base + kTcKeys, at.span.hi);  // of what is there
                if (begin < newest.low || end - 1 > oldest.limit) {
                    failed |= !wait_bar(x.full + slot, phase, lim, err);
                    tc_fence_after();
                    x.hidden[tid] = hidden;
                    weights_sync();  // all weights are there
                    // the keys behind what the oldest token sees, then those before what the newest one does
                    const int from = max(base, oldest.limit + 1), to = min(base + kTcKeys - 1, newest.limit);
                    const int low = max(base, oldest.low), high = min(min(base + kTcKeys, newest.low), from) - 1;
                    const int late = max(to - from + 1, 0), some = late + max(high - low + 1, 0);
                    auto value_at = [&](int c, int k) {  // of this thread's column
                        return reinterpret_cast<__nv_bfloat16*>(sm + slot * Lay::kTileBytes + (2 * c + tid / 64) * kPanel + sw128_off(k, tid & 63));
                    };
                    // what no token of the unit sees, though another unit of the row does
                    for (int c = 0; c < kBlocks; ++c) {
                        for (int k = max(newest.limit + 1, base) - base; k < end - base; ++k) *value_at(c, k) = __float2bfloat16_rn(0.f);
                        for (int k = begin - base; k < min(oldest.low, end) - base; ++k) *value_at(c, k) = __float2bfloat16_rn(0.f);
                    }
#pragma unroll 1
                    for (int c = 0; c < 4 * kBlocks; ++c) {  // 128 columns, eight rows
                        const int q = c & 3;
                        float sum[8];
                        take8(64 * (c / 4) + 8 * q, sum);
#pragma unroll 1
                        for (int j = 0; j < some; ++j) {
                            const int k = (j < late ? from + j : low + j - late) - base;
                            __nv_bfloat16* value = value_at(c / 4, k);
                            const float v = __bfloat162float(*value);
                            if (q == 3) *value = __float2bfloat16_rn(0.f);
                            const uint8_t* w = sm + Lay::kP + k * 128;
                            const unsigned blind = x.hidden[k] >> 8 * q;
                            float whi[8], wlo[8];
                            unpack8(*reinterpret_cast<const uint4*>(w + ((q ^ (k & 7)) << 4)), whi);
                            unpack8(*reinterpret_cast<const uint4*>(w + (((4 + q) ^ (k & 7)) << 4)), wlo);
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float with = fmaf(whi[e] + wlo[e], v, sum[e]);
                                if (!(blind >> e & 1)) sum[e] = with;
                            }
                        }
                        put8(64 * (c / 4) + 8 * q, sum);
                    }
                    tmem_st_wait();
                }
                tc_fence_before();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive1(&x.weighed);
                    mbar_arrive1(x.empty + slot);
                }
                step_slot();
            }
            if (stop) break;
            // The unit's sums, and its way out. They take the place of the last step's maxima, which a warp may still be reading if that step moved a
            // reference (a unit of one step always does): the four warps meet first.
            weights_sync();
            x.over[warp][lane] = across(l, [](float p, float q) { return p + q; });
            failed |= !wait_bar(&x.added, (n - 1) & 1, lim, err);
            tc_fence_after();
            weights_sync();
            const float total = (x.over[0][lane] + x.over[1][lane]) + (x.over[2][lane] + x.over[3][lane]);
            const bool done = n_steps == at.steps;
            const float inv = !done ? 1.f : total == 0.f ? 0.f : 1.f / total;  // a row that sees nothing is zero
            __nv_bfloat16* to = static_cast<__nv_bfloat16*>(a.o) + (static_cast<long long>(at.b) * a.N * a.Hq + head * a.G) * a.d;
            float* part = done ? nullptr : part_of(a, blockIdx.x, at.step == 0 ? 1 : 0, D, kTcRows);
            int t = unit_row / a.G, h = unit_row - t * a.G;
#pragma unroll 1
            for (int r0 = 0; r0 < valid; r0 += 8) {
                float hi[kBlocks][8], lo[kBlocks][8];
#pragma unroll
                for (int c = 0; c < kBlocks; ++c) {
                    take8(64 * c + r0, hi[c]);
                    take8(64 * c + 32 + r0, lo[c]);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float by = __shfl_sync(0xffffffffu, inv, r0 + e);
                    if (r0 + e < valid) {
#pragma unroll
                        for (int c = 0; c < kBlocks; ++c) {
                            const int column = 128 * c + tid;
                            const float v = (hi[c][e] + lo[c][e]) * by;
                            if (part) part[(r0 + e) * D + column] = v;
                            else if (column < a.d) to[(static_cast<long long>(t) * a.Hq + h) * a.d + column] = __float2bfloat16_rn(v);
                        }
                    }
                    if (++h == a.G) {
                        h = 0;
                        ++t;
                    }
                }
            }
            if (part && warp == 0) {
                part[kTcRows * D + lane] = top;
                part[kTcRows * D + kTcRows + lane] = total;
            }
            tc_fence_before();
            at.next(a, row_span, n_steps);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 4) tmem_dealloc(tmem, Lay::kColumns);
}

}  // namespace
}  // namespace gdn2
