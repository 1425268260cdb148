// attn_decode.cu -- attention of a row's newest tokens over its pages of keys and values (attn_common.cuh):
//     o = softmax(scale q K^T over the visible tokens) V,   token n of N sees the tokens up to length - N + n (and within the window)
//
// Every key and value is read once for 4 N H_q / H_kv operations per element: bound by memory. A unit is the cache of one key head of one
// row against 16 or 32 of its query rows (N tokens times the heads of the group); its keys are cut into steps of 16 per warp. All units'
// steps, one after another, are dealt out to the blocks in equal stretches, found from the lengths on the device: a long row is split over
// many blocks and short rows share one, whatever the batch. Each warp streams its own keys through its own stages of shared memory, by
// asynchronous copies that run ahead across units, and keeps its own running maximum, sum and output: no block barrier but at a unit's end,
// where the warps' results are joined. A unit that lies in one block leaves as the result; of one that does not, each block leaves its part
// in the workspace, and a second launch joins the parts in their order (no atomics).
//
// 131072 tokens of 8 key heads of 128 in bf16: 88 us, 6.1 TB/s (0.90 of the copy rate); 64 rows of 0 to 16384 tokens, 2 heads of 256: 162 us
// (0.93). Of the time, some 12 us are the way in (lengths, table, first keys) and out (parts), whatever the length. The products have 16
// rows where a tensor-memory product has 128, so they run on warp-wide matrix instructions: their pipe is a quarter busy at the copy rate.
// More than 16 query rows (drafted tokens) are another matter: with two tiles a warp the latency of a step's chain bounds it, so heads wider
// than 64 take attn_decode_tc.cuh (16 rows of 8192 tokens, 4 tokens of 32/4 heads of 128: 61 us, with two tiles here 72; heads of 256, 8 rows: 62 and,
// each tile reading everything, 99).
#include "attn_common.cuh"

namespace gdn2 {
namespace {

constexpr int kTile = 16;   // query rows of a matrix instruction; a unit has one or two such tiles
constexpr int kKeys = 16;   // keys of a warp's step
constexpr int kKept = 256;  // rows whose slots and lengths a block keeps
constexpr float kNone = -INFINITY;

struct DecodeArgs {
    const void *q, *k, *v;
    void* o;
    float* parts;
    long long ld_q;
    Cache cache;
    int B, N, Hq, Hkv, G, d, tiles, window;  // tiles: units per key head
    bool whole;                              // a block per unit
    unsigned page_inverse;                   // 2^32 / page, rounded up (page 1: 2^32 - 1)
    float scale;  // times log2 e
    long long wait_ns;
};

// What a row asks for: the keys [lo, hi) that its earliest and latest tokens see between them. Its steps start at a multiple of a warp's keys,
// so that with pages of such multiples a warp's step lies in one page.
struct Span {
    int slot, lo, hi;
    __device__ __forceinline__ int base() const { return lo & ~(kKeys - 1); }
};
__device__ __forceinline__ Span span_of(const DecodeArgs& a, int slot, int length) {
    return Span{slot, a.window ? max(length - a.N - a.window + 1, 0) : 0, length};
}
__device__ __forceinline__ Span span_of(const DecodeArgs& a, int b) {
    const int slot = a.cache.row_of(b);
    return slot < 0 ? Span{-1, 0, 0} : span_of(a, slot, a.cache.length_of(slot));
}

// 16-byte vectors of a row's output, which has up to 2^31 elements (and so more bytes than an int counts); d is a multiple of 16.
__host__ __device__ constexpr int vectors_of(int N, int Hq, int d, int esize) { return N * Hq * d / (16 / esize); }
static_assert(vectors_of(4096, 512, 256, 4) == 1 << 27 && vectors_of(4096, 4096, 64, 2) == 1 << 27, "counted without overflow");

template <int kStep>
__device__ __forceinline__ int steps_of(const Span& s) {
    return s.hi > s.lo ? (s.hi - s.base() + kStep - 1) / kStep : 0;
}

// Inclusive sum over the block's threads in order; total: of all of them.
template <int kThreads>
__device__ __forceinline__ long long block_scan(long long v, long long* red, long long& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += o;
    }
    __syncthreads();  // the last call's readers
    if (lane == 31) red[warp] = v;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w == warp) v += total;
        total += red[w];
    }
    return v;
}

// Steps and tolls of a block: all blocks together cover them. One is enough (900 tokens of 4 key heads: 9.7 us; with two at least 12.4, four 13.8).
__device__ __forceinline__ long long steps_per_block(long long total, int blocks) {
    const long long per = (total + blocks - 1) / blocks;
    return per > 0 ? per : 1;
}

// ---------------------------------------------------------------------------------------------------------------------------------

__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Place of 16-byte chunk c of row r in a tile whose rows are `chunks` long: neighbouring rows' equal chunks lie in other banks.
__device__ __forceinline__ int place(int r, int c, int chunks) { return r * chunks + (c ^ (r & 7)); }

// W warps and S stages, M tiles of query rows per unit.
template <typename T, int D, int W, int S, int M>
struct Layout {
    static constexpr int kThreads = 32 * W, kStep = kKeys * W, kRows = kTile * M;
    static constexpr int kChunks = D * (int)sizeof(T) / 16;                         // 16-byte chunks of a key
    static constexpr int kHalf = kKeys * kChunks * 16, kStage = 2 * kHalf;          // K and V
    static constexpr int kQ = kRows * kChunks * 16, kOut = kRows * D * 4;
    static constexpr int kProb = sizeof(T) == 4 ? W * (kKeys * kRows + kRows) * 4 : 0;  // fp32: a step's weights and factors, per warp
    static constexpr int kSmem = W * S * kStage + kQ + kOut + kProb;
};

// What a unit costs beside its steps, in steps: its queries' way in, the joining of its warps, and its way out. Stretches are dealt out by steps
// and toll, or a block that gets a run of rows of one token each would take as long as several: 59 rows of which every other holds a few
// tokens take 26 us (51 without toll, 32 with 1, 29 with 8), 64 ragged rows 162 (169, 168, 160).
constexpr int kToll = 4;
__device__ __forceinline__ long long cost_of(int steps, int units) { return steps > 0 ? static_cast<long long>(steps + kToll) * units : 0; }

// All rows' costs in a row, dealt out in stretches: a thread has a run of rows, `mine` their cost, `behind` the cost up to and with them.
template <int kThreads, int kStep>
struct Dealing {
    int run, first, last;
    long long mine, behind, total;
    template <typename Rows>
    __device__ __forceinline__ void count(const DecodeArgs& a, const Rows& rows, int units, long long* red) {
        run = (a.B + kThreads - 1) / kThreads;
        first = min(static_cast<int>(threadIdx.x) * run, a.B);
        last = min(first + run, a.B);
        mine = 0;
#pragma unroll 8
        for (int b = first; b < last; ++b) mine += cost_of(steps_of<kStep>(rows(b)), units);
        behind = block_scan<kThreads>(mine, red, total);
    }
    // Leaves the row that holds place v among all costs, and the cost before that row; with a barrier behind it. The whole block takes part; a run
    // of several rows is looked at once more, a thread per row.
    template <typename Rows>
    __device__ __forceinline__ void find(const DecodeArgs& a, const Rows& rows, int units, long long v, long long* red, int* row, long long* before) const {
        if (v >= behind - mine && v < behind) {
            *row = first;
            *before = behind - mine;
        }
        __syncthreads();
        if (run == 1 || *row < 0) return;
        const int from = *row;
        long long at = *before;
        for (int i = 0; i < run; i += kThreads) {
            const int b = from + i + threadIdx.x;
            const long long n = i + static_cast<int>(threadIdx.x) < run && b < a.B ? cost_of(steps_of<kStep>(rows(b)), units) : 0;
            long long sum;
            const long long upto = at + block_scan<kThreads>(n, red, sum);  // its barriers lie behind everyone's look at row and before
            if (v >= upto - n && v < upto) {
                *row = b;
                *before = upto - n;
            }
            at += sum;
        }
        __syncthreads();
    }
};

// Where a block's walk over its stretch stands, and the steps (and tolls) that are left of it. The lanes of a warp walk together.
template <int kStep>
struct Cursor {
    int b, ht, step, steps;  // row; key head and tiles of query rows; step of the unit and its steps
    long long left;
    Span span;
    // To row b or the first after it that has steps, 32 rows at a look; nothing is left behind the last one.
    template <typename Rows>
    __device__ __forceinline__ void settle(const DecodeArgs& a, const Rows& rows) {
        const int lane = threadIdx.x & 31;
        for (; b < a.B; b += 32) {
            const Span s = b + lane < a.B ? rows(b + lane) : Span{-1, 0, 0};
            const int n = steps_of<kStep>(s);
            const unsigned some = __ballot_sync(0xffffffffu, n > 0);
            if (some) {
                const int from = __ffs(some) - 1;
                b += from;
                steps = __shfl_sync(0xffffffffu, n, from);
                span = Span{__shfl_sync(0xffffffffu, s.slot, from), __shfl_sync(0xffffffffu, s.lo, from), __shfl_sync(0xffffffffu, s.hi, from)};
                return;
            }
        }
        span = Span{-1, 0, 0};
        steps = 0;
        left = 0;
    }
    // Goes on; true when that is another unit.
    template <typename Rows>
    __device__ __forceinline__ bool next(const DecodeArgs& a, const Rows& rows, int by) {
        step += by;
        left -= by;
        if (step < steps || left <= 0) return false;
        step = 0;
        left -= kToll;
        if (++ht < a.Hkv * a.tiles) return true;
        ht = 0;
        ++b;
        settle(a, rows);
        return true;
    }
};

// Sets a block's walk to the start of its stretch of all steps and tolls; false: the block has nothing to do. The whole block takes part.
template <int kThreads, int kStep, typename Rows>
__device__ __forceinline__ bool begin_stretch(const DecodeArgs& a, const Rows& rows, int units, long long* red, int* row, long long* first, Cursor<kStep>& at) {
    Dealing<kThreads, kStep> all;
    all.count(a, rows, units, red);
    const long long per = steps_per_block(all.total, gridDim.x);
    const long long begin = blockIdx.x * per, end = begin + per < all.total ? begin + per : all.total;
    if (begin >= end) return false;
    all.find(a, rows, units, begin, red, row, first);
    if (*row < 0) return false;  // not with lengths that stay as they are
    at.b = *row;
    at.left = end - begin;
    at.settle(a, rows);
    if (at.left <= 0) return false;
    // a unit's toll lies in front of its steps
    const long long in = begin - *first;
    at.ht = static_cast<int>(in / (at.steps + kToll));
    const int place = static_cast<int>(in - static_cast<long long>(at.ht) * (at.steps + kToll));
    at.step = max(place - kToll, 0);
    at.left -= max(kToll - place, 0);
    return at.left > 0;
}

// The part of a query row of the unit: which of the row's tokens it is, and the keys it sees, [low, limit].
struct Limits {
    int low, limit;
};
__device__ __forceinline__ Limits limits_of(const DecodeArgs& a, const Span& s, int row) {
    const int n = row / a.G;
    if (row >= a.N * a.G) return {0, -1};
    const int last = s.hi - a.N + n;
    return {a.window ? max(last - a.window + 1, 0) : 0, last};
}

// bf16: both products on matrix instructions of 16 x 8 x 16, a warp's 16 keys as two columns' worth of scores and one depth of V. Weights
// enter the second product as two bf16 parts (2^-17), so that the result's only rounding is its own; the sum takes them in fp32. The maximum
// that weights refer to follows the scores only where they pass it by 8: until then a weight is at most 2^8, and the output is not rescaled
// (64 rows: 175 -> 170 us). One tile keeps its queries in registers up to 128 wide; two share every fragment of K and V that is read.
template <int D, int M>
struct WarpBf16 {
    static constexpr int kChunks = D / 8, kDepth = D / 16;
    static constexpr bool kHeld = M == 1 && D <= 128;
    float o[M][D / 8][4], m[M][2], l[M][2];
    Limits lim[M][2];
    uint32_t held[kHeld ? kDepth : 1][4];

    __device__ __forceinline__ void begin(const DecodeArgs& a, const Span& s, int unit_row) {
        const int g = (threadIdx.x & 31) / 4;
#pragma unroll
        for (int k = 0; k < M; ++k) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                lim[k][h] = limits_of(a, s, unit_row + kTile * k + g + 8 * h);
                m[k][h] = kNone;
                l[k][h] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[k][i][j] = 0.f;
        }
    }
    // With the unit's queries in shared memory.
    __device__ __forceinline__ void queries(uint32_t qt) {
        if constexpr (kHeld) {
            const int lane = threadIdx.x & 31;
#pragma unroll
            for (int i = 0; i < kDepth; ++i) ldm4(held[i], qt + 16 * place((lane & 7) + ((lane >> 3) & 1) * 8, 2 * i + (lane >> 4), kChunks));
        }
    }

    // o += weights V. kMasked: with V's keys under masks (zeros where hidden), and for the lane's rows of which `mine` has a bit alone.
    template <bool kMasked>
    __device__ __forceinline__ void add_values(uint32_t vt, const uint32_t (&hi)[M][4], const uint32_t (&lo)[M][4], uint32_t m0 = 0, uint32_t m1 = 0,
                                               unsigned mine = 0) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            uint32_t r[4];
            ldm4t(r, vt + 16 * place((lane & 7) + ((lane >> 3) & 1) * 8, 2 * i + (lane >> 4), kChunks));
#pragma unroll
            for (int k = 0; k < M; ++k) {
                if constexpr (kMasked) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float (&c)[4] = o[k][2 * i + h];
                        float t[4] = {c[0], c[1], c[2], c[3]};
                        mma(t, hi[k], r[2 * h] & m0, r[2 * h + 1] & m1);
                        mma(t, lo[k], r[2 * h] & m0, r[2 * h + 1] & m1);
                        if (mine >> (2 * k) & 1) {
                            c[0] = t[0];
                            c[1] = t[1];
                        }
                        if (mine >> (2 * k + 1) & 1) {
                            c[2] = t[2];
                            c[3] = t[3];
                        }
                    }
                } else {
                    mma(o[k][2 * i], hi[k], r[0], r[1]);
                    mma(o[k][2 * i + 1], hi[k], r[2], r[3]);
                    mma(o[k][2 * i], lo[k], r[0], r[1]);
                    mma(o[k][2 * i + 1], lo[k], r[2], r[3]);
                }
            }
        }
    }

    // Keys base .. base + 15 of the row, those that `there` has a bit for (the others' places hold zeros); all: every row sees them. Rows that
    // the unit does not have see what they like: their queries are zeros, and nobody reads them.
    __device__ __forceinline__ void step(const DecodeArgs& a, const unsigned char* q, const unsigned char* kv, const unsigned char* values, int base,
                                         unsigned there, bool all, int unit_row, int first, int last, const Span& span, float*) {
        const int lane = threadIdx.x & 31, t = lane & 3;
        const uint32_t qt = smem_u32(q), kt = smem_u32(kv), vt = smem_u32(values);
        float s[M][2][4] = {};
#pragma unroll
        for (int i = 0; i < kDepth; ++i) {
            uint32_t kb[4];
            ldm4(kb, kt + 16 * place((lane & 7) + (lane >> 4) * 8, 2 * i + ((lane >> 3) & 1), kChunks));
#pragma unroll
            for (int k = 0; k < M; ++k) {
                uint32_t qa[4];
                if constexpr (kHeld) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) qa[j] = held[i][j];
                } else {
                    ldm4(qa, qt + 16 * place(kTile * k + (lane & 7) + ((lane >> 3) & 1) * 8, 2 * i + (lane >> 4), kChunks));
                }
                mma(s[k][0], qa, kb[0], kb[1]);
                mma(s[k][1], qa, kb[2], kb[3]);
            }
        }
        uint32_t hi[M][4], lo[M][4];
#pragma unroll
        for (int k = 0; k < M; ++k) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[k][i][j] *= a.scale;
            if (!all || there != 0xffffu) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int key = 8 * i + 2 * t + (j & 1), at = base + key;
                        const Limits& x = lim[k][j >> 1];
                        if (!(there >> key & 1) || at < x.low || at > x.limit) s[k][i][j] = kNone;
                    }
            }
            float top[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x = fmaxf(fmaxf(s[k][0][2 * h], s[k][0][2 * h + 1]), fmaxf(s[k][1][2 * h], s[k][1][2 * h + 1]));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                top[h] = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
            }
            if (__any_sync(0xffffffffu, top[0] > m[k][0] + 8.f || top[1] > m[k][1] + 8.f)) {
                float f[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float now = top[h] > m[k][h] + 8.f ? top[h] : m[k][h];  // each row by itself: its bits are not another's matter
                    f[h] = now == kNone ? 0.f : ex2_approx(m[k][h] - now);
                    m[k][h] = now;
                    l[k][h] *= f[h];
                }
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    o[k][i][0] *= f[0]; o[k][i][1] *= f[0]; o[k][i][2] *= f[1]; o[k][i][3] *= f[1];
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float ref = m[k][h] == kNone ? 0.f : m[k][h];  // no key yet: every weight is 2^-inf = 0
#pragma unroll
                for (int i = 0; i < 2; ++i) {  // (row, keys 0-7), (row + 8, keys 0-7), then keys 8-15
                    const float x = ex2_approx(s[k][i][2 * h] - ref), y = ex2_approx(s[k][i][2 * h + 1] - ref);
                    l[k][h] += x + y;
                    const uint32_t u = pack2(x, y);
                    hi[k][2 * i + h] = u;
                    lo[k][2 * i + h] = pack2(x - __uint_as_float(u << 16), y - __uint_as_float(u & 0xffff0000u));
                }
            }
        }
        if (all) {
            add_values<false>(vt, hi, lo);
            return;
        }
        // A key that one token sees and another does not may hold a value that is not finite, which a weight of 0 would not keep out:
        // token by token, with the values hidden from it as zeros, and no product of another token's kept.
        for (int n = first; n <= last; ++n) {
            const Limits x = limits_of(a, span, n * a.G);
            auto sees = [&](int key) { return base + key >= x.low && base + key <= x.limit; };
            const uint32_t m0 = (sees(2 * t) ? 0xffffu : 0u) | (sees(2 * t + 1) ? 0xffff0000u : 0u);
            const uint32_t m1 = (sees(2 * t + 8) ? 0xffffu : 0u) | (sees(2 * t + 9) ? 0xffff0000u : 0u);
            unsigned mine = 0;
#pragma unroll
            for (int k = 0; k < 2 * M; ++k) mine |= static_cast<unsigned>((unit_row + lane / 4 + 8 * k) / a.G == n) << k;
            add_values<true>(vt, hi, lo, m0, m1, mine);
        }
    }

    // Reference maximum and sum of each row, from the lanes that hold them.
    __device__ __forceinline__ void statistics(float* ms, float* ls) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int k = 0; k < M; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[k][h] += __shfl_xor_sync(0xffffffffu, l[k][h], 1);
                l[k][h] += __shfl_xor_sync(0xffffffffu, l[k][h], 2);
                if ((lane & 3) == 0) {
                    ms[kTile * k + lane / 4 + 8 * h] = m[k][h];
                    ls[kTile * k + lane / 4 + 8 * h] = l[k][h];
                }
            }
    }

    // Adds this warp's output, each row times its factor, to the block's: one W-th of the columns a round, each warp another one.
    template <int W>
    __device__ __forceinline__ void add_to(float* out, const float* factor, int round) {
        const int lane = threadIdx.x & 31, t = lane & 3, mine = (threadIdx.x / 32 + round) % W;
        constexpr int kPart = D / 8 / W;
#pragma unroll
        for (int c = 0; c < W; ++c) {
            if (c != mine) continue;
#pragma unroll
            for (int k = 0; k < M; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = kTile * k + lane / 4 + 8 * h;
                    const float f = factor[row];
#pragma unroll
                    for (int i = c * kPart; i < (c + 1) * kPart; ++i) {
                        float2* p = reinterpret_cast<float2*>(out + row * D + 8 * i + 2 * t);
                        float2 v = round ? *p : make_float2(0.f, 0.f);
                        v.x = fmaf(f, o[k][i][2 * h], v.x);
                        v.y = fmaf(f, o[k][i][2 * h + 1], v.y);
                        *p = v;
                    }
                }
        }
    }
};

// fp32: on CUDA cores. Scores: a lane takes one of the 16 keys and every other query row; values: a lane takes D / 32 columns. Rows are
// counted up to a power of two, so that the loops over them unroll and their loads run ahead.
template <int D>
struct WarpF32 {
    static constexpr int kRows = kTile, kCols = D / 32, kHalf = kRows / 2, kChunks = D / 4;
    float o[kRows][kCols], m[kHalf], l[kHalf];
    Limits lim[kHalf];
    int rows;

    // The lane's column c: runs of four, 128 apart.
    __device__ __forceinline__ static int column(int lane, int c) { return D == 64 ? 2 * lane + c : c / 4 * 128 + 4 * lane + c % 4; }

    __device__ __forceinline__ void queries(uint32_t) {}
    __device__ __forceinline__ void begin(const DecodeArgs& a, const Span& s, int unit_row) {
        const int half = (threadIdx.x & 31) / 16;
        rows = min(kRows, a.N * a.G - unit_row);
#pragma unroll
        for (int i = 0; i < kHalf; ++i) {
            lim[i] = limits_of(a, s, unit_row + 2 * i + half);
            m[i] = kNone;
            l[i] = 0.f;
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int c = 0; c < kCols; ++c) o[r][c] = 0.f;
    }

    __device__ __forceinline__ void step(const DecodeArgs& a, const unsigned char* q, const unsigned char* k, const unsigned char* v, int base,
                                         unsigned there, bool all, int unit_row, int, int, const Span& span, float* prob) {
        if (rows <= 2) step_rows<2>(a, q, k, v, base, there, all, unit_row, span, prob);
        else if (rows <= 4) step_rows<4>(a, q, k, v, base, there, all, unit_row, span, prob);
        else if (rows <= 8) step_rows<8>(a, q, k, v, base, there, all, unit_row, span, prob);
        else step_rows<16>(a, q, k, v, base, there, all, unit_row, span, prob);
    }

    template <int R>
    __device__ __forceinline__ void step_rows(const DecodeArgs& a, const unsigned char* qs, const unsigned char* ks, const unsigned char* vs, int base,
                                              unsigned there, bool all, int unit_row, const Span& span, float* prob) {
        const int lane = threadIdx.x & 31, key = lane & 15, half = lane / 16;
        float s[R / 2][2] = {};
#pragma unroll 4
        for (int c = 0; c < kChunks; c += 2)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float4 k = *reinterpret_cast<const float4*>(ks + 16 * place(key, c + e, kChunks));
#pragma unroll
                for (int i = 0; i < R / 2; ++i) {
                    const float4 q = *reinterpret_cast<const float4*>(qs + 16 * place(2 * i + half, c + e, kChunks));
                    s[i][e] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, s[i][e]))));
                }
            }
        float* factor = prob + kKeys * kRows;
#pragma unroll
        for (int i = 0; i < R / 2; ++i) {
            const int at = base + key;
            const float z = (there >> key & 1) && at >= lim[i].low && at <= lim[i].limit ? (s[i][0] + s[i][1]) * a.scale : kNone;
            float x = z;
#pragma unroll
            for (int d = 8; d; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
            const float now = fmaxf(m[i], x), ref = now == kNone ? 0.f : now;
            const float f = exp2f(m[i] - ref), p = exp2f(z - ref);
            m[i] = now;
            l[i] = fmaf(l[i], f, p);  // this lane's keys
            prob[key * kRows + 2 * i + half] = p;
            if (key == 0) factor[2 * i + half] = f;
        }
        __syncwarp();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float f = factor[r];
#pragma unroll
            for (int c = 0; c < kCols; ++c) o[r][c] *= f;
        }
        auto value = [&](int j, float (&x)[kCols]) {
            if constexpr (D == 64) {
                const float2 u = *reinterpret_cast<const float2*>(vs + 16 * place(j, lane / 2, kChunks) + 8 * (lane & 1));
                x[0] = u.x;
                x[1] = u.y;
            } else {
#pragma unroll
                for (int g = 0; g < kCols / 4; ++g) {
                    const float4 u = *reinterpret_cast<const float4*>(vs + 16 * place(j, 32 * g + lane, kChunks));
                    x[4 * g] = u.x; x[4 * g + 1] = u.y; x[4 * g + 2] = u.z; x[4 * g + 3] = u.w;
                }
            }
        };
        if (all) {
#pragma unroll 4
            for (int j = 0; j < kKeys; ++j) {
                float x[kCols];
                alignas(16) float p[R];
                value(j, x);
                if constexpr (R == 2) {
                    *reinterpret_cast<float2*>(p) = *reinterpret_cast<const float2*>(prob + j * kRows);
                } else {
#pragma unroll
                    for (int r = 0; r < R; r += 4) *reinterpret_cast<float4*>(p + r) = *reinterpret_cast<const float4*>(prob + j * kRows + r);
                }
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int c = 0; c < kCols; ++c) o[r][c] = fmaf(p[r], x[c], o[r][c]);
            }
        } else {  // a value that is not finite is kept out of the rows that do not see its key
            for (int j = 0; j < kKeys; ++j) {
                float x[kCols];
                value(j, x);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const Limits see = limits_of(a, span, unit_row + r);
                    if (base + j < see.low || base + j > see.limit) continue;
                    const float p = prob[j * kRows + r];
#pragma unroll
                    for (int c = 0; c < kCols; ++c) o[r][c] = fmaf(p, x[c], o[r][c]);
                }
            }
        }
        __syncwarp();
    }

    __device__ __forceinline__ void statistics(float* ms, float* ls) {
        const int lane = threadIdx.x & 31, half = lane / 16;
#pragma unroll
        for (int i = 0; i < kHalf; ++i) {
#pragma unroll
            for (int d = 8; d; d >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
            if ((lane & 15) == 0) {
                ms[2 * i + half] = m[i];
                ls[2 * i + half] = l[i];
            }
        }
    }

    // As for bf16, by rows.
    template <int W>
    __device__ __forceinline__ void add_to(float* out, const float* factor, int round) {
        const int lane = threadIdx.x & 31, mine = (threadIdx.x / 32 + round) % W;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (r / (kRows / W) != mine) continue;
            const float f = factor[r];
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
                float* p = out + r * D + column(lane, c);
                *p = fmaf(f, o[r][c], round ? *p : 0.f);
            }
        }
    }
};

template <typename T, int D, int M>
struct WarpOf;
template <int D, int M>
struct WarpOf<__nv_bfloat16, D, M> {
    using type = WarpBf16<D, M>;
};
template <int D>
struct WarpOf<float, D, 1> {
    using type = WarpF32<D>;
};

// A block's part of a unit that it does not hold whole: the output of its rows, their maxima and sums. Two per block: of the unit that began
// before its stretch, and of the one that goes on behind it.
__host__ __device__ constexpr long long part_floats(int D, int rows) { return static_cast<long long>(rows) * (D + 2); }
__device__ __forceinline__ float* part_of(const DecodeArgs& a, long long block, int which, int D, int rows) {
    return a.parts + (block * 2 + which) * part_floats(D, rows);
}

// kPaged: pages are multiples of a warp's keys, so a warp's step lies in one page.
template <typename T, int D, int W, int S, int M, bool kPaged>
__global__ void __launch_bounds__(32 * W) decode_kernel(const __grid_constant__ DecodeArgs a) {
    using Lay = Layout<T, D, W, S, M>;
    constexpr int kThreads = Lay::kThreads, kStep = Lay::kStep, kChunks = Lay::kChunks, kEl = 16 / (int)sizeof(T), kRows = Lay::kRows;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ long long red[W], shared_first;
    __shared__ int shared_row;
    __shared__ int2 kept[kKept];
    __shared__ unsigned seen[W][S];  // which of a stage's keys were copied
    __shared__ float sm[W][kRows], sl[W][kRows], sf[W][kRows], top[kRows], sum[kRows];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    const int units = a.Hkv * a.tiles;
    unsigned char* stages = smem + warp * S * Lay::kStage;
    unsigned char* qs = smem + W * S * Lay::kStage;
    float* out = reinterpret_cast<float*>(qs + Lay::kQ);
    float* prob = out + kRows * D + warp * (kKeys * kRows + kRows);

    // Rows without a visible key: a warp clears one.
    auto clear_row = [&](int b) {
        const int n = vectors_of(a.N, a.Hq, a.d, sizeof(T));
        uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(a.o) + static_cast<long long>(b) * a.N * a.Hq * a.d);
        for (int i = lane; i < n; i += 32) o[i] = make_uint4(0, 0, 0, 0);
    };
    // The rows' slots and lengths, of the first ones from shared memory.
    auto row_span = [&](int b) { return b < kKept ? span_of(a, kept[b].x, kept[b].y) : span_of(a, b); };
    if (!a.whole) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the joining blocks may come up meanwhile; they wait for all of this

    Cursor<kStep> at;
    if (a.whole) {
        at.b = blockIdx.x / units;
        at.span = span_of(a, at.b);
        at.steps = steps_of<kStep>(at.span);
        at.ht = blockIdx.x - at.b * units;
        at.step = 0;
        at.left = at.steps;
        if (at.steps == 0) {
            if (at.ht == 0 && warp == 0 && at.span.slot >= 0) clear_row(at.b);
            return;
        }
    } else {
        // this block's stretch of all steps and tolls, and the row that holds its first
        for (int b = tid; b < min(a.B, kKept); b += kThreads) {
            const Span s = span_of(a, b);
            kept[b] = make_int2(s.slot, s.hi);
        }
        if (tid == 0) shared_row = -1;
        __syncthreads();
        for (int b = blockIdx.x * W + warp; b < a.B; b += gridDim.x * W) {
            const Span s = row_span(b);
            if (s.slot >= 0 && steps_of<kStep>(s) == 0) clear_row(b);
        }
        if (!begin_stretch<kThreads, kStep>(a, row_span, units, red, &shared_row, &shared_first, at)) return;
    }
    Cursor<kStep> ahead = at;

    // The copies of one step, all lanes taking part; `from`: where its keys lie (found a step ahead). Keys that no token of the row sees, or
    // that have no page, are not read: their places become zeros, since what is there may not be finite.
    const int chunks = a.d / kEl;
    const unsigned char *kp = static_cast<const unsigned char*>(a.k), *vp = static_cast<const unsigned char*>(a.v);
    const unsigned row_bytes = a.d * (int)sizeof(T);
    int ahead_head = ahead.ht / a.tiles;
    auto first_key = [&]() { return ahead.span.base() + ahead.step * kStep + warp * kKeys; };
    // kPaged: of the step's first key; else of key `lane`. In rows of the pools; negative: nowhere.
    auto where = [&]() -> long long {
        const int t = first_key() + (kPaged ? 0 : lane & (kKeys - 1));
        if (t >= ahead.span.hi || (!kPaged && t < ahead.span.lo)) return -1;
        int i = __umulhi(t, a.page_inverse), in = t - i * a.cache.page;  // t / page, give or take one
        if (in < 0) {
            --i;
            in += a.cache.page;
        } else if (in >= a.cache.page) {
            ++i;
            in -= a.cache.page;
        }
        const int p = a.cache.entry(ahead.span.slot, i);
        if (p < 0) return -1;
        return (static_cast<long long>(p) * a.Hkv + ahead_head) * a.cache.page + in;
    };
    long long from = where();
    constexpr int kPer = kKeys * kChunks / 32, kRowsPer = kChunks < 32 ? 32 / kChunks : 1;  // copies per lane, rows that one of them spans
    const int lane_row = kChunks < 32 ? lane / kChunks : 0, lane_chunk = lane % kChunks;
    auto copy = [&](int stage) {
        if (ahead.left > 0) {
            const uint32_t kt = smem_u32(stages + stage * Lay::kStage);
            unsigned there;
            if constexpr (kPaged) {
                const int t = first_key(), hi = min(max(ahead.span.hi - t, 0), kKeys), lo = min(max(ahead.span.lo - t, 0), kKeys);
                there = from < 0 ? 0u : ((1u << hi) - 1u) & ~((1u << lo) - 1u);
            } else {
                there = __ballot_sync(0xffffffffu, from >= 0) & 0xffffu;
            }
            if (lane == 0) seen[warp][stage] = there;
            if (kPaged && kChunks <= 32 && there == 0xffffu && chunks == kChunks) {
                const size_t at = static_cast<size_t>(from + lane_row) * (kChunks * 16) + lane_chunk * 16;
                const unsigned char *ks = kp + at, *vs = vp + at;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const uint32_t to = kt + 16 * place(i * kRowsPer + lane_row, lane_chunk, kChunks);
                    copy16(to, ks + i * kRowsPer * kChunks * 16, true);
                    copy16(to + Lay::kHalf, vs + i * kRowsPer * kChunks * 16, true);
                }
            } else if (there) {
#pragma unroll 4
                for (int i = 0; i < kPer; ++i) {
                    const int n = i * 32 + lane, r = n / kChunks, c = n % kChunks;
                    const long long row = kPaged ? from + r : __shfl_sync(0xffffffffu, from, r);
                    const bool ok = (there >> r & 1) && c < chunks;
                    const size_t at = ok ? static_cast<size_t>(row) * row_bytes + c * 16 : 0;
                    const uint32_t to = kt + 16 * place(r, c, kChunks);
                    copy16(to, kp + at, ok);
                    copy16(to + Lay::kHalf, vp + at, ok);
                }
            }
            if (ahead.next(a, row_span, 1)) ahead_head = ahead.ht / a.tiles;
            if (ahead.left > 0) from = where();
        }
        copies_commit();
    };
#pragma unroll
    for (int s = 0; s < S - 1; ++s) copy(s);

    typename WarpOf<T, D, M>::type acc;
    int stage = 0;
    while (at.left > 0) {
        const int unit_row = at.ht % a.tiles * kRows, head = at.ht / a.tiles;
        const int n_steps = static_cast<int>(at.left < at.steps - at.step ? at.left : at.steps - at.step);
        const int valid = min(kRows, a.N * a.G - unit_row);
        // the unit's queries, zeros for rows that it does not have
        for (int i = tid; i < kRows * kChunks; i += kThreads) {
            const int r = i / kChunks, c = i % kChunks, row = unit_row + r, n = row / a.G;
            const T* src = static_cast<const T*>(a.q) + (static_cast<long long>(at.b) * a.N + n) * a.ld_q +
                           static_cast<long long>(head * a.G + row - n * a.G) * a.d + c * kEl;
            uint4 u = make_uint4(0, 0, 0, 0);
            if (r < valid && c < chunks) u = __ldg(reinterpret_cast<const uint4*>(src));
            *reinterpret_cast<uint4*>(qs + 16 * place(r, c, kChunks)) = u;
        }
        acc.begin(a, at.span, unit_row);
        const int first = unit_row / a.G, last = (unit_row + valid - 1) / a.G;  // its tokens
        const Limits newest = limits_of(a, at.span, last * a.G), oldest = limits_of(a, at.span, first * a.G);
        __syncthreads();
        acc.queries(smem_u32(qs));
        for (int i = 0; i < n_steps; ++i) {
            copies_wait<S - 2>();
            __syncwarp();  // everyone's copies of this stage have landed, and the stage before it has been read
            copy(stage == 0 ? S - 1 : stage - 1);
            const int base = at.span.base() + (at.step + i) * kStep + warp * kKeys;
            const unsigned there = seen[warp][stage];
            if (there && base <= newest.limit && base + kKeys > oldest.low) {  // a key that some row sees
                const unsigned char* k = stages + stage * Lay::kStage;
                // one token a row sees whatever was copied
                const bool all = a.N == 1 || (base >= newest.low && base + kKeys - 1 <= oldest.limit);
                acc.step(a, qs, k, k + Lay::kHalf, base, there, all, unit_row, first, last, at.span, prob);
            }
            stage = stage == S - 1 ? 0 : stage + 1;
        }
        // the warps' results as one
        acc.statistics(sm[warp], sl[warp]);
        __syncthreads();
        if (tid < kRows) {
            float m = kNone, l = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) m = fmaxf(m, sm[w][tid]);
            const float ref = m == kNone ? 0.f : m;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float f = exp2f(sm[w][tid] - ref);
                sf[w][tid] = f;
                l = fmaf(f, sl[w][tid], l);
            }
            top[tid] = m;
            sum[tid] = l;
        }
        __syncthreads();
#pragma unroll 1
        for (int round = 0; round < W; ++round) {
            acc.template add_to<W>(out, sf[warp], round);
            __syncthreads();
        }
        if (n_steps == at.steps) {
            for (int i = tid; i < valid * (a.d / 8); i += kThreads) {
                const int r = i / (a.d / 8), c = i % (a.d / 8) * 8, row = unit_row + r, n = row / a.G;
                const float inv = sum[r] == 0.f ? 0.f : 1.f / sum[r];  // a row that sees nothing is zero
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = out[r * D + c + e] * inv;
                Vec8<T>::store(static_cast<T*>(a.o) + ((static_cast<long long>(at.b) * a.N + n) * a.Hq + head * a.G + row - n * a.G) * a.d + c, x);
            }
        } else {
            // which of the block's two parts: a unit whose first step is the block's own goes on behind it
            float* part = part_of(a, blockIdx.x, at.step == 0 ? 1 : 0, D, kRows);
            for (int i = tid; i < valid * (D / 4); i += kThreads) reinterpret_cast<float4*>(part)[i] = reinterpret_cast<const float4*>(out)[i];
            if (tid < kRows) {
                part[kRows * D + tid] = top[tid];
                part[kRows * D + kRows + tid] = sum[tid];
            }
        }
        at.next(a, row_span, n_steps);
        __syncthreads();  // the block's output, statistics and queries are free again
    }
}

}  // namespace
}  // namespace gdn2

#include "attn_decode_tc.cuh"

namespace gdn2 {
namespace {

// Joins the parts of a unit that several blocks hold: one block per end of a stretch and four query rows, which acts where that end is the first
// inside its unit's steps. It comes up while the parts are still being made, where there is room, and finds its place meanwhile; then it is
// the latency of reading what other SMs wrote that counts, so its warps ask for several parts each at once, and for all statistics behind
// them. Small blocks, since all of them should fit beside each other: with a block per row and the statistics asked for along with each part,
// 16 drafts took 73 us (then 63), 512 tokens of 2 key heads 11.7 (8.9), rows of 20000, 3000 and 7 tokens of 2 key heads 22.2 (19.9); with blocks of 8
// warps 68, 10.4 and 21.3.
constexpr int kJoinRows = 4, kJoinWarps = 4, kMaxBlocks = 512;

template <typename T, int D, int W, int M>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ DecodeArgs a, int blocks) {
    constexpr int kStep = kKeys * W, kRows = kTile * M, kThreads = 32 * kJoinWarps, kVecs = D <= 128 ? 1 : D / 128, kAtOnce = (M == 2 ? 2 : 4) / kVecs;
    __shared__ long long red[kJoinWarps], before;
    __shared__ int shared_row;
    __shared__ float4 factors[kMaxBlocks], sums[kMaxBlocks];  // of a part's four rows
    __shared__ float inverse[kJoinRows];
    __shared__ float4 outs[kJoinWarps][kJoinRows][D / 4];
    const int units = a.Hkv * a.tiles, tid = threadIdx.x, warp = tid / 32, lane = tid & 31, r0 = blockIdx.y * kJoinRows;
    auto row_span = [&](int b) { return span_of(a, b); };
    if (tid == 0) shared_row = -1;
    Dealing<kThreads, kStep> all;
    all.count(a, row_span, units, red);
    const long long per = steps_per_block(all.total, blocks), v = (blockIdx.x + 1) * per;
    all.find(a, row_span, units, v, red, &shared_row, &before);
    int b = -1, ht = 0, c0 = 0, n = 0;
    if (shared_row >= 0) {
        b = shared_row;
        const int steps = steps_of<kStep>(row_span(b));
        ht = static_cast<int>((v - before) / (steps + kToll));
        const long long start = before + static_cast<long long>(ht) * (steps + kToll) + kToll;
        c0 = static_cast<int>(start / per);
        n = static_cast<int>((start + steps - 1) / per) - c0 + 1;
        if (c0 != static_cast<int>(blockIdx.x) || n == 1) b = -1;
    }
    const int tile = ht % a.tiles, head = ht / a.tiles, row0 = tile * kRows + r0, valid = min(kJoinRows, a.N * a.G - row0);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (b < 0 || valid <= 0) return;
    auto part = [&](int i) { return part_of(a, c0 + i, i == 0 ? 1 : 0, D, kRows); };
    const bool lead = D >= 128 || lane < D / 4;
    float4 x[kAtOnce][kJoinRows][kVecs], o[kJoinRows][kVecs] = {};
    auto ask = [&](int first) {
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int i = first + k * kJoinWarps;
#pragma unroll
            for (int r = 0; r < kJoinRows; ++r)
#pragma unroll
                for (int g = 0; g < kVecs; ++g)
                    if (i < n && r < valid && lead) x[k][r][g] = *reinterpret_cast<const float4*>(part(i) + (r0 + r) * D + 128 * g + 4 * lane);
        }
    };
    ask(warp);
    for (int i = tid; i < n; i += kThreads) {
        const float* p = part(i) + kRows * D + r0;
        factors[i] = *reinterpret_cast<const float4*>(p);
        sums[i] = *reinterpret_cast<const float4*>(p + kRows);
    }
    __syncthreads();
    if (warp < kJoinRows) {  // a row each: maxima to factors, sums to their sum
        float *f = reinterpret_cast<float*>(factors) + warp, *s = reinterpret_cast<float*>(sums) + warp;
        float m = kNone, l = 0.f;
        for (int i = lane; i < n; i += 32) m = fmaxf(m, f[kJoinRows * i]);
#pragma unroll
        for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        const float ref = m == kNone ? 0.f : m;
        for (int i = lane; i < n; i += 32) {
            const float e = exp2f(f[kJoinRows * i] - ref);
            f[kJoinRows * i] = e;
            l = fmaf(e, s[kJoinRows * i], l);
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        if (lane == 0) inverse[warp] = l == 0.f ? 0.f : 1.f / l;
    }
    __syncthreads();
    for (int first = warp; first < n; first += kAtOnce * kJoinWarps) {
        if (first != warp) ask(first);
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int i = first + k * kJoinWarps;
            if (i >= n) break;
            const float4 f4 = factors[i];
            const float f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
            for (int r = 0; r < kJoinRows; ++r)
#pragma unroll
                for (int g = 0; g < kVecs; ++g) {
                    o[r][g].x = fmaf(f[r], x[k][r][g].x, o[r][g].x);
                    o[r][g].y = fmaf(f[r], x[k][r][g].y, o[r][g].y);
                    o[r][g].z = fmaf(f[r], x[k][r][g].z, o[r][g].z);
                    o[r][g].w = fmaf(f[r], x[k][r][g].w, o[r][g].w);
                }
        }
    }
#pragma unroll
    for (int r = 0; r < kJoinRows; ++r)
#pragma unroll
        for (int g = 0; g < kVecs; ++g)
            if (lead) outs[warp][r][32 * g + lane] = o[r][g];
    __syncthreads();
    for (int i = tid; i < valid * a.d; i += kThreads) {
        const int r = i / a.d, c = i - r * a.d, t = (row0 + r) / a.G;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) sum += reinterpret_cast<const float*>(outs[w][r])[c];
        static_cast<T*>(a.o)[((static_cast<long long>(b) * a.N + t) * a.Hq + head * a.G + row0 + r - t * a.G) * a.d + c] = from_f32<T>(sum * inverse[r]);
    }
}

// Widths that a kernel is built for, and blocks per SM: some 128 KB of copies in flight on an SM, which its share of the copy rate takes.
int width_of(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }
// Query rows of a unit, in tiles: over bf16 caches two share the copies of K and V where there are two.
int tiles_of(int rows, gdn2_dtype dt) { return dt == GDN2_BF16 && rows > kTile ? 2 : 1; }
int blocks_of(int d, int tiles, gdn2_dtype dt) {
    const int D = width_of(d);
    const int blocks = sm_count() * (dt == GDN2_BF16 ? (D == 64 ? (tiles == 2 ? 2 : 3) : D == 128 && tiles == 1 ? 2 : 1) : D == 64 ? 2 : 1);
    return blocks < kMaxBlocks ? blocks : kMaxBlocks;
}

template <typename T, int D, int W, int M>
cudaError_t launch_join(const DecodeArgs& a, int blocks, cudaStream_t s) {
    if (a.whole || blocks < 2) return cudaSuccess;
    cudaLaunchConfig_t cfg{};
    const int rows = a.N * a.G < kTile * M ? a.N * a.G : kTile * M;
    cfg.gridDim = dim3(blocks - 1, (rows + kJoinRows - 1) / kJoinRows);
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_kernel<T, D, W, M>, a, blocks);
}

template <typename T, int D, int W, int S, int M, bool kPaged>
cudaError_t launch(DecodeArgs& a, int blocks, cudaStream_t s) {
    using Lay = Layout<T, D, W, S, M>;
    static_assert(Lay::kSmem + 6144 <= 232448, "shared memory of a block");
    // the kernel's shared memory, asked for once per device
    static std::atomic<unsigned long long> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const unsigned long long bit = e == cudaSuccess && dev >= 0 && dev < 64 ? 1ULL << dev : 0;
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(decode_kernel<T, D, W, S, M, kPaged>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::kSmem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    const int units = a.B * a.Hkv * a.tiles;  // of all rows
    decode_kernel<T, D, W, S, M, kPaged><<<a.whole ? units : blocks, Lay::kThreads, Lay::kSmem, s>>>(a);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_join<T, D, W, M>(a, blocks, s);
}

bool pool_map(CUtensorMap* m, const void* p, int d, int page, long long planes) {
    const uint64_t dims[3] = {(uint64_t)d, (uint64_t)page, (uint64_t)planes};
    const uint64_t st[2] = {(uint64_t)d * 2, (uint64_t)page * d * 2};
    const uint32_t box[3] = {64, kKeys, 1};
    return make_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p, dims, st, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D>
cudaError_t launch_tc(DecodeArgs& a, int blocks, cudaStream_t s) {
    static_assert(TcLayout<D>::kSmall + sizeof(TcSmall<D>) + 1024 <= 232448, "shared memory of a block");
    const cudaError_t e = cudaFuncSetAttribute(decode_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
    if (e != cudaSuccess) return e;
    g_launched.store(true, std::memory_order_relaxed);
    a.wait_ns = wait_limit_ns();
    CacheMaps maps{};
    const long long planes = static_cast<long long>(a.cache.n_pages) * a.Hkv;
    const bool mapped = a.cache.page % kKeys == 0 && planes > 0 && planes < (1LL << 31) && pool_map(&maps.k, a.k, a.d, a.cache.page, planes) &&
                        pool_map(&maps.v, a.v, a.d, a.cache.page, planes);
    // the whole shared memory: one block per SM, and no operand descriptor reaches past the block's own
    decode_tc_kernel<D><<<a.whole ? a.B * a.Hkv * a.tiles : blocks, kTcThreads, 232448, s>>>(a, maps, mapped);
    const cudaError_t l = cudaGetLastError();
    return l != cudaSuccess ? l : launch_join<__nv_bfloat16, D, kTcKeys / kKeys, kTcRows / kTile>(a, blocks, s);
}

template <typename T, int D, int W, int S, int M>
cudaError_t launch(DecodeArgs& a, int blocks, cudaStream_t s) {
    return a.cache.page % kKeys ? launch<T, D, W, S, M, false>(a, blocks, s) : launch<T, D, W, S, M, true>(a, blocks, s);
}

// A block per unit, and no parts to join, where no row can be long: the start is quicker (no look at the other rows) and there is no second
// launch. With few units their blocks leave SMs idle, the more the longer their rows. In us, whole against in stretches: one row of 77 tokens
// and 4 key heads 6.2 / 7.6, of 500 12.5 / 9.0; 16 rows of 400 and 4 heads 12.4 / 12.4, 64 rows 17.8 / 22.6; 64 rows of 1000 and 2 heads
// 25.3 / 24.0, 256 rows 55 / 62.
bool whole_units(long long units, int max_pages, int page) {
    const long long keys = static_cast<long long>(max_pages) * page;
    return keys <= 256 || (keys <= 1024 && units * 512 >= keys * sm_count());
}

gdn2_status decode_check(int B, int N, int Hq, int Hkv, int d, gdn2_dtype dt) {
    if (!attn_dtype_ok(dt) || B < 0 || N < 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || Hq % Hkv) return GDN2_ERR_INVALID_ARG;
    if (d % 16 || d > 256 || Hq > 4096 || N > 4096 || B > 65535) return GDN2_ERR_UNSUPPORTED;
    const long long tiles = ((long long)N * (Hq / Hkv) + kTile - 1) / kTile;
    if (tiles * Hkv * B >= (1LL << 31) || (long long)N * Hq * d >= (1LL << 31)) return GDN2_ERR_UNSUPPORTED;
    return GDN2_OK;
}

}  // namespace

int attn_decode_read_clear_status(cudaStream_t s) { return read_clear_status(s); }

}  // namespace gdn2

using namespace gdn2;

extern "C" {

size_t gdn2_attn_decode_workspace_size(int B, int N, int Hq, int Hkv, int d, int max_pages, int page, gdn2_dtype dt) {
    if (decode_check(B, N, Hq, Hkv, d, dt) != GDN2_OK || B == 0 || N == 0 || max_pages <= 0 || page <= 0) return 0;
    const int rows = N * (Hq / Hkv), tiles = tiles_of(rows, dt);
    if (whole_units(static_cast<long long>(B) * Hkv * ((rows + kTile * tiles - 1) / (kTile * tiles)), max_pages, page)) return 0;
    return sizeof(float) * 2 * blocks_of(d, tiles, dt) * static_cast<size_t>(part_floats(width_of(d), kTile * tiles));
}

gdn2_status gdn2_attn_decode(const void* q, long long ld_q, const void* k_pages, const void* v_pages, const int32_t* table,
                             const int32_t* lengths, const int32_t* slots, int n_slots, int n_pages, int max_pages, int page, void* o, int B,
                             int N, int Hq, int Hkv, int d, float scale, int window, gdn2_dtype dt, void* workspace, size_t ws_bytes,
                             void* stream) {
    gdn2_status st = decode_check(B, N, Hq, Hkv, d, dt);
    if (st != GDN2_OK) return st;
    if (window < 0) return GDN2_ERR_INVALID_ARG;
    if ((st = cache_check(table, lengths, slots, n_slots, n_pages, max_pages, page)) != GDN2_OK) return st;
    if (B == 0 || N == 0) return GDN2_OK;
    const long long width = (long long)Hq * d;
    if (!q || !o || ld_q < width || (n_pages && (!k_pages || !v_pages))) return GDN2_ERR_INVALID_ARG;
    if (ld_q >= (1LL << 31)) return GDN2_ERR_UNSUPPORTED;
    if (!aligned16(q) || ld_q % 8 || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(o)) return GDN2_ERR_MISALIGNED;
    const size_t need = gdn2_attn_decode_workspace_size(B, N, Hq, Hkv, d, max_pages, page, dt);
    if (need && (!workspace || ws_bytes < need)) return GDN2_ERR_WORKSPACE;
    if (need && !aligned16(workspace)) return GDN2_ERR_MISALIGNED;
    DecodeArgs a{};
    a.q = q; a.o = o; a.ld_q = ld_q;
    a.k = n_pages ? k_pages : q;  // never read: an address for copies of nothing
    a.v = n_pages ? v_pages : q;
    a.parts = static_cast<float*>(workspace);
    a.cache = Cache{table, lengths, slots, n_slots, n_pages, max_pages, page};
    a.B = B; a.N = N; a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv; a.d = d;
    const int tiles = tiles_of(N * a.G, dt);
    a.tiles = (N * a.G + kTile * tiles - 1) / (kTile * tiles);
    a.whole = whole_units(static_cast<long long>(B) * Hkv * a.tiles, max_pages, page);
    a.window = static_cast<long long>(window) >= static_cast<long long>(max_pages) * page ? 0 : window;
    a.page_inverse = page == 1 ? 0xffffffffu : static_cast<unsigned>(((1ULL << 32) + page - 1) / page);
    a.scale = scale * 1.44269504f;
    const int blocks = blocks_of(d, tiles, dt), D = width_of(d);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    using BF = __nv_bfloat16;
    cudaError_t e;
    if (dt == GDN2_F32)
        e = D == 64 ? launch<float, 64, 4, 3, 1>(a, blocks, s) : D == 128 ? launch<float, 128, 4, 3, 1>(a, blocks, s) : launch<float, 256, 2, 2, 1>(a, blocks, s);
    else if (tiles == 2)
        e = D == 64 ? launch<BF, 64, 4, 5, 2>(a, blocks, s) : D == 128 ? launch_tc<128>(a, blocks, s) : launch_tc<256>(a, blocks, s);
    else
        e = D == 64 ? launch<BF, 64, 4, 4, 1>(a, blocks, s) : D == 128 ? launch<BF, 128, 4, 3, 1>(a, blocks, s) : launch<BF, 256, 4, 3, 1>(a, blocks, s);
    return e == cudaSuccess ? GDN2_OK : GDN2_ERR_CUDA;
}

}  // extern "C"
