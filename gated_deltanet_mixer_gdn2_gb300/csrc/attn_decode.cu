// attn_decode.cu -- attention of a row's newest tokens over its pages of keys and values (attn_common.cuh):
//     o = softmax(scale q K^T over the visible tokens) V,   token n of N sees the tokens up to length - N + n (and within the window)
//
// Every key and value is read once for 4 N H_q / H_kv operations per element: bound by memory. A unit is the cache of one key head of one
// row against up to 16 of its query rows (N tokens times the heads of the group, the matrix instruction's height); its keys are cut into
// steps of 16 per warp. All units' steps, one after another, are dealt out to the blocks in equal stretches, found from the lengths on the
// device: a long row is split over many blocks and short rows share one, whatever the batch. Each warp streams its own keys through its own
// stages of shared memory, by asynchronous copies that run ahead across units, and keeps its own running maximum, sum and output: no block
// barrier but at a unit's end, where the warps' results are joined. A unit that lies in one block leaves as the result; of one that does
// not, each block leaves its part in the workspace, and a second launch joins the parts in their order (no atomics).
#include "attn_common.cuh"

namespace gdn2 {
namespace {

constexpr int kRows = 16;   // query rows of a unit
constexpr int kKeys = 16;   // keys of a warp's step
constexpr float kNone = -INFINITY;

struct DecodeArgs {
    const void *q, *k, *v;
    void* o;
    float* parts;
    long long ld_q;
    Cache cache;
    int B, N, Hq, Hkv, G, d, tiles, window, min_steps;
    float scale;  // times log2 e
};

// What a row asks for: the keys [lo, hi) that its earliest and latest tokens see between them.
struct Span {
    int slot, lo, hi;
};
__device__ __forceinline__ Span span_of(const DecodeArgs& a, int b) {
    Span s{a.cache.row_of(b), 0, 0};
    if (s.slot < 0) return s;
    s.hi = a.cache.length_of(s.slot);
    if (a.window) s.lo = max(s.hi - a.N - a.window + 1, 0);
    return s;
}

template <int kStep>
__device__ __forceinline__ int steps_of(const Span& s) {
    return (s.hi - s.lo + kStep - 1) / kStep;
}

template <int kThreads>
__device__ __forceinline__ long long block_sum(long long v, long long* red) {
#pragma unroll
    for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    long long t = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) t += red[w];
    return t;
}

// Steps of a block: enough that all blocks together cover them, at least min_steps.
__device__ __forceinline__ long long steps_per_block(const DecodeArgs& a, long long total, int blocks) {
    const long long per = (total + blocks - 1) / blocks;
    return per > a.min_steps ? per : a.min_steps;
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

template <typename T, int D, int W, int S>
struct Layout {
    static constexpr int kThreads = 32 * W, kStep = kKeys * W;
    static constexpr int kChunks = D * (int)sizeof(T) / 16;               // 16-byte chunks of a key
    static constexpr int kTile = kKeys * kChunks * 16, kStage = 2 * kTile;  // K and V
    static constexpr int kQ = kRows * kChunks * 16, kOut = kRows * D * 4;
    static constexpr int kProb = sizeof(T) == 4 ? W * (kKeys * kRows + kRows) * 4 : 0;  // fp32: a step's weights and factors, per warp
    static constexpr int kSmem = W * S * kStage + kQ + kOut + kProb;
};

// Where a block's walk over the steps stands.
template <int kStep>
struct Cursor {
    int b, ht, step, steps;  // row; key head and tile of query rows; step of the unit and its steps
    Span span;
    // To row b or the first after it that has steps; b = B at the end.
    __device__ __forceinline__ void settle(const DecodeArgs& a) {
        for (; b < a.B; ++b) {
            span = span_of(a, b);
            steps = steps_of<kStep>(span);
            if (steps > 0) return;
        }
        span = Span{-1, 0, 0};
        steps = 0;
    }
    __device__ __forceinline__ void next(const DecodeArgs& a, int by) {
        step += by;
        if (step < steps) return;
        step = 0;
        if (++ht < a.Hkv * a.tiles) return;
        ht = 0;
        ++b;
        settle(a);
    }
};

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
// enter the second product as two bf16 parts (2^-17), so that the result's only rounding is its own; the sum takes them in fp32.
template <int D>
struct WarpBf16 {
    float o[D / 8][4], m[2], l[2];
    Limits lim[2];
    int row0, row1;  // of the unit

    __device__ __forceinline__ void begin(const DecodeArgs& a, const Span& s, int tile) {
        const int g = (threadIdx.x & 31) / 4;
        row0 = tile * kRows + g;
        row1 = row0 + 8;
        lim[0] = limits_of(a, s, row0);
        lim[1] = limits_of(a, s, row1);
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
        m[0] = m[1] = kNone;
        l[0] = l[1] = 0.f;
    }

    // o += weights V. kMasked: with V's keys under masks (zeros where hidden), and for the rows r0 and r1 (of this lane) alone.
    template <bool kMasked>
    __device__ __forceinline__ void add_values(uint32_t vt, const uint32_t (&hi)[4], const uint32_t (&lo)[4], uint32_t m0 = 0, uint32_t m1 = 0,
                                               bool r0 = true, bool r1 = true) {
        const int lane = threadIdx.x & 31;
        constexpr int kChunks = D / 8;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            uint32_t r[4];
            ldm4t(r, vt + 16 * place((lane & 7) + ((lane >> 3) & 1) * 8, 2 * i + (lane >> 4), kChunks));
            if constexpr (kMasked) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float (&c)[4] = o[2 * i + h];
                    float t[4] = {c[0], c[1], c[2], c[3]};
                    mma(t, hi, r[2 * h] & m0, r[2 * h + 1] & m1);
                    mma(t, lo, r[2 * h] & m0, r[2 * h + 1] & m1);
                    c[0] = r0 ? t[0] : c[0];
                    c[1] = r0 ? t[1] : c[1];
                    c[2] = r1 ? t[2] : c[2];
                    c[3] = r1 ? t[3] : c[3];
                }
                continue;
            }
            mma(o[2 * i], hi, r[0], r[1]);
            mma(o[2 * i + 1], hi, r[2], r[3]);
            mma(o[2 * i], lo, r[0], r[1]);
            mma(o[2 * i + 1], lo, r[2], r[3]);
        }
    }

    // Keys base .. base + 15 of the row, those that `there` has a bit for (the others' places hold zeros); all: every row sees them. Rows that
    // the unit does not have see what they like: their queries are zeros, and nobody reads them.
    __device__ __forceinline__ void step(const DecodeArgs& a, uint32_t qt, uint32_t kt, uint32_t vt, int base, unsigned there, bool all, int first,
                                         int last, const Span& span, float*) {
        const int lane = threadIdx.x & 31, t = lane & 3;
        constexpr int kChunks = D / 8;
        float s[2][4] = {};
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            uint32_t qa[4], kb[4];
            ldm4(qa, qt + 16 * place((lane & 7) + ((lane >> 3) & 1) * 8, 2 * i + (lane >> 4), kChunks));
            ldm4(kb, kt + 16 * place((lane & 7) + (lane >> 4) * 8, 2 * i + ((lane >> 3) & 1), kChunks));
            mma(s[0], qa, kb[0], kb[1]);
            mma(s[1], qa, kb[2], kb[3]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] *= a.scale;
                if (!all || there != 0xffffu) {
                    const int key = 8 * i + 2 * t + (j & 1), at = base + key;
                    const Limits& x = lim[j >> 1];
                    if (!(there >> key & 1) || at < x.low || at > x.limit) s[i][j] = kNone;
                }
            }
        float f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float x = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
            const float now = fmaxf(m[h], x), ref = now == kNone ? 0.f : now;  // no key yet: every weight is 2^-inf = 0
            f[h] = ex2_approx(m[h] - ref);
            m[h] = now;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float p = ex2_approx(s[i][2 * h + j] - ref);
                    s[i][2 * h + j] = p;
                    sum += p;
                }
            l[h] = fmaf(l[h], f[h], sum);
        }
        if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                o[i][0] *= f[0]; o[i][1] *= f[0]; o[i][2] *= f[1]; o[i][3] *= f[1];
            }
        }
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // (row, keys 0-7), (row + 8, keys 0-7), then keys 8-15
            const float x = s[i >> 1][2 * (i & 1)], y = s[i >> 1][2 * (i & 1) + 1];
            hi[i] = pack2(x, y);
            lo[i] = pack2(x - __uint_as_float(hi[i] << 16), y - __uint_as_float(hi[i] & 0xffff0000u));
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
            add_values<true>(vt, hi, lo, m0, m1, row0 / a.G == n, row1 / a.G == n);
        }
    }

    // Maximum and sum of each row, from the lanes that hold them.
    __device__ __forceinline__ void statistics(float* ms, float* ls) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            if ((lane & 3) == 0) {
                ms[lane / 4 + 8 * h] = m[h];
                ls[lane / 4 + 8 * h] = l[h];
            }
        }
    }

    // Adds this warp's output, each row times its factor, to the block's.
    __device__ __forceinline__ void add_to(float* out, const float* factor, bool fresh) {
        const int lane = threadIdx.x & 31, g = lane / 4, t = lane & 3;
        const float f0 = factor[g], f1 = factor[g + 8];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            float2* p0 = reinterpret_cast<float2*>(out + g * D + 8 * i + 2 * t);
            float2* p1 = reinterpret_cast<float2*>(out + (g + 8) * D + 8 * i + 2 * t);
            float2 v0 = fresh ? make_float2(0.f, 0.f) : *p0, v1 = fresh ? make_float2(0.f, 0.f) : *p1;
            v0.x = fmaf(f0, o[i][0], v0.x); v0.y = fmaf(f0, o[i][1], v0.y);
            v1.x = fmaf(f1, o[i][2], v1.x); v1.y = fmaf(f1, o[i][3], v1.y);
            *p0 = v0;
            *p1 = v1;
        }
    }
};

// fp32: on CUDA cores. Scores: a lane takes one of the 16 keys and every other query row; values: a lane takes D / 32 columns.
template <int D>
struct WarpF32 {
    static constexpr int kCols = D / 32, kHalf = kRows / 2;
    float o[kRows][kCols], m[kHalf], l[kHalf];
    Limits lim[kHalf];
    int tile_row, rows;

    __device__ __forceinline__ void begin(const DecodeArgs& a, const Span& s, int tile) {
        const int half = (threadIdx.x & 31) / 16;
        tile_row = tile * kRows;
        rows = min(kRows, a.N * a.G - tile_row);
#pragma unroll
        for (int i = 0; i < kHalf; ++i) {
            lim[i] = limits_of(a, s, tile_row + 2 * i + half);
            m[i] = kNone;
            l[i] = 0.f;
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int c = 0; c < kCols; ++c) o[r][c] = 0.f;
    }

    __device__ __forceinline__ void step(const DecodeArgs& a, uint32_t qt, uint32_t kt, uint32_t vt, int base, unsigned there, bool all, int first,
                                         int last, const Span& span, float* prob) {
        const int lane = threadIdx.x & 31, key = lane & 15, half = lane / 16;
        constexpr int kChunks = D / 4;
        float s[kHalf];
#pragma unroll
        for (int i = 0; i < kHalf; ++i) s[i] = 0.f;
        for (int c = 0; c < kChunks; ++c) {
            float k[4], q[4];
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(k[0]), "=f"(k[1]), "=f"(k[2]), "=f"(k[3]) : "r"(kt + 16 * place(key, c, kChunks)) : "memory");
#pragma unroll
            for (int i = 0; i < kHalf; ++i) {
                if (2 * i >= rows) continue;
                asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(q[0]), "=f"(q[1]), "=f"(q[2]), "=f"(q[3]) : "r"(qt + 16 * place(2 * i + half, c, kChunks)) : "memory");
#pragma unroll
                for (int e = 0; e < 4; ++e) s[i] = fmaf(q[e], k[e], s[i]);
            }
        }
        float* factor = prob + kKeys * kRows;
#pragma unroll
        for (int i = 0; i < kHalf; ++i) {
            if (2 * i >= rows) continue;
            const int at = base + key;
            s[i] = (there >> key & 1) && at >= lim[i].low && at <= lim[i].limit ? s[i] * a.scale : kNone;
            float x = s[i];
#pragma unroll
            for (int d = 8; d; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
            const float now = fmaxf(m[i], x), ref = now == kNone ? 0.f : now;
            const float f = exp2f(m[i] - ref), p = exp2f(s[i] - ref);
            m[i] = now;
            l[i] = fmaf(l[i], f, p);  // this lane's keys
            prob[key * kRows + 2 * i + half] = p;
            if (key == 0) factor[2 * i + half] = f;
        }
        __syncwarp();
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (r >= rows) continue;
            const float f = factor[r];
#pragma unroll
            for (int c = 0; c < kCols; ++c) o[r][c] *= f;
        }
        for (int j = 0; j < kKeys; ++j) {
            float v[kCols];
#pragma unroll
            for (int c = 0; c < kCols; c += 2) {
                const int col = kCols * lane + c;
                asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v[c]), "=f"(v[c + 1]) : "r"(vt + 16 * place(j, col / 4, kChunks) + 4 * (col & 3)) : "memory");
            }
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (r >= rows) continue;
                if (!all) {  // a value that is not finite is kept out of the rows that do not see its key
                    const Limits x = limits_of(a, span, tile_row + r);
                    if (base + j < x.low || base + j > x.limit) continue;
                }
                const float p = prob[j * kRows + r];
#pragma unroll
                for (int c = 0; c < kCols; ++c) o[r][c] = fmaf(p, v[c], o[r][c]);
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

    __device__ __forceinline__ void add_to(float* out, const float* factor, bool fresh) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
                float* p = out + r * D + kCols * lane + c;
                *p = fmaf(factor[r], o[r][c], fresh ? 0.f : *p);
            }
    }
};

template <typename T, int D>
struct WarpOf;
template <int D>
struct WarpOf<__nv_bfloat16, D> {
    using type = WarpBf16<D>;
};
template <int D>
struct WarpOf<float, D> {
    using type = WarpF32<D>;
};

// A block's part of a unit that it does not hold whole: the output of its rows, their maxima and sums. Two per block: of the unit that began
// before its stretch, and of the one that goes on behind it.
__device__ __forceinline__ float* part_of(const DecodeArgs& a, long long block, int which, int D) {
    return a.parts + (block * 2 + which) * (static_cast<long long>(kRows) * D + 2 * kRows);
}

template <typename T, int D, int W, int S>
__global__ void __launch_bounds__(32 * W) decode_kernel(const __grid_constant__ DecodeArgs a) {
    using Lay = Layout<T, D, W, S>;
    constexpr int kThreads = Lay::kThreads, kStep = Lay::kStep, kChunks = Lay::kChunks, kEl = 16 / (int)sizeof(T);
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ long long red[W], shared_first;
    __shared__ int shared_row;
    __shared__ unsigned seen[W][S];  // which of a stage's keys were copied
    __shared__ float sm[W][kRows], sl[W][kRows], sf[W][kRows], top[kRows], sum[kRows];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    const int units = a.Hkv * a.tiles;
    unsigned char* stages = smem + warp * S * Lay::kStage;
    unsigned char* qs = smem + W * S * Lay::kStage;
    float* out = reinterpret_cast<float*>(qs + Lay::kQ);
    float* prob = out + kRows * D + warp * (kKeys * kRows + kRows);

    // rows without a visible key
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        const Span s = span_of(a, b);
        if (s.slot < 0 || steps_of<kStep>(s) > 0) continue;
        T* o = static_cast<T*>(a.o) + static_cast<long long>(b) * a.N * a.Hq * a.d;
        for (int i = tid; i < a.N * a.Hq * a.d; i += kThreads) o[i] = from_f32<T>(0.f);
    }

    // this block's stretch of steps
    long long mine = 0;
    for (int b = tid; b < a.B; b += kThreads) mine += steps_of<kStep>(span_of(a, b));
    const long long total = block_sum<kThreads>(mine, red) * units;
    const long long per = steps_per_block(a, total, gridDim.x);
    const long long begin = blockIdx.x * per, end = begin + per < total ? begin + per : total;
    if (begin >= end) return;

    // its first row: the last whose steps before it are no more than `begin`, among those that have any
    long long before = 0;
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        const int b = b0 + tid;
        const long long n = b < a.B ? static_cast<long long>(steps_of<kStep>(span_of(a, b))) * units : 0;
        long long incl = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += v;
        }
        __syncthreads();
        if (lane == 31) red[warp] = incl;
        if (tid == 0) shared_row = -1;
        __syncthreads();
        long long base = before;
        for (int w = 0; w < W; ++w) {
            if (w < warp) base += red[w];
            before += red[w];
        }
        if (n && begin >= base + incl - n && begin < base + incl) {
            shared_row = b;
            shared_first = base + incl - n;
        }
        __syncthreads();
        if (shared_row >= 0) break;
    }
    if (shared_row < 0) return;  // not with lengths that stay as they are: `begin` lies before `total`
    Cursor<kStep> at;
    at.b = shared_row;
    at.settle(a);
    {
        const long long in = begin - shared_first;
        at.ht = static_cast<int>(in / at.steps);
        at.step = static_cast<int>(in - static_cast<long long>(at.ht) * at.steps);
    }
    Cursor<kStep> ahead = at;
    long long left = end - begin, unread = left;

    // The copies of one step: lane i < 16 finds where key i lies, all lanes copy. Keys that no token of the row sees, or that have no
    // page, are zeros.
    const int chunks = a.d / kEl;
    const T *kp = static_cast<const T*>(a.k), *vp = static_cast<const T*>(a.v);
    auto where = [&]() -> long long {
        const int t = ahead.span.lo + ahead.step * kStep + warp * kKeys + (lane & 15);
        if (t >= ahead.span.hi) return -1;
        const int i = t / a.cache.page, p = a.cache.entry(ahead.span.slot, i);
        if (p < 0) return -1;
        return ((static_cast<long long>(p) * a.Hkv + ahead.ht / a.tiles) * a.cache.page + (t - i * a.cache.page)) * a.d;
    };
    long long from = where();
    auto copy = [&](int stage) {
        if (unread > 0) {
            const uint32_t kt = smem_u32(stages + stage * Lay::kStage), vt = kt + Lay::kTile;
            const unsigned there = __ballot_sync(0xffffffffu, from >= 0) & 0xffffu;
            if (lane == 0) seen[warp][stage] = there;
            constexpr int kPer = kKeys * kChunks / 32;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int n = i * 32 + lane, r = n / kChunks, c = n % kChunks;
                const long long src = __shfl_sync(0xffffffffu, from, r);
                const bool ok = src >= 0 && c < chunks;
                const long long e = ok ? src + c * kEl : 0;
                copy16(kt + 16 * place(r, c, kChunks), kp + e, ok);
                copy16(vt + 16 * place(r, c, kChunks), vp + e, ok);
            }
            if (--unread > 0) {
                ahead.next(a, 1);
                from = where();
            }
        }
        copies_commit();
    };
#pragma unroll
    for (int s = 0; s < S - 1; ++s) copy(s);

    typename WarpOf<T, D>::type acc;
    int stage = 0;
    const uint32_t qt = smem_u32(qs);
    while (left > 0) {
        const int tile = at.ht % a.tiles, head = at.ht / a.tiles, n_steps = static_cast<int>(left < at.steps - at.step ? left : at.steps - at.step);
        if (n_steps <= 0) return;
        const int valid = min(kRows, a.N * a.G - tile * kRows);
        // the unit's queries, zeros for rows that it does not have
        for (int i = tid; i < kRows * kChunks; i += kThreads) {
            const int r = i / kChunks, c = i % kChunks, row = tile * kRows + r, n = row / a.G;
            const T* src = static_cast<const T*>(a.q) + (static_cast<long long>(at.b) * a.N + n) * a.ld_q +
                           static_cast<long long>(head * a.G + row - n * a.G) * a.d + c * kEl;
            uint4 u = make_uint4(0, 0, 0, 0);
            if (r < valid && c < chunks) u = __ldg(reinterpret_cast<const uint4*>(src));
            *reinterpret_cast<uint4*>(qs + 16 * place(r, c, kChunks)) = u;
        }
        acc.begin(a, at.span, tile);
        const int first = tile * kRows / a.G, last = (tile * kRows + valid - 1) / a.G;  // its tokens
        const int all_low = limits_of(a, at.span, last * a.G).low, all_limit = limits_of(a, at.span, first * a.G).limit;
        __syncthreads();
        for (int i = 0; i < n_steps; ++i) {
            copies_wait<S - 2>();
            __syncwarp();  // everyone's copies of this stage have landed, and the stage before it has been read
            copy(stage == 0 ? S - 1 : stage - 1);
            const int base = at.span.lo + (at.step + i) * kStep + warp * kKeys;
            const unsigned there = seen[warp][stage];
            if (there) {
                const uint32_t kt = smem_u32(stages + stage * Lay::kStage);
                // one token a row sees whatever was copied
                const bool all = a.N == 1 || (base >= all_low && base + kKeys - 1 <= all_limit);
                acc.step(a, qt, kt, kt + Lay::kTile, base, there, all, first, last, at.span, prob);
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
        for (int w = 0; w < W; ++w) {
            if (w == warp) acc.add_to(out, sf[w], w == 0);
            __syncthreads();
        }
        const bool whole = n_steps == at.steps;
        if (whole) {
            for (int i = tid; i < valid * (a.d / 8); i += kThreads) {
                const int r = i / (a.d / 8), c = i % (a.d / 8) * 8, row = tile * kRows + r, n = row / a.G;
                const float inv = sum[r] == 0.f ? 0.f : 1.f / sum[r];  // a row that sees nothing is zero
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = out[r * D + c + e] * inv;
                Vec8<T>::store(static_cast<T*>(a.o) + ((static_cast<long long>(at.b) * a.N + n) * a.Hq + head * a.G + row - n * a.G) * a.d + c, x);
            }
        } else {
            // which of the block's two parts: a unit whose first step is the block's own goes on behind it
            float* part = part_of(a, blockIdx.x, at.step == 0 ? 1 : 0, D);
            for (int i = tid; i < valid * (D / 4); i += kThreads) reinterpret_cast<float4*>(part)[i] = reinterpret_cast<const float4*>(out)[i];
            if (tid < kRows) {
                part[kRows * D + tid] = top[tid];
                part[kRows * D + kRows + tid] = sum[tid];
            }
        }
        left -= n_steps;
        if (left > 0) at.next(a, n_steps);
        __syncthreads();  // the block's output, statistics and queries are free again
    }
}

// Joins the parts of a unit that several blocks hold: one block per unit and four of its rows, a warp per row.
template <typename T, int D, int W>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ DecodeArgs a, int blocks) {
    constexpr int kStep = kKeys * W;
    __shared__ long long red[4];
    const int units = a.Hkv * a.tiles, b = blockIdx.x / units, ht = blockIdx.x % units, tile = ht % a.tiles, head = ht / a.tiles;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, r = blockIdx.y * 4 + warp, row = tile * kRows + r;
    const Span s = span_of(a, b);
    const int steps = steps_of<kStep>(s);
    if (steps <= 1) return;
    long long lead = 0, all = 0;
    for (int i = threadIdx.x; i < a.B; i += 128) {
        const long long n = steps_of<kStep>(span_of(a, i));
        all += n;
        if (i < b) lead += n;
    }
    lead = block_sum<128>(lead, red);
    all = block_sum<128>(all, red);
    const long long per = steps_per_block(a, all * units, blocks), start = lead * units + static_cast<long long>(ht) * steps;
    const int c0 = static_cast<int>(start / per), c1 = static_cast<int>((start + steps - 1) / per);
    if (c0 == c1 || row >= a.N * a.G) return;
    auto part = [&](int c) { return part_of(a, c, c == c0 ? 1 : 0, D); };
    float m = kNone;
    for (int c = c0 + lane; c <= c1; c += 32) m = fmaxf(m, part(c)[kRows * D + r]);
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float ref = m == kNone ? 0.f : m;
    constexpr int kCols = D / 32;
    float l = 0.f, x[kCols] = {};
#pragma unroll 4
    for (int c = c0; c <= c1; ++c) {
        const float* p = part(c);
        const float f = exp2f(p[kRows * D + r] - ref);
        l = fmaf(f, p[kRows * D + kRows + r], l);
#pragma unroll
        for (int i = 0; i < kCols; i += 2) {
            const float2 v = *reinterpret_cast<const float2*>(p + r * D + kCols * lane + i);
            x[i] = fmaf(f, v.x, x[i]);
            x[i + 1] = fmaf(f, v.y, x[i + 1]);
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int n = row / a.G;
    T* o = static_cast<T*>(a.o) + ((static_cast<long long>(b) * a.N + n) * a.Hq + head * a.G + row - n * a.G) * a.d;
#pragma unroll
    for (int i = 0; i < kCols; ++i)
        if (kCols * lane + i < a.d) o[kCols * lane + i] = from_f32<T>(x[i] * inv);
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 152;
    return n > 0 ? n : 152;
}

// Warps and stages per block and blocks per SM: some 128 KB of copies in flight on an SM, which its share of the copy rate takes.
int width_of(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }
int blocks_of(int d, gdn2_dtype dt) {
    const int D = width_of(d);
    return sm_count() * (dt == GDN2_BF16 ? (D == 64 ? 3 : D == 128 ? 2 : 1) : D == 64 ? 2 : 1);
}

template <typename T, int D, int W, int S>
cudaError_t launch(DecodeArgs& a, int blocks, cudaStream_t s) {
    using Lay = Layout<T, D, W, S>;
    static_assert(Lay::kSmem + 4096 <= 232448, "shared memory of a block");
    cudaError_t e = cudaFuncSetAttribute(decode_kernel<T, D, W, S>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::kSmem);
    if (e != cudaSuccess) return e;
    decode_kernel<T, D, W, S><<<blocks, Lay::kThreads, Lay::kSmem, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    // a row of a single step lies in one block
    if (static_cast<long long>(a.cache.max_pages) * a.cache.page <= Lay::kStep) return e;
    const int rows = a.N * a.G < kRows ? a.N * a.G : kRows;
    join_kernel<T, D, W><<<dim3(a.B * a.Hkv * a.tiles, (rows + 3) / 4), 128, 0, s>>>(a, blocks);
    return cudaGetLastError();
}

gdn2_status decode_check(int B, int N, int Hq, int Hkv, int d, gdn2_dtype dt) {
    if (!attn_dtype_ok(dt) || B < 0 || N < 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || Hq % Hkv) return GDN2_ERR_INVALID_ARG;
    if (d % 16 || d > 256 || Hq > 4096 || N > 4096 || B > 65535) return GDN2_ERR_UNSUPPORTED;
    const long long tiles = ((long long)N * (Hq / Hkv) + kRows - 1) / kRows;
    if (tiles * Hkv * B >= (1LL << 31) || (long long)N * Hq * d >= (1LL << 31)) return GDN2_ERR_UNSUPPORTED;
    return GDN2_OK;
}

}  // namespace
}  // namespace gdn2

using namespace gdn2;

extern "C" {

size_t gdn2_attn_decode_workspace_size(int B, int N, int Hq, int Hkv, int d, gdn2_dtype dt) {
    if (decode_check(B, N, Hq, Hkv, d, dt) != GDN2_OK || B == 0 || N == 0) return 0;
    return sizeof(float) * 2 * blocks_of(d, dt) * (static_cast<size_t>(kRows) * width_of(d) + 2 * kRows);
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
    if (!workspace || ws_bytes < gdn2_attn_decode_workspace_size(B, N, Hq, Hkv, d, dt)) return GDN2_ERR_WORKSPACE;
    if (!aligned16(workspace)) return GDN2_ERR_MISALIGNED;
    DecodeArgs a{};
    a.q = q; a.o = o; a.ld_q = ld_q;
    a.k = n_pages ? k_pages : q;  // never read: an address for copies of nothing
    a.v = n_pages ? v_pages : q;
    a.parts = static_cast<float*>(workspace);
    a.cache = Cache{table, lengths, slots, n_slots, n_pages, max_pages, page};
    a.B = B; a.N = N; a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv; a.d = d;
    a.tiles = (N * a.G + kRows - 1) / kRows;
    a.window = static_cast<long long>(window) >= static_cast<long long>(max_pages) * page ? 0 : window;
    a.min_steps = 2;
    a.scale = scale * 1.44269504f;
    const int blocks = blocks_of(d, dt), D = width_of(d);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    using BF = __nv_bfloat16;
    cudaError_t e;
    if (dt == GDN2_BF16)
        e = D == 64 ? launch<BF, 64, 4, 4>(a, blocks, s) : D == 128 ? launch<BF, 128, 4, 3>(a, blocks, s) : launch<BF, 256, 4, 3>(a, blocks, s);
    else
        e = D == 64 ? launch<float, 64, 4, 3>(a, blocks, s) : D == 128 ? launch<float, 128, 4, 3>(a, blocks, s) : launch<float, 256, 2, 2>(a, blocks, s);
    return e == cudaSuccess ? GDN2_OK : GDN2_ERR_CUDA;
}

}  // extern "C"
