// attn_prologue.cu -- what an attention layer does to its queries and keys between projection and attention, in one pass: RMS norm
// over each head and rotation by position; for serving with k and v written to the pages of a cache; and the gradients.
//     n = w x / sqrt(mean(x^2) + eps)        (y_a, y_b) = (n_a cos - n_b sin, n_b cos + n_a sin),  angle = position * inv_freq
// for the pairs (a, b) of the first `rot` elements: (j, j + rot / 2), or (2 j, 2 j + 1) when interleaved.
//
// Bound by memory: every element is read once and written once for some 10 operations, which are packed two by two. A head's row belongs to
// a group of lanes, eight elements each (both sides of four pairs), whose sum of squares comes by shuffles; a group keeps to one token, whose
// cosines and sines it holds in registers, and has several rows' loads in flight. A block has eight tokens, whose angles it forms together.
//
// 16384 tokens of 32 + 8 heads of 128 in bf16: 60 us, 5.6 TB/s (0.83 of the copy rate), the issue slots 59% busy; a third of a wave of blocks is
// what is lost. Two rows in flight 64 us, a group's own stretch of heads without block barriers 66, tokens by fours 66 and by sixteens 61, elements
// side by side with the pairs' other sides by shuffles 82. In fp32 106 us (0.93). Gradients: 98 us (0.76), 155 in fp32 (0.96).
#include "attn_common.cuh"

namespace gdn2 {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 8;    // tokens of a tile at most: the angles of a tile are formed once, two or so per thread
constexpr int kMaxD = 256;
constexpr int kGradBlocks = 2;  // per SM

struct PrologueArgs {
    const void *q, *k, *v;
    long long ld_q, ld_k, ld_v;
    const float *q_weight, *k_weight, *inv_freq;
    const int* positions;
    Seqs seqs;
    Cache cache;  // table == nullptr: no cache
    void *q_out, *k_out, *v_out;  // k_out and v_out are the pools where there is a cache
    // gradients
    const void *gq, *gk;
    long long ld_gq, ld_gk, ld_dq, ld_dk;
    float* parts;
    int Hq, Hkv, d, rot, tokens, tiles;
    float eps, inv_d;
};

// inv_freq as turns per position in 64-bit fixed point, modulo one turn: f / (2 pi) = m 2^(e - 150) / (2 pi) with m the 24 bits of f, and
// kTurns = 2^66 / (2 pi). position * turns, wrapping, is the angle modulo a turn to 2^-64 (1 + |f| / 2 pi) per position: 2^-33 of a turn
// for any 32-bit position and frequencies of about one, where a 32-bit product would lose the angle from some ten thousand positions on.
__device__ __forceinline__ unsigned long long turns_of(float f) {
    constexpr unsigned long long kTurns = 11743562013128004906ull;
    const unsigned bits = __float_as_uint(f);
    const int e = (bits >> 23) & 255;
    const unsigned long long m = e ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
    const unsigned long long lo = m * kTurns, hi = __umul64hi(m, kTurns);
    const int s = 152 - (e ? e : 1);
    const unsigned long long t = s >= 128 ? 0 : s >= 64 ? hi >> (s - 64) : s > 0 ? (hi << (64 - s)) | (lo >> s) : s > -64 ? lo << -s : 0;
    return bits >> 31 ? 0 - t : t;
}

// What the threads of a block share: of each token of the tile its position and where it goes, and the angles.
struct TileShared {
    float cs[kTokens][kMaxD / 2], sn[kTokens][kMaxD / 2];
    int position[kTokens], live[kTokens], page[kTokens], at[kTokens];
    unsigned long long turns[kMaxD / 2];
    float bad[kMaxD / 2];  // 0, or NaN where the frequency is not finite
};

__device__ __forceinline__ void frequencies(const PrologueArgs& a, TileShared& sh) {
    for (int j = threadIdx.x; j < a.rot / 2; j += kThreads) {
        const float f = a.inv_freq[j];
        sh.turns[j] = turns_of(f);
        sh.bad[j] = f - f;
    }
}

// Positions, destinations and angles of the tile's tokens. A barrier before (for turns, and the last tile's readers) and one inside.
__device__ __forceinline__ void enter_tile(const PrologueArgs& a, TileShared& sh, long long row0, long long rows) {
    const int t = threadIdx.x;
    if (t < a.tokens) {
        const long long r = row0 + t;
        int seq = 0, start = 0, end = 0;
        bool live = r < rows && find_row(a.seqs, static_cast<int>(r), seq, start, end);
        int at = static_cast<int>(r) - start, page = -1;
        if (a.cache.table && live) {
            const int slot = a.cache.row_of(seq);
            live = slot >= 0;
            if (live) {
                at += a.cache.length_of(slot) - (end - start);  // its place in the row; negative where the lengths do not count it
                if (at >= 0) page = a.cache.entry(slot, at / a.cache.page);
            }
        }
        sh.live[t] = live;
        sh.position[t] = a.positions && live ? a.positions[r] : at;
        sh.page[t] = page;
        sh.at[t] = at >= 0 && a.cache.table ? at % a.cache.page : 0;
    }
    __syncthreads();
    const int half = a.rot / 2;
    for (int i = t; i < a.tokens * half; i += kThreads) {
        const int k = i / half, j = i - k * half;
        const unsigned long long turn = static_cast<unsigned long long>(static_cast<long long>(sh.position[k])) * sh.turns[j];
        float s, c;
        sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f, &s, &c);
        sh.cs[k][j] = c + sh.bad[j];
        sh.sn[k][j] = s + sh.bad[j];
    }
    __syncthreads();
}

// A lane's eight elements of a head: two runs of four, at e0 and e1. Rotated by halves they are both sides of four pairs, so a rotation needs
// no other lane; else they lie side by side.
struct Place {
    int e0, e1;
    bool mine, turned;  // within the head; rotated
};
template <bool kPairs>
__device__ __forceinline__ Place place_of(int lane, int d, int rot) {
    Place p{8 * lane, 8 * lane + 4, 8 * lane < d, 8 * lane < rot};
    if (!p.mine) {  // reads along, for nothing
        p.e0 = 0;
        p.e1 = 4;
    } else if (!kPairs && p.turned) {
        p.e0 = 4 * lane;
        p.e1 = 4 * lane + rot / 2;
    }
    return p;
}

// Eight elements as they are loaded, and as four packed pairs of fp32.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint2 u[2];
    static constexpr int kFlight = 3, kGradFlight = 3, kBlocks = 4;  // rows on their way, blocks per SM
    __device__ __forceinline__ void load(const __nv_bfloat16* p, const Place& at) {
        u[0] = __ldg(reinterpret_cast<const uint2*>(p + at.e0));
        u[1] = __ldg(reinterpret_cast<const uint2*>(p + at.e1));
    }
    __device__ __forceinline__ void get(uint64_t (&x)[4]) const {
        x[0] = bf16x2_widen(u[0].x); x[1] = bf16x2_widen(u[0].y); x[2] = bf16x2_widen(u[1].x); x[3] = bf16x2_widen(u[1].y);
    }
    __device__ __forceinline__ void set(const uint64_t (&x)[4]) {
        u[0] = make_uint2(bf16x2_narrow(x[0]), bf16x2_narrow(x[1]));
        u[1] = make_uint2(bf16x2_narrow(x[2]), bf16x2_narrow(x[3]));
    }
    __device__ __forceinline__ void store(__nv_bfloat16* p, const Place& at) const {
        *reinterpret_cast<uint2*>(p + at.e0) = u[0];
        *reinterpret_cast<uint2*>(p + at.e1) = u[1];
    }
};
template <>
struct Raw8<float> {
    ulonglong2 u[2];
    static constexpr int kFlight = 2, kGradFlight = 2, kBlocks = 3;
    __device__ __forceinline__ void load(const float* p, const Place& at) {
        u[0] = __ldg(reinterpret_cast<const ulonglong2*>(p + at.e0));
        u[1] = __ldg(reinterpret_cast<const ulonglong2*>(p + at.e1));
    }
    __device__ __forceinline__ void get(uint64_t (&x)[4]) const { x[0] = u[0].x; x[1] = u[0].y; x[2] = u[1].x; x[3] = u[1].y; }
    __device__ __forceinline__ void set(const uint64_t (&x)[4]) {
        u[0] = make_ulonglong2(x[0], x[1]);
        u[1] = make_ulonglong2(x[2], x[3]);
    }
    __device__ __forceinline__ void store(float* p, const Place& at) const {
        *reinterpret_cast<ulonglong2*>(p + at.e0) = u[0];
        *reinterpret_cast<ulonglong2*>(p + at.e1) = u[1];
    }
};

// The lane's weights of a side, ones without.
__device__ __forceinline__ void weights_of(const float* weight, const Place& at, uint64_t (&wv)[4]) {
    if (weight) {
        const float4 p = __ldg(reinterpret_cast<const float4*>(weight + at.e0)), q = __ldg(reinterpret_cast<const float4*>(weight + at.e1));
        wv[0] = f32x2(p.x, p.y); wv[1] = f32x2(p.z, p.w); wv[2] = f32x2(q.x, q.y); wv[3] = f32x2(q.z, q.w);
    } else {
        wv[0] = wv[1] = wv[2] = wv[3] = f32x2(1.f, 1.f);
    }
}

// x . y of the lane's elements
__device__ __forceinline__ float lane_dot(const uint64_t (&x)[4], const uint64_t (&y)[4]) {
    uint64_t s = mul_f32x2(x[0], y[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) s = fma_f32x2(x[i], y[i], s);
    float lo, hi;
    f32x2_split(s, lo, hi);
    return lo + hi;
}
// Sums over the group's lanes, n of them side by side; all lanes of the warp take part.
template <int L, int n>
__device__ __forceinline__ void group_sums(float (&v)[n]) {
#pragma unroll
    for (int m = L / 2; m; m >>= 1)
#pragma unroll
        for (int i = 0; i < n; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], m);
}

// The lane's part of a token's rotation. By halves: x[0], x[1] are the first sides a, x[2], x[3] the second sides b of its pairs.
template <bool kPairs>
struct Turn {
    uint64_t c[kPairs ? 4 : 2], s[kPairs ? 4 : 2];
    __device__ __forceinline__ void set(const TileShared& sh, int token, const Place& at) {
        if (!at.turned) return;
        if constexpr (kPairs) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = at.e0 / 2 + i;
                c[i] = f32x2(sh.cs[token][j], sh.cs[token][j]);
                s[i] = f32x2(-sh.sn[token][j], sh.sn[token][j]);
            }
        } else {
            const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(&sh.cs[token][at.e0]), v = *reinterpret_cast<const ulonglong2*>(&sh.sn[token][at.e0]);
            c[0] = u.x; c[1] = u.y; s[0] = v.x; s[1] = v.y;
        }
    }
    // Rotates x in place; kBack: by the opposite angle.
    template <bool kBack>
    __device__ __forceinline__ void apply(uint64_t (&x)[4], bool turned) const {
        if (!turned) return;
        if constexpr (kPairs) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float lo, hi;
                f32x2_split(x[i], lo, hi);
                x[i] = fma_f32x2(x[i], c[i], mul_f32x2(kBack ? f32x2(-hi, -lo) : f32x2(hi, lo), s[i]));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint64_t a = x[i], b = x[2 + i];
                const uint64_t bs = mul_f32x2(b, s[i]), as = mul_f32x2(a, s[i]);
                x[i] = kBack ? fma_f32x2(a, c[i], bs) : sub_f32x2(mul_f32x2(a, c[i]), bs);
                x[2 + i] = kBack ? sub_f32x2(mul_f32x2(b, c[i]), as) : fma_f32x2(b, c[i], as);
            }
        }
    }
};

// The groups of a block lie `tokens` apart for one token; blockIdx.y shares its heads out further.
template <typename T, int L, bool kPairs>
__global__ void __launch_bounds__(kThreads, Raw8<T>::kBlocks) prologue_kernel(const __grid_constant__ PrologueArgs a) {
    __shared__ __align__(16) TileShared sh;
    const long long rows = a.seqs.offsets ? a.seqs.T : static_cast<long long>(a.seqs.B) * a.seqs.T;
    const long long row0 = static_cast<long long>(blockIdx.x) * a.tokens;
    const int lane = threadIdx.x % L, group = threadIdx.x / L, per = kThreads / L / a.tokens;
    const int token = group % a.tokens, base = blockIdx.y * per, part = base + group / a.tokens, step = per * gridDim.y;
    const Place at = place_of<kPairs>(lane, a.d, a.rot);
    const long long r = row0 + token, r_in = r < rows ? r : rows - 1;
    const int d = a.d;
    constexpr int kFlight = Raw8<T>::kFlight;
    // Heads part, part + step, .. of one side. Rows of no sequence and of inactive slots are loaded before that is known, and dropped.
    const T *qs = static_cast<const T*>(a.q) + r_in * a.ld_q, *ks = static_cast<const T*>(a.k) + r_in * a.ld_k;
    auto fetch = [&](Raw8<T>& to, const T* src, int h, int H) {
        if (h < H) to.load(src + h * d, at);
    };
    Raw8<T> raw[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) fetch(raw[u], qs, part + u * step, a.Hq);  // on their way while the tile's positions and angles are formed
    frequencies(a, sh);
    enter_tile(a, sh, row0, rows);

    const bool live = sh.live[token] && at.mine;
    Turn<kPairs> turn;
    turn.set(sh, token, at);
    const int page = sh.page[token];
    // keys and values: in the cache, heads lie a page apart
    const int kv_step = a.cache.table ? a.cache.page * d : d;
    const long long kv = a.cache.table ? (static_cast<long long>(page) * a.Hkv * a.cache.page + sh.at[token]) * d : r * a.Hkv * d;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const int H = side ? a.Hkv : a.Hq, rounds = (H - base + step - 1) / step, to_step = side ? kv_step : d;
        const T* src = side ? ks : qs;
        T* to = side ? static_cast<T*>(a.k_out) + kv : static_cast<T*>(a.q_out) + r * a.Hq * d;
        const float* weight = side ? a.k_weight : a.q_weight;
        uint64_t wv[4];
        weights_of(weight, at, wv);
        const int last = live && (!side || !a.cache.table || page >= 0) ? H : 0;  // heads behind it are not stored
        if (side) {
#pragma unroll
            for (int u = 0; u < kFlight; ++u) fetch(raw[u], src, part + u * step, H);
        }
        int h = part;
        for (int i = 0; i < rounds; i += kFlight) {
#pragma unroll
            for (int u = 0; u < kFlight; ++u) {
                if (u && i + u >= rounds) break;
                uint64_t x[4];
                raw[u].get(x);
                fetch(raw[u], src, h + kFlight * step, H);
                if (weight) {  // without weights there is no norm
                    float ss[1] = {at.mine ? lane_dot(x, x) : 0.f};
                    group_sums<L>(ss);
                    const float inv = rsqrtf(fmaf(ss[0], a.inv_d, a.eps));
                    const uint64_t inv2 = f32x2(inv, inv);
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = mul_f32x2(x[e], mul_f32x2(wv[e], inv2));
                }
                turn.template apply<false>(x, at.turned);
                if (h < last) {
                    Raw8<T> y;
                    y.set(x);
                    y.store(to + static_cast<long long>(h) * to_step, at);
                }
                h += step;
            }
        }
    }
    if (a.cache.table && live && page >= 0) {  // values pass as they are
        const T* vs = static_cast<const T*>(a.v) + r * a.ld_v;
        T* vo = static_cast<T*>(a.v_out) + kv;
#pragma unroll 4
        for (int g = part; g < a.Hkv; g += step) {
            Raw8<T> v;
            v.load(vs + g * d, at);
            v.store(vo + static_cast<long long>(g) * kv_step, at);
        }
    }
}

// Gradients: dn = dy turned back; dw = sum over tokens and heads of dn xh with xh = x inv; dx = inv (w dn - xh mean(w dn xh)).
// Blocks walk tiles one after another and leave one partial sum of the weights' gradients each.
template <typename T, int L, bool kPairs>
__global__ void __launch_bounds__(kThreads, kGradBlocks) prologue_grad_kernel(const __grid_constant__ PrologueArgs a) {
    __shared__ __align__(16) TileShared sh;
    __shared__ __align__(16) float red[kThreads / L][L * 8];
    const long long rows = a.seqs.offsets ? a.seqs.T : static_cast<long long>(a.seqs.B) * a.seqs.T;
    const int lane = threadIdx.x % L, group = threadIdx.x / L, groups = kThreads / L;
    const int token = group % a.tokens, part = group / a.tokens, step = groups / a.tokens;
    const Place at = place_of<kPairs>(lane, a.d, a.rot);
    // the lane's sums of q's weight, and of k's in its own places of shared memory: registers are wanted for loads
    uint64_t acc[4];
    ulonglong2* const own[2] = {reinterpret_cast<ulonglong2*>(&red[group][at.e0]), reinterpret_cast<ulonglong2*>(&red[group][at.e1])};
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = 0;
    if (at.mine) *own[0] = *own[1] = make_ulonglong2(0, 0);
    frequencies(a, sh);
    constexpr int kFlight = Raw8<T>::kGradFlight;
    Raw8<T> rx[kFlight], rg[kFlight];
    for (int tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
        const long long row0 = static_cast<long long>(tile) * a.tokens;
        const long long r = row0 + token, r_in = r < rows ? r : rows - 1;
        const T *gs = static_cast<const T*>(a.gq) + r_in * a.ld_gq + part * a.d, *xs = static_cast<const T*>(a.q) + r_in * a.ld_q + part * a.d;
        int next = part;
        auto fetch = [&](int u, int H, bool normed) {
            if (next < H) {
                rg[u].load(gs, at);
                if (normed) rx[u].load(xs, at);
            }
            next += step;
            gs += step * a.d;
            xs += step * a.d;
        };
#pragma unroll
        for (int u = 0; u < kFlight; ++u) fetch(u, a.Hq, a.q_weight);
        __syncthreads();
        enter_tile(a, sh, row0, rows);
        const bool live = sh.live[token] && at.mine;
        Turn<kPairs> turn;
        turn.set(sh, token, at);
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            const int H = side ? a.Hkv : a.Hq;
            const float* weight = side ? a.k_weight : a.q_weight;
            T* out = static_cast<T*>(side ? a.k_out : a.q_out) + r * (side ? a.ld_dk : a.ld_dq) + part * a.d;
            uint64_t wv[4];
            weights_of(weight, at, wv);
            if (side) {
                gs = static_cast<const T*>(a.gk) + r_in * a.ld_gk + part * a.d;
                xs = static_cast<const T*>(a.k) + r_in * a.ld_k + part * a.d;
                next = part;
#pragma unroll
                for (int u = 0; u < kFlight; ++u) fetch(u, H, weight);
            }
            const int rounds = (H + step - 1) / step;
            int h = part;
            uint64_t sum[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] = side ? 0 : acc[e];
            for (int i = 0; i < rounds; i += kFlight) {
#pragma unroll
                for (int u = 0; u < kFlight; ++u) {
                    if (u && i + u >= rounds) break;
                    uint64_t g[4], x[4];
                    rg[u].get(g);
                    if (weight) rx[u].get(x);
                    fetch(u, H, weight);
                    turn.template apply<true>(g, at.turned);
                    const bool here = live && h < H;
                    if (weight) {
                        uint64_t gw[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) gw[e] = mul_f32x2(g[e], wv[e]);
                        float sums[2] = {at.mine ? lane_dot(x, x) : 0.f, at.mine ? lane_dot(gw, x) : 0.f};
                        group_sums<L>(sums);
                        const float inv = rsqrtf(fmaf(sums[0], a.inv_d, a.eps)), m = -inv * sums[1] * inv * a.inv_d;
                        const uint64_t inv2 = f32x2(inv, inv), m2 = f32x2(m, m);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint64_t more = fma_f32x2(g[e], mul_f32x2(x[e], inv2), sum[e]);
                            sum[e] = here ? more : sum[e];  // what is not a head of a token may be anything
                            g[e] = mul_f32x2(inv2, fma_f32x2(x[e], m2, gw[e]));
                        }
                    }
                    if (here) {
                        Raw8<T> y;
                        y.set(g);
                        y.store(out, at);
                    }
                    out += step * a.d;
                    h += step;
                }
            }
            if (!side) {
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[e] = sum[e];
            } else if (weight && at.mine) {
                ulonglong2 p = *own[0], q = *own[1];
                *own[0] = make_ulonglong2(add_f32x2(p.x, sum[0]), add_f32x2(p.y, sum[1]));
                *own[1] = make_ulonglong2(add_f32x2(q.x, sum[2]), add_f32x2(q.y, sum[3]));
            }
        }
    }
    if (!a.parts) return;
#pragma unroll
    for (int side = 1; side >= 0; --side) {
        __syncthreads();
        if (!side) {
            if (at.mine) {
                *own[0] = make_ulonglong2(acc[0], acc[1]);
                *own[1] = make_ulonglong2(acc[2], acc[3]);
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < a.d; c += kThreads) {
            float v = 0.f;
#pragma unroll 8
            for (int k = 0; k < groups; ++k) v += red[k][c];
            a.parts[(static_cast<long long>(blockIdx.x) * 2 + side) * a.d + c] = v;
        }
    }
}

// The blocks' partial sums, added in a fixed order: 32 columns a block, its warps each a share of the parts.
__global__ void __launch_bounds__(1024) weight_grad_kernel(const float* parts, int n, int d, float* dq_weight, float* dk_weight) {
    __shared__ float red[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, side = blockIdx.y, c = blockIdx.x * 32 + lane;
    float* out = side ? dk_weight : dq_weight;
    if (!out) return;
    float v = 0.f;
    if (c < d) {
#pragma unroll 8
        for (int k = warp; k < n; k += 32) v += parts[(static_cast<long long>(k) * 2 + side) * d + c];
    }
    red[warp][lane] = v;
    __syncthreads();
    v = red[lane][warp];
#pragma unroll
    for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    if (lane == 0 && blockIdx.x * 32 + warp < d) out[blockIdx.x * 32 + warp] = v;
}

template <typename T, int L>
cudaError_t launch(const PrologueArgs& a, dim3 grid, bool pairs, bool grad, cudaStream_t s) {
    if (grad) {
        if (pairs) prologue_grad_kernel<T, L, true><<<grid, kThreads, 0, s>>>(a);
        else prologue_grad_kernel<T, L, false><<<grid, kThreads, 0, s>>>(a);
    } else {
        if (pairs) prologue_kernel<T, L, true><<<grid, kThreads, 0, s>>>(a);
        else prologue_kernel<T, L, false><<<grid, kThreads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch(const PrologueArgs& a, dim3 grid, bool pairs, bool grad, cudaStream_t s) {
    return a.d <= 64 ? launch<T, 8>(a, grid, pairs, grad, s) : a.d <= 128 ? launch<T, 16>(a, grid, pairs, grad, s) : launch<T, 32>(a, grid, pairs, grad, s);
}

// Lanes of a head's row, and tokens of a tile: eight, but fewer while that leaves fewer blocks than the SMs hold (4 x 152).
int lanes_of(int d) { return d <= 64 ? 8 : d <= 128 ? 16 : 32; }
int tokens_of(int d, long long rows) {
    int t = kTokens;
    while (t > 1 && rows < 608LL * t) t /= 2;
    const int groups = kThreads / lanes_of(d);
    return t < groups ? t : groups;
}

int grad_blocks(int d, long long rows) {
    const int t = tokens_of(d, rows);
    const long long tiles = (rows + t - 1) / t, most = static_cast<long long>(kGradBlocks) * sm_count();
    return static_cast<int>(tiles < most ? tiles : most);
}

gdn2_status shape_check(int B, int T, int Hq, int Hkv, int d, int rot, const float* inv_freq, float eps, bool packed, gdn2_dtype dt) {
    if (!attn_dtype_ok(dt) || B < 0 || T < 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || rot < 0 || rot > d || !(eps >= 0.f)) return GDN2_ERR_INVALID_ARG;
    if (d % 16 || d > kMaxD || rot % 16 || Hq > 4096 || Hkv > 4096) return GDN2_ERR_UNSUPPORTED;
    if (rot && !inv_freq) return GDN2_ERR_INVALID_ARG;
    if ((packed ? (long long)T : (long long)B * T) >= (1LL << 30) || B >= (1 << 30)) return GDN2_ERR_UNSUPPORTED;
    return GDN2_OK;
}

gdn2_status rows_check(const void* p, long long ld, long long width) {
    if (!p || ld < width) return GDN2_ERR_INVALID_ARG;
    if (ld >= (1LL << 31)) return GDN2_ERR_UNSUPPORTED;
    return aligned16(p) && ld % 8 == 0 ? GDN2_OK : GDN2_ERR_MISALIGNED;
}

gdn2_status params_check(const float* q_weight, const float* k_weight, const float* inv_freq, const int32_t* positions, const int32_t* offsets) {
    return aligned16(q_weight) && aligned16(k_weight) && aligned_to(inv_freq, 4) && aligned_to(positions, 4) && aligned_to(offsets, 4)
               ? GDN2_OK
               : GDN2_ERR_MISALIGNED;
}

// Where tiles of one token leave SMs idle, the heads of a token are shared out over blocks too.
dim3 forward_grid(PrologueArgs& a, long long rows) {
    a.tokens = tokens_of(a.d, rows);
    const long long tiles = (rows + a.tokens - 1) / a.tokens;
    a.tiles = static_cast<int>(tiles);
    const int heads = a.Hq + a.Hkv + (a.cache.table ? a.Hkv : 0), groups = kThreads / lanes_of(a.d) / a.tokens;
    long long y = 1;
    if (tiles < 152) {
        y = (heads + groups - 1) / groups;
        if (y > 304 / tiles) y = 304 / tiles;
        if (y < 1) y = 1;
    }
    return dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(y));
}

gdn2_status run_forward(PrologueArgs& a, bool pairs, gdn2_dtype dt, cudaStream_t s) {
    const dim3 grid = forward_grid(a, a.seqs.rows());
    const cudaError_t e = dt == GDN2_BF16 ? launch<__nv_bfloat16>(a, grid, pairs, false, s) : launch<float>(a, grid, pairs, false, s);
    return e == cudaSuccess ? GDN2_OK : GDN2_ERR_CUDA;
}

}  // namespace
}  // namespace gdn2

using namespace gdn2;

extern "C" {

gdn2_status gdn2_attn_prologue(const void* q, long long ld_q, const void* k, long long ld_k, const float* q_weight, const float* k_weight,
                               const float* inv_freq, const int32_t* positions, const int32_t* offsets, void* q_out, void* k_out, int B,
                               int T, int Hq, int Hkv, int d, int rot, int interleaved, float eps, gdn2_dtype dt, void* stream) {
    gdn2_status st = shape_check(B, T, Hq, Hkv, d, rot, inv_freq, eps, offsets != nullptr, dt);
    if (st != GDN2_OK || (st = params_check(q_weight, k_weight, inv_freq, positions, offsets)) != GDN2_OK) return st;
    const Seqs seqs{offsets, B, T};
    if (B == 0 || seqs.rows() == 0) return GDN2_OK;
    if ((st = rows_check(q, ld_q, (long long)Hq * d)) != GDN2_OK || (st = rows_check(k, ld_k, (long long)Hkv * d)) != GDN2_OK) return st;
    if (!q_out || !k_out) return GDN2_ERR_INVALID_ARG;
    if (!aligned16(q_out) || !aligned16(k_out)) return GDN2_ERR_MISALIGNED;
    PrologueArgs a{};
    a.q = q; a.k = k; a.ld_q = ld_q; a.ld_k = ld_k;
    a.q_weight = q_weight; a.k_weight = k_weight; a.inv_freq = inv_freq; a.positions = positions;
    a.seqs = seqs; a.q_out = q_out; a.k_out = k_out;
    a.Hq = Hq; a.Hkv = Hkv; a.d = d; a.rot = rot; a.eps = eps; a.inv_d = 1.f / d;
    return run_forward(a, interleaved != 0, dt, static_cast<cudaStream_t>(stream));
}

gdn2_status gdn2_attn_prologue_paged(const void* q, long long ld_q, const void* k, long long ld_k, const void* v, long long ld_v,
                                     const float* q_weight, const float* k_weight, const float* inv_freq, const int32_t* positions,
                                     const int32_t* offsets, void* q_out, void* k_pages, void* v_pages, const int32_t* table,
                                     const int32_t* lengths, const int32_t* slots, int n_slots, int n_pages, int max_pages, int page, int B,
                                     int T, int Hq, int Hkv, int d, int rot, int interleaved, float eps, gdn2_dtype dt, void* stream) {
    gdn2_status st = shape_check(B, T, Hq, Hkv, d, rot, inv_freq, eps, offsets != nullptr, dt);
    if (st != GDN2_OK || (st = params_check(q_weight, k_weight, inv_freq, positions, offsets)) != GDN2_OK) return st;
    if ((st = cache_check(table, lengths, slots, n_slots, n_pages, max_pages, page)) != GDN2_OK) return st;
    const Seqs seqs{offsets, B, T};
    if (B == 0 || seqs.rows() == 0) return GDN2_OK;
    if ((st = rows_check(q, ld_q, (long long)Hq * d)) != GDN2_OK || (st = rows_check(k, ld_k, (long long)Hkv * d)) != GDN2_OK ||
        (st = rows_check(v, ld_v, (long long)Hkv * d)) != GDN2_OK)
        return st;
    if (!q_out || (n_pages && (!k_pages || !v_pages))) return GDN2_ERR_INVALID_ARG;
    if (!aligned16(q_out) || !aligned16(k_pages) || !aligned16(v_pages)) return GDN2_ERR_MISALIGNED;
    PrologueArgs a{};
    a.q = q; a.k = k; a.v = v; a.ld_q = ld_q; a.ld_k = ld_k; a.ld_v = ld_v;
    a.q_weight = q_weight; a.k_weight = k_weight; a.inv_freq = inv_freq; a.positions = positions;
    a.seqs = seqs; a.cache = Cache{table, lengths, slots, n_slots, n_pages, max_pages, page};
    a.q_out = q_out; a.k_out = k_pages; a.v_out = v_pages;
    a.Hq = Hq; a.Hkv = Hkv; a.d = d; a.rot = rot; a.eps = eps; a.inv_d = 1.f / d;
    return run_forward(a, interleaved != 0, dt, static_cast<cudaStream_t>(stream));
}

size_t gdn2_attn_prologue_backward_workspace_size(int B, int T, int d, int packed) {
    const long long rows = packed ? (long long)T : (long long)B * T;
    if (B <= 0 || T <= 0 || d <= 0 || d % 16 || d > kMaxD || rows >= (1LL << 30)) return 0;
    return sizeof(float) * 2 * d * grad_blocks(d, rows);
}

gdn2_status gdn2_attn_prologue_backward(const void* q, long long ld_q, const void* k, long long ld_k, const float* q_weight,
                                        const float* k_weight, const float* inv_freq, const int32_t* positions, const int32_t* offsets,
                                        const void* dq_out, long long ld_dqo, const void* dk_out, long long ld_dko, void* dq,
                                        long long ld_dq, void* dk, long long ld_dk, float* dq_weight, float* dk_weight, int B, int T, int Hq,
                                        int Hkv, int d, int rot, int interleaved, float eps, gdn2_dtype dt, void* workspace, size_t ws_bytes,
                                        void* stream) {
    gdn2_status st = shape_check(B, T, Hq, Hkv, d, rot, inv_freq, eps, offsets != nullptr, dt);
    if (st != GDN2_OK || (st = params_check(q_weight, k_weight, inv_freq, positions, offsets)) != GDN2_OK) return st;
    if ((q_weight && !dq_weight) || (k_weight && !dk_weight) || (!q_weight && dq_weight) || (!k_weight && dk_weight)) return GDN2_ERR_INVALID_ARG;
    if (!aligned_to(dq_weight, 4) || !aligned_to(dk_weight, 4)) return GDN2_ERR_MISALIGNED;
    const Seqs seqs{offsets, B, T};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (B == 0 || seqs.rows() == 0) {  // sums over no rows
        cudaError_t e = cudaSuccess;
        if (dq_weight) e = cudaMemsetAsync(dq_weight, 0, sizeof(float) * d, s);
        if (dk_weight && e == cudaSuccess) e = cudaMemsetAsync(dk_weight, 0, sizeof(float) * d, s);
        return e == cudaSuccess ? GDN2_OK : GDN2_ERR_CUDA;
    }
    const long long wq = (long long)Hq * d, wk = (long long)Hkv * d;
    const struct { const void* p; long long ld, w; } t[] = {{q, ld_q, wq}, {k, ld_k, wk}, {dq_out, ld_dqo, wq}, {dk_out, ld_dko, wk}, {dq, ld_dq, wq}, {dk, ld_dk, wk}};
    for (const auto& r : t)
        if ((st = rows_check(r.p, r.ld, r.w)) != GDN2_OK) return st;
    PrologueArgs a{};
    a.tokens = tokens_of(d, seqs.rows());
    a.tiles = static_cast<int>((seqs.rows() + a.tokens - 1) / a.tokens);
    const int blocks = grad_blocks(d, seqs.rows());
    if (q_weight || k_weight) {
        if (!workspace || ws_bytes < sizeof(float) * 2 * d * blocks) return GDN2_ERR_WORKSPACE;
        if (!aligned16(workspace)) return GDN2_ERR_MISALIGNED;
        a.parts = static_cast<float*>(workspace);
    }
    a.q = q; a.k = k; a.ld_q = ld_q; a.ld_k = ld_k;
    a.q_weight = q_weight; a.k_weight = k_weight; a.inv_freq = inv_freq; a.positions = positions;
    a.seqs = seqs; a.q_out = dq; a.k_out = dk; a.ld_dq = ld_dq; a.ld_dk = ld_dk;
    a.gq = dq_out; a.gk = dk_out; a.ld_gq = ld_dqo; a.ld_gk = ld_dko;
    a.Hq = Hq; a.Hkv = Hkv; a.d = d; a.rot = rot; a.eps = eps; a.inv_d = 1.f / d;
    cudaError_t e = dt == GDN2_BF16 ? launch<__nv_bfloat16>(a, dim3(blocks), interleaved != 0, true, s)
                                    : launch<float>(a, dim3(blocks), interleaved != 0, true, s);
    if (e == cudaSuccess && a.parts) {
        weight_grad_kernel<<<dim3((d + 31) / 32, 2), 1024, 0, s>>>(a.parts, blocks, d, dq_weight, dk_weight);
        e = cudaGetLastError();
    }
    return e == cudaSuccess ? GDN2_OK : GDN2_ERR_CUDA;
}

}  // extern "C"
