// attn_prologue.cu -- what an attention layer does to its queries and keys between projection and attention, in one pass: RMS norm
// over each head and rotation by position; for serving with k and v written to the pages of a cache; and the gradients.
//     n = w x / sqrt(mean(x^2) + eps)        (y_a, y_b) = (n_a cos - n_b sin, n_b cos + n_a sin),  angle = position * inv_freq
// for the pairs (a, b) of the first `rot` elements: (j, j + rot / 2), or (2 j, 2 j + 1) when interleaved.
//
// Bound by memory: every element is read once and written once for some 10 operations. A head's row belongs to a group of lanes, eight
// elements each, so that its sum of squares and the pairs' other halves come by shuffles; a group keeps to one token, whose cosines
// and sines it holds in registers, and has several rows' loads in flight.
#include "attn_common.cuh"

namespace gdn2 {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 8;    // tokens of a tile at most: the angles of a tile are formed once, two or so per thread
constexpr int kMaxD = 256;

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
// kTurns = 2^66 / (2 pi). position * turns, wrapping, is the angle modulo a turn to 2^-64 per position: exact enough (2^-33 of a turn) for
// any 32-bit position, where a 32-bit product would lose the angle from some ten thousand positions on.
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
    int position[kTokens], live[kTokens], page[kTokens], at[kTokens];
    float cs[kTokens][kMaxD / 2], sn[kTokens][kMaxD / 2];
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

template <typename T>
struct Raw8;  // eight elements as they are loaded
template <>
struct Raw8<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = u; }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static constexpr int kFlight = 4;
};
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldg(reinterpret_cast<const float4*>(p));
        b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void store(float* p) const {
        reinterpret_cast<float4*>(p)[0] = a;
        reinterpret_cast<float4*>(p)[1] = b;
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    static constexpr int kFlight = 2;
};

template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int m = L / 2; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// The lane's part of a token's rotation: elements 8 lane .. 8 lane + 7.
template <bool kPairs>
struct Turn {
    float c[8], s[8];  // of each element; kPairs: of its four pairs, in the first half
    int partner;       // lane with the pairs' other halves; negative: these elements are not rotated
    __device__ __forceinline__ void set(const PrologueArgs& a, const TileShared& sh, int token, int lane) {
        const int half = a.rot / 2, i0 = 8 * lane;
        partner = -1;
        if (i0 >= a.rot) return;
        if constexpr (kPairs) {
            partner = lane;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c[i] = sh.cs[token][i0 / 2 + i];
                s[i] = sh.sn[token][i0 / 2 + i];
            }
        } else {
            const bool low = i0 < half;
            partner = low ? lane + half / 8 : lane - half / 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                c[i] = sh.cs[token][(low ? i0 : i0 - half) + i];
                s[i] = low ? -sh.sn[token][i0 + i] : sh.sn[token][i0 - half + i];  // a cos - b sin, b cos + a sin
            }
        }
    }
    // Rotates x in place; back: by the opposite angle. All lanes of the warp take part; `first` is the group's first lane.
    template <bool kBack>
    __device__ __forceinline__ void apply(float (&x)[8], int first) const {
        if constexpr (kPairs) {
            if (partner < 0) return;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float p = x[2 * i], q = x[2 * i + 1], sv = kBack ? -s[i] : s[i];
                x[2 * i] = fmaf(p, c[i], -q * sv);
                x[2 * i + 1] = fmaf(q, c[i], p * sv);
            }
        } else {
            const int from = first + (partner < 0 ? 0 : partner);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float o = __shfl_sync(0xffffffffu, x[i], from);
                if (partner >= 0) x[i] = fmaf(x[i], c[i], o * (kBack ? -s[i] : s[i]));
            }
        }
    }
};

// Group geometry of a block: kThreads / L groups, those of one token apart by `tokens`.
template <typename T, int L, bool kPairs>
__global__ void __launch_bounds__(kThreads, 3) prologue_kernel(const __grid_constant__ PrologueArgs a) {
    __shared__ TileShared sh;
    __shared__ __align__(16) float w[2][kMaxD];
    const long long rows = a.seqs.offsets ? a.seqs.T : static_cast<long long>(a.seqs.B) * a.seqs.T;
    const long long row0 = static_cast<long long>(blockIdx.x) * a.tokens;
    for (int j = threadIdx.x; j < a.d; j += kThreads) {
        w[0][j] = a.q_weight ? a.q_weight[j] : 1.f;
        w[1][j] = a.k_weight ? a.k_weight[j] : 1.f;
    }
    frequencies(a, sh);
    enter_tile(a, sh, row0, rows);

    const int lane = threadIdx.x % L, group = threadIdx.x / L, groups = kThreads / L, first = (threadIdx.x & 31) - lane;
    const int token = group % a.tokens, part = group / a.tokens + blockIdx.y * (groups / a.tokens), step = groups / a.tokens * gridDim.y;
    const bool mine = 8 * lane < a.d;
    const bool live = sh.live[token];
    Turn<kPairs> turn;
    turn.set(a, sh, token, lane);
    const int page = sh.page[token], at = sh.at[token];
    const long long r = row0 + token;
    const int heads = a.Hq + a.Hkv + (a.cache.table ? a.Hkv : 0);
    constexpr int kFlight = Raw8<T>::kFlight;
    for (int h0 = part; __any_sync(0xffffffffu, h0 < heads); h0 += kFlight * step) {
        Raw8<T> raw[kFlight];
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const int h = h0 + u * step;
            if (!live || !mine || h >= heads) continue;
            const T* row = h < a.Hq           ? static_cast<const T*>(a.q) + r * a.ld_q + static_cast<long long>(h) * a.d
                           : h < a.Hq + a.Hkv ? static_cast<const T*>(a.k) + r * a.ld_k + static_cast<long long>(h - a.Hq) * a.d
                                              : static_cast<const T*>(a.v) + r * a.ld_v + static_cast<long long>(h - a.Hq - a.Hkv) * a.d;
            raw[u].load(row + 8 * lane);
        }
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const int h = h0 + u * step;
            if (!__any_sync(0xffffffffu, h < heads)) break;
            const bool here = live && mine && h < heads;
            const int kind = h < a.Hq ? 0 : h < a.Hq + a.Hkv ? 1 : 2, hk = h - a.Hq - (kind == 2 ? a.Hkv : 0);
            float x[8];
            if (here) {
                raw[u].get(x);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = 0.f;
            }
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
            ss = group_sum<L>(ss);
            if ((kind ? a.k_weight : a.q_weight) && mine) {  // without weights there is no norm
                const float inv = rsqrtf(fmaf(ss, a.inv_d, a.eps));
                const float4 w0 = *reinterpret_cast<const float4*>(&w[kind & 1][8 * lane]), w1 = *reinterpret_cast<const float4*>(&w[kind & 1][8 * lane + 4]);
                const float wv[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] *= inv * wv[i];
            }
            turn.template apply<false>(x, first);
            if (!here) continue;
            if (kind == 0) {
                Vec8<T>::store(static_cast<T*>(a.q_out) + (r * a.Hq + h) * a.d + 8 * lane, x);
            } else if (!a.cache.table) {
                Vec8<T>::store(static_cast<T*>(a.k_out) + (r * a.Hkv + hk) * a.d + 8 * lane, x);
            } else if (page >= 0) {
                const long long to = ((static_cast<long long>(page) * a.Hkv + hk) * a.cache.page + at) * a.d + 8 * lane;
                if (kind == 1) Vec8<T>::store(static_cast<T*>(a.k_out) + to, x);
                else raw[u].store(static_cast<T*>(a.v_out) + to);
            }
        }
    }
}

// Gradients: dn = dy turned back; dw = sum over tokens and heads of dn xh with xh = x inv; dx = inv (w dn - xh mean(w dn xh)).
// Blocks walk tiles one after another and leave one partial sum of the weights' gradients each.
template <typename T, int L, bool kPairs>
__global__ void __launch_bounds__(kThreads, 3) prologue_grad_kernel(const __grid_constant__ PrologueArgs a) {
    __shared__ TileShared sh;
    __shared__ __align__(16) float red[kThreads / L][L * 8];
    const long long rows = a.seqs.offsets ? a.seqs.T : static_cast<long long>(a.seqs.B) * a.seqs.T;
    const int lane = threadIdx.x % L, group = threadIdx.x / L, groups = kThreads / L, first = (threadIdx.x & 31) - lane;
    const int token = group % a.tokens, part = group / a.tokens, step = groups / a.tokens;
    const bool mine = 8 * lane < a.d;
    float acc[2][8] = {};
    frequencies(a, sh);
    for (int tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
        const long long row0 = static_cast<long long>(tile) * a.tokens;
        __syncthreads();
        enter_tile(a, sh, row0, rows);
        const bool live = sh.live[token];
        Turn<kPairs> turn;
        turn.set(a, sh, token, lane);
        const long long r = row0 + token;
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            const int H = side ? a.Hkv : a.Hq;
            const float* weight = side ? a.k_weight : a.q_weight;
            const T* xs = static_cast<const T*>(side ? a.k : a.q) + r * (side ? a.ld_k : a.ld_q) + 8 * lane;
            const T* gs = static_cast<const T*>(side ? a.gk : a.gq) + r * (side ? a.ld_gk : a.ld_gq) + 8 * lane;
            T* out = static_cast<T*>(side ? a.k_out : a.q_out) + r * (side ? a.ld_dk : a.ld_dq) + 8 * lane;
            float wv[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) wv[i] = weight && mine ? __ldg(weight + 8 * lane + i) : 1.f;
            constexpr int kFlight = 2;
            for (int h0 = part; __any_sync(0xffffffffu, h0 < H); h0 += kFlight * step) {
                Raw8<T> rx[kFlight], rg[kFlight];
#pragma unroll
                for (int u = 0; u < kFlight; ++u) {
                    const int h = h0 + u * step;
                    if (!live || !mine || h >= H) continue;
                    rg[u].load(gs + static_cast<long long>(h) * a.d);
                    if (weight) rx[u].load(xs + static_cast<long long>(h) * a.d);
                }
#pragma unroll
                for (int u = 0; u < kFlight; ++u) {
                    const int h = h0 + u * step;
                    if (!__any_sync(0xffffffffu, h < H)) break;
                    const bool here = live && mine && h < H;
                    float g[8], x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) g[i] = x[i] = 0.f;
                    if (here) {
                        rg[u].get(g);
                        if (weight) rx[u].get(x);
                    }
                    turn.template apply<true>(g, first);
                    if (weight) {
                        float ss = 0.f, gx = 0.f;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            ss = fmaf(x[i], x[i], ss);
                            gx = fmaf(g[i] * wv[i], x[i], gx);
                        }
                        ss = group_sum<L>(ss);
                        gx = group_sum<L>(gx);
                        const float inv = rsqrtf(fmaf(ss, a.inv_d, a.eps)), m = gx * inv * a.inv_d;
                        if (here) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float xh = x[i] * inv;
                                acc[side][i] = fmaf(g[i], xh, acc[side][i]);
                                g[i] = inv * fmaf(-xh, m, g[i] * wv[i]);
                            }
                        }
                    }
                    if (here) Vec8<T>::store(out + static_cast<long long>(h) * a.d, g);
                }
            }
        }
    }
    if (!a.parts) return;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) red[group][8 * lane + i] = acc[side][i];
        __syncthreads();
        for (int c = threadIdx.x; c < a.d; c += kThreads) {
            float v = 0.f;
            for (int k = 0; k < groups; ++k) v += red[k][c];
            a.parts[(static_cast<long long>(blockIdx.x) * 2 + side) * a.d + c] = v;
        }
    }
}

// The blocks' partial sums, added in their order: 32 columns a block, its warps each a share of the parts.
__global__ void __launch_bounds__(kThreads) weight_grad_kernel(const float* parts, int n, int d, float* dq_weight, float* dk_weight) {
    __shared__ float red[kThreads / 32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, side = blockIdx.y, c = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (c < d)
        for (int k = warp; k < n; k += kThreads / 32) v += parts[(static_cast<long long>(k) * 2 + side) * d + c];
    red[warp][lane] = v;
    __syncthreads();
    float* out = side ? dk_weight : dq_weight;
    if (warp == 0 && c < d && out) {
        for (int k = 1; k < kThreads / 32; ++k) v += red[k][lane];
        out[c] = v;
    }
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 152;
    return n > 0 ? n : 152;
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

// Lanes of a head's row, and tokens of a tile: as many as there are blocks for all SMs without, eight at most.
int lanes_of(int d) { return d <= 64 ? 8 : d <= 128 ? 16 : 32; }
int tokens_of(int d, long long rows) {
    int t = kTokens;
    while (t > 1 && rows < 608LL * t) t /= 2;
    const int groups = kThreads / lanes_of(d);
    return t < groups ? t : groups;
}

int grad_blocks(int d, long long rows) {
    const int t = tokens_of(d, rows);
    const long long tiles = (rows + t - 1) / t, most = 3LL * sm_count();
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
        weight_grad_kernel<<<dim3((d + 31) / 32, 2), kThreads, 0, s>>>(a.parts, blocks, d, dq_weight, dk_weight);
        e = cudaGetLastError();
    }
    return e == cudaSuccess ? GDN2_OK : GDN2_ERR_CUDA;
}

}  // extern "C"
