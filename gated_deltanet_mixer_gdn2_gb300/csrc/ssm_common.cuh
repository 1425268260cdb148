// ssm_common.cuh -- shared by the selective state-space operators: where the sequences of a call lie
// (equal lengths, or packed one after the other), how they are cut into units, and the gate functions.
#pragma once

#include "common.cuh"
#include "ptx.cuh"

namespace gdn2 {

// The sequences of a call. offsets == nullptr: B sequences of T tokens, sequence b at rows b*T.. .
// Otherwise sequence b is rows [offsets[b], offsets[b+1]) of T rows in all. Offsets live on the device
// and cannot be checked on the host, so every use goes through span(), which clamps them to [0, T], and what
// lies in a workspace per unit through held(): wrong offsets give wrong results, never an access outside the
// tensors or the workspace.
struct Seqs {
    const int* offsets;
    int B, T;
    __device__ __forceinline__ void span(int b, int& start, int& len) const {
        if (!offsets) {
            start = b * T;
            len = T;
            return;
        }
        const int lo = min(max(__ldg(offsets + b), 0), T), hi = min(max(__ldg(offsets + b + 1), 0), T);
        start = lo;
        len = max(hi - lo, 0);
    }
    // Token rows [lo, hi) of all sequences together: each ends where the next one starts, so with ascending offsets they are
    // one stretch. Rows before and behind it belong to no sequence.
    __device__ __forceinline__ void covered(long long& lo, long long& hi) const {
        lo = offsets ? min(max(__ldg(offsets), 0), T) : 0;
        hi = offsets ? min(max(__ldg(offsets + B), 0), T) : static_cast<long long>(B) * T;
    }
    long long rows() const { return offsets ? (long long)T : (long long)B * T; }
    // Units of `unit` tokens over all sequences, an empty sequence counted as one unit: exact for equal
    // lengths, an upper bound (unknown to the host) for packed ones.
    __host__ __device__ long long units(int unit) const {
        if (!offsets) return (long long)B * (T > 0 ? (T + unit - 1) / unit : 1);
        return static_cast<long long>(T / unit) + B;
    }
    // Units of one sequence.
    __host__ __device__ __forceinline__ static int units_of(int len, int unit) { return len > unit ? (len + unit - 1) / unit : 1; }
    // How many of a sequence's `count` units from number `base` on a workspace of `room` = units(unit) entries holds: all,
    // unless the offsets do not ascend, for then the lengths add up to more than T. The rest is neither written nor read.
    __host__ __device__ __forceinline__ static int held(long long base, int count, int room) {
        return room - base >= count ? count : room > base ? static_cast<int>(room - base) : 0;
    }
};

// One unit of a sequence: its place among the sequence's units and its tokens.
struct Unit {
    int seq, k, count;  // unit k of `count` of sequence seq
    int row, len;       // first token row and tokens (0 for an empty sequence)
};

// Unit number `idx` of a call. False past the last one. Every lane of the calling warp gets the answer;
// the warps of a block may call it independently.
__device__ __forceinline__ bool find_unit(const Seqs& s, int unit, int idx, Unit& u) {
    int start = 0, len = 0;
    if (!s.offsets) {
        const int per = Seqs::units_of(s.T, unit);
        u.seq = idx / per;
        if (u.seq >= s.B) return false;
        u.k = idx - u.seq * per;
        start = u.seq * s.T;
        len = s.T;
    } else {
        // 32 sequences at a time: their unit counts, a warp prefix sum, and the lane that holds idx
        const int lane = threadIdx.x & 31;
        int base = 0, found = -1;
        for (int b0 = 0; b0 < s.B; b0 += 32) {
            int st = 0, ln = 0, n = 0;
            if (b0 + lane < s.B) {
                s.span(b0 + lane, st, ln);
                n = Seqs::units_of(ln, unit);
            }
            int incl = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += v;
            }
            const unsigned m = __ballot_sync(0xffffffffu, idx < base + incl);
            if (m) {
                const int src = __ffs(m) - 1;
                found = b0 + src;
                u.k = idx - base - __shfl_sync(0xffffffffu, incl - n, src);
                start = __shfl_sync(0xffffffffu, st, src);
                len = __shfl_sync(0xffffffffu, ln, src);
                break;
            }
            base += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (found < 0) return false;
        u.seq = found;
    }
    u.count = Seqs::units_of(len, unit);
    u.row = start + u.k * unit;
    u.len = min(unit, len - u.k * unit);
    return true;
}

// Units of the sequences before `seq`, by a whole warp (64 bits: offsets that do not ascend may add up to any length).
__device__ __forceinline__ long long units_before(const Seqs& s, int unit, int seq) {
    if (!s.offsets) return static_cast<long long>(seq) * Seqs::units_of(s.T, unit);
    const int lane = threadIdx.x & 31;
    long long n = 0;
    for (int b = lane; b < seq; b += 32) {
        int start, len;
        s.span(b, start, len);
        n += Seqs::units_of(len, unit);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) n += __shfl_xor_sync(0xffffffffu, n, d);
    return n;
}

// The sequence that holds token row r and the row its successor starts at; false if no sequence holds it.
__device__ __forceinline__ bool find_row(const Seqs& s, int r, int& seq, int& start, int& end) {
    if (!s.offsets) {
        seq = r / s.T;
        start = seq * s.T;
        end = start + s.T;
        return true;
    }
    int lo = 0, hi = s.B;  // the last sequence that starts at or before r
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (__ldg(s.offsets + m) <= r) lo = m; else hi = m;
    }
    int len;
    s.span(lo, start, len);
    seq = lo;
    end = start + len;
    return r >= start && r < end;
}

// 1 / (1 + e^-v) with the hardware's approximations, each within 2 units in the last place, of an argument rounded once: relative
// error 2^-22 + 2^-23 |v| where e^-v counts (1e-6 at v = -20)
__device__ __forceinline__ float ssm_sigmoid(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2_approx(-kLog2e * v)));
    return r;
}
// log(1 + e^v), exact to fp32 for either sign
__device__ __forceinline__ float ssm_softplus(float v) { return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))); }

// Log-decays enter every exponential floored (common.cuh): a full reset (g = -inf) keeps sums finite. NaN stays NaN (fmaxf
// would make it a reset).
__device__ __forceinline__ float ssm_gate(float g) { return g < kGateFloor ? kGateFloor : g; }

constexpr float kLn2 = 0.69314718056f;

// e^g as the fp32 sum x + y. A state that decays by 1 - 1e-3 a token is multiplied by thousands of factors in which one
// value's rounding, repeated, would add up to 1e-5 and more; with its remainder the factor is exact to 2^-24 |g|.
__device__ __forceinline__ float2 ssm_decay(float g) {
    const float a = expf(g);
    return make_float2(a, a >= 0.5f && a <= 2.f ? expm1f(g) - (a - 1.f) : 0.f);  // a - 1 is exact there
}

inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// One tensor of the scan: pointer and row (token) stride in elements; heads and channels are dense.
struct Rows {
    const void* p;
    long long ld;
};
struct RowsOut {
    void* p;
    long long ld;
};

struct ScanShape {
    Seqs seqs;
    int H, G, P, N;
    gdn2_dtype dt;
};

struct ScanIn {
    Rows x, bm, cm;            // [rows, H, P], [rows, G, N], [rows, G, N]
    const void *step, *g;      // [rows, H]
    const float *d, *s0;       // [H] or null; [B, H, N, P] or null
};

// Launchers of the two kernel families (ssm_scan.cu: CUDA cores; ssm_tc*.cu: tensor cores).
size_t ssm_simt_fwd_workspace(const ScanShape& sh);
cudaError_t launch_ssm_simt_fwd(const ScanShape& sh, const ScanIn& in, void* y, float* s1, void* ws, cudaStream_t s);

struct ScanGrads {
    Rows dy;                     // [rows, H, P]
    const float* ds1;            // [B, H, N, P] or null
    RowsOut dx, dbm, dcm;        // like x, bm, cm
    void *dstep, *dg;            // [rows, H]
    float *dd, *ds0;             // [H] or null; [B, H, N, P] or null
};
size_t ssm_simt_bwd_workspace(const ScanShape& sh);
cudaError_t launch_ssm_simt_bwd(const ScanShape& sh, const ScanIn& in, const ScanGrads& gr, void* ws, cudaStream_t s);

// From units' increments to the states at their starts (back: the adjoints at their ends), one or two directions.
struct ChainJob {
    const float* first;   // state before the first unit, or null
    float *last, *states; // state after the last unit, or null; increments, replaced
    const float* decay;
    int back;
};
cudaError_t launch_ssm_chain(const ScanShape& sh, int unit, const ChainJob* jobs, int n, cudaStream_t s);

// dB and dC from the head shares and dD from the units' parts (ssm_scan.cu).
cudaError_t launch_ssm_grad_sums(const ScanShape& sh, const ScanGrads& gr, const float* part, int splits, const float* dd_part, int units,
                                 cudaStream_t s);

bool ssm_tc_shape(const ScanShape& sh);
size_t ssm_tc_fwd_workspace(const ScanShape& sh);
size_t ssm_tc_bwd_workspace(const ScanShape& sh);
cudaError_t launch_ssm_tc_bwd(const ScanShape& sh, const ScanIn& in, const ScanGrads& gr, void* ws, cudaStream_t s, long long wait_ns);
cudaError_t launch_ssm_tc_fwd(const ScanShape& sh, const ScanIn& in, void* y, float* s1, void* ws, cudaStream_t s, long long wait_ns);

}  // namespace gdn2
