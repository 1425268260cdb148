// ssm_tc.cuh -- shared by the tensor-core kernels of the selective state-space scan: warp-uniform waits and
// products, tensor maps, and launchers used across their translation units. Everything inside the anonymous
// namespace has internal linkage; each translation unit has its own device status word.
#pragma once

#include <atomic>

#include "ssm_common.cuh"
#include "tc_common.cuh"

namespace gdn2 {
namespace {

constexpr int kQ = 128;    // tokens per chunk
constexpr int kCols = 64;  // value columns per block
constexpr uint32_t kTileBytes = 16384;  // [128 rows][64 bf16], 128-byte swizzle

// Bounded wait on a barrier's phase by a converged warp: the first try inline, the loop out of line (inlined at
// every wait it made half of the kernel's code). The outcome is the warp's; a warp that gives up records it.
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, long long lim, volatile int* err) {
    return warp_wait(reinterpret_cast<uint64_t*>(__cvta_shared_to_generic(bar)), parity, lim, err);
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, long long lim, volatile int* err) {
    if (__all_sync(0xffffffffu, lim > 0 && mbar_try_wait(bar, parity))) return true;
    return wait_on(smem_u32(bar), parity, lim, err);
}

// One elected lane of a converged warp issues; the operands are warp-uniform, so that descriptors advance
// in uniform registers (an `if (lane == 0)` around the loop made every product of 8 steps take 1200 cycles to issue).
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t e;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
    return e;
}
// A value that is the same in all lanes, in a form that the compiler knows to be.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// Shared-memory descriptor: the constant upper word (stride 1024, version, 128-byte swizzle) and the lower one, which
// holds the start address and the leading offset and advances by plain addition of bytes / 16 (no carry out of
// the 14-bit address: shared memory ends below 256 KB).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return ((saddr & 0x3FFFFu) >> 4) | (lbo >> 4 << 16); }

__device__ __forceinline__ void mma_by(uint32_t lead, uint32_t d, uint32_t ad, uint32_t bd, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p, e;\n .reg .b64 a, b;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %5, 0;\n mov.b64 a, {%1, %6};\n"
        " mov.b64 b, {%2, %6};\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d), "r"(ad), "r"(bd), "r"(id),
        "r"(acc), "r"(lead), "r"(kDescHi)
        : "memory");
}
__device__ __forceinline__ void mma_ts_by(uint32_t lead, uint32_t d, uint32_t at, uint32_t bd, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p, e;\n .reg .b64 b;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %5, 0;\n mov.b64 b, {%2, %6};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d), "r"(at), "r"(bd), "r"(id), "r"(acc), "r"(lead),
        "r"(kDescHi)
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// A product over up to 8 steps of 16 along K (`steps` 4 or 8), the operands' start advancing by a step and, after four
// steps, by a jump more. Unrolled to a handful of instructions per step: the other warps of the issuing warp's
// scheduler leave it few slots (under a full load of multiplications a rolled loop took 1200 cycles per step, this one
// 240; alone both take the tensor core's 48).
template <bool kFromTmem, int kDa, int kDb, int kJa, int kJb>
__device__ __forceinline__ void mma_steps(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc, int steps) {
#pragma unroll
    for (int s = 0; s < 8; ++s) {
        if (s >= 4 && steps <= 4) break;
        const uint32_t as = a + s * kDa + (s >= 4 ? kJa : 0), bs = b + s * kDb + (s >= 4 ? kJb : 0);
        if (kFromTmem) mma_ts_by(lead, d, as, bs, id, s ? 1 : acc);
        else mma_by(lead, d, as, bs, id, s ? 1 : acc);
    }
}
// Operand advances in descriptor units (16 bytes): K-major tiles hold 64 channels in 128-byte rows (32 bytes a step, the
// next tile after four); MN-major ones a token or state row per 128 bytes (16 rows a step).
constexpr int kStepK = 2, kJumpK = (kTileBytes >> 4) - 8, kStepMn = 128;

__device__ __forceinline__ void commit_by(uint32_t lead, uint64_t* bar) {
    asm volatile(
        "{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar)), "r"(lead)
        : "memory");
}

__device__ __forceinline__ float4 exp2_4(float4 v) {
    return make_float4(ex2_approx(v.x), ex2_approx(v.y), ex2_approx(v.z), ex2_approx(v.w));
}

// [rows, heads, width] bf16 with a row stride, as (width, heads, rows); box (64, 1, box_rows)
bool rows_map(CUtensorMap* m, const void* p, long long ld, int width, int heads, long long rows, int box_rows) {
    const uint64_t dims[3] = {(uint64_t)width, (uint64_t)heads, (uint64_t)rows};
    const uint64_t st[2] = {(uint64_t)width * 2, (uint64_t)ld * 2};
    const uint32_t box[3] = {64, 1, (uint32_t)box_rows};
    return make_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p, dims, st, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Whether this translation unit's kernels have been launched or captured in this process. Until then their status word
// holds nothing, and reading it (two waits of the stream) would only make the other kernels' status later.
std::atomic<bool> g_launched{false};

int read_clear_status(cudaStream_t s) {
    if (!g_launched.load(std::memory_order_relaxed)) return 0;
    int v = 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_status_tc, sizeof(int), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess) return -1;
    if (cudaStreamSynchronize(s) != cudaSuccess) return -1;
    const int zero = 0;
    if (v && cudaMemcpyToSymbolAsync(g_status_tc, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s) != cudaSuccess) return -1;
    cudaStreamSynchronize(s);
    return v;
}

}  // namespace

// One walk of the states over chunks (ssm_tc_walk.cu): forward of B and x, or backward of C and dy.
struct WalkJob {
    Rows keys, values;       // B and x, or C and dy
    const float* first;      // [B][H][N][P] state at the sequences' start (back: adjoint at their end), or null
    float* last;             // [B][H][N][P] at the other end, or null
    float* states;           // [units][H][N][P]: what a unit adds (increments), or its starting state
    float* decay;            // [units][H] log-decay of a unit, natural units (increments)
    void* save;              // the state before every chunk: [chunks][H][P / 64] bf16 tiles in the operand layout, or null
    int back;
};
// Increments of every unit from zero states (increments != 0), or the walk from the units' starting states (cut)
// or the sequences' (one unit each). exact: the states are results in fp32.
cudaError_t launch_ssm_walk_tc(const ScanShape& sh, const void* step, const void* g, const WalkJob* jobs, int n_jobs, int unit,
                               int increments, int cut, int exact, cudaStream_t s, long long wait_ns);
}  // namespace gdn2
