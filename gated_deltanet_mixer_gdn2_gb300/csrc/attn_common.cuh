// attn_common.cuh -- shared by the operators of attention layers: the paged cache of keys and values, and the position rotation.
#pragma once

#include <atomic>

#include "ssm_common.cuh"

namespace gdn2 {

// A cache of keys and values in pages. Row `slot` of the table names the pages of one sequence in order: its token t lies in page
// table[slot][t / page] at t % page, in each pool as [n_pages, H_kv, page, d]. lengths[slot] counts its tokens, those of the present
// call among them. All of it lives on the device and cannot be checked on the host: lengths are clamped to what the table can name,
// and an entry outside [0, n_pages) is no page, so that wrong ones give wrong results, never an access outside the pools.
struct Cache {
    const int *table, *lengths, *slots;
    int n_slots, n_pages, max_pages, page;
    // The table row of batch row b; negative where the row is inactive.
    __device__ __forceinline__ int row_of(int b) const {
        const int s = slots ? __ldg(slots + b) : b;
        return s >= 0 && s < n_slots ? s : -1;
    }
    __device__ __forceinline__ int length_of(int row) const {
        return static_cast<int>(min(max(static_cast<long long>(__ldg(lengths + row)), 0LL), static_cast<long long>(max_pages) * page));
    }
    __device__ __forceinline__ int entry(int row, int i) const {
        const int p = __ldg(table + static_cast<long long>(row) * max_pages + i);
        return p >= 0 && p < n_pages ? p : -1;
    }
};

// SMs of the current device, asked for once per device (a call's grid and workspace go by it). 152 where there is none.
inline int sm_count() {
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 152;
    if (dev < kDevices && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 152;
    if (dev < kDevices) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

inline bool attn_dtype_ok(gdn2_dtype dt) { return dt == GDN2_F32 || dt == GDN2_BF16; }

// Sizes of a cache: every index of a table fits an int, as does the number of a row's tokens.
inline gdn2_status cache_check(const int32_t* table, const int32_t* lengths, const int32_t* slots, int n_slots, int n_pages, int max_pages,
                               int page) {
    if (!table || !lengths || n_slots < 0 || n_pages < 0 || max_pages <= 0 || page <= 0) return GDN2_ERR_INVALID_ARG;
    if (page > 65536 || static_cast<long long>(max_pages) * page >= (1LL << 30) || static_cast<long long>(n_slots) * max_pages >= (1LL << 40))
        return GDN2_ERR_UNSUPPORTED;
    if (!aligned_to(table, 4) || !aligned_to(lengths, 4) || !aligned_to(slots, 4)) return GDN2_ERR_MISALIGNED;
    return GDN2_OK;
}

}  // namespace gdn2
