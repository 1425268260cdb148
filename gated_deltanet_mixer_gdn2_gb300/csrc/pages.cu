// pages.cu -- the pages of a cache (attn_common.cuh) and the rows of pools: making room, sharing, giving back, copying. Pages are counted:
// refs[p] table entries name page p, and a page that none names is free. Everything is on the device, so that a serving step needs no
// answer on the host and can be captured. Free pages are given out lowest first and in the order of the requests: the same calls leave
// the same tables, whatever the blocks' order.
//
// Bound by latency: a call is a few dependent passes over some kilobytes, and over all counts. One cluster of blocks does a whole call in one launch, its
// passes ordered by cluster barriers. A token for 64 rows takes 9.5 us with a pool of 1250 pages, 11 with 10^5, 14.7 with 10^6; for 1024 rows 18 and 29
// with the larger ones; a fork of 8 rows of up to 200 pages 13 to 14. What a shortened row holds is looked at by a warp per row: 8192 tokens behind
// a row shortened to nothing take 14.6 us, 131072 (pages of 16) 108, against 19 with the pages given back first.
// The copies are bound by memory: 32 KB pieces, eight 16-byte loads in flight per thread.
#include <cooperative_groups.h>

#include <climits>

#include "attn_common.cuh"

namespace gdn2 {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kCluster = 8;  // the portable size

struct PagesArgs {
    int *table, *lengths, *refs;
    const int *src, *dst;       // fork: from row src[i] to row dst[i]; append, release: dst
    const int* tokens;          // append: tokens of each request, or each of `every`
    int *copy_from, *copy_to, *ok, *active;
    int n, every, n_slots, n_pages, max_pages, page;
};

__device__ __forceinline__ bool is_row(const PagesArgs& a, int s) { return s >= 0 && s < a.n_slots; }
__device__ __forceinline__ bool is_page(const PagesArgs& a, int p) { return p >= 0 && p < a.n_pages; }
__device__ __forceinline__ int length_of(const PagesArgs& a, int s) {
    return static_cast<int>(min(max(static_cast<long long>(a.lengths[s]), 0LL), static_cast<long long>(a.max_pages) * a.page));
}

// Empties the rows dst[i]. An entry is taken by an exchange, so that a row listed twice is given back once.
__device__ __forceinline__ void release_rows(const PagesArgs& a, long long first, long long step) {
    const long long entries = static_cast<long long>(a.n) * a.max_pages;
    for (long long e = first; e < entries; e += step) {
        const int i = static_cast<int>(e / a.max_pages), j = static_cast<int>(e - static_cast<long long>(i) * a.max_pages), s = a.dst[i];
        if (!is_row(a, s)) continue;
        const int p = atomicExch(a.table + static_cast<long long>(s) * a.max_pages + j, -1);
        if (is_page(a, p)) atomicSub(a.refs + p, 1);
        if (j == 0) a.lengths[s] = 0;
    }
}

// What request i asks for: pages for the entries [first, behind) of its row. part: of append, the entry of a page that has tokens and gets more, -1 for
// none. False: the request cannot be met at all.
struct Want {
    int row, first, behind, part;
};
__device__ __forceinline__ bool want_of(const PagesArgs& a, int i, bool fork, Want& w) {
    w = Want{a.dst[i], 0, 0, -1};
    if (!is_row(a, w.row)) return false;
    if (fork) {
        const int s = a.src[i];
        if (!is_row(a, s)) return false;
        const int len = length_of(a, s);
        w.first = len / a.page;
        w.behind = w.first + (len % a.page != 0 && is_page(a, a.table[static_cast<long long>(s) * a.max_pages + w.first]));
        return true;
    }
    const long long len = length_of(a, w.row), more = a.tokens ? a.tokens[i] : a.every;
    if (more < 0) return false;
    const long long have = (len + a.page - 1) / a.page, want = (len + more + a.page - 1) / a.page;
    if (want > a.max_pages) return false;
    w.first = static_cast<int>(have);
    w.behind = static_cast<int>(want);
    if (more > 0 && len % a.page != 0) w.part = w.first - 1;
    return true;
}

// append: a row whose length was lowered still names the pages behind it. They are its own, and come first. False: other rows name a page too that
// the request's tokens would get to, the row's last one or one behind it (its length was lowered to before its fork), and nothing is written
// there. A row that was never shortened ends at its first entry. Each lane has a request (can: one that may be met); from its second page on the
// warp looks at 32 entries together.
__device__ __forceinline__ bool keep_own(const PagesArgs& a, bool can, Want& w) {
    const int lane = threadIdx.x & 31;
    auto names = [&](int row, int i) {  // entries that name this one's page; 0 where it is none
        const int p = a.table[static_cast<long long>(row) * a.max_pages + i];
        return is_page(a, p) ? __ldcg(a.refs + p) : 0;
    };
    bool shared = can && w.part >= 0 && names(w.row, w.part) > 1, on = false;
    if (can && !shared && w.first < w.behind) {
        const int n = names(w.row, w.first);
        shared = n > 1;
        on = n == 1 && ++w.first < w.behind;
    }
    for (unsigned left = __ballot_sync(0xffffffffu, on); left; left &= left - 1) {
        const int l = __ffs(left) - 1, row = __shfl_sync(0xffffffffu, w.row, l), behind = __shfl_sync(0xffffffffu, w.behind, l);
        int at = __shfl_sync(0xffffffffu, w.first, l), n = 1;
        for (; at < behind && n == 1; at += 32) {  // n: of the first entry that is not the row's own
            const int here = at + lane < behind ? names(row, at + lane) : 0;
            const unsigned others = __ballot_sync(0xffffffffu, here != 1);
            if (!others) continue;
            const int first = __ffs(others) - 1;
            n = __shfl_sync(0xffffffffu, here, first);
            at += first - 32;
        }
        if (lane == l) {
            w.first = min(at, behind);
            shared = n > 1;
        }
    }
    return can && !shared;
}

// What becomes of a request is settled by the first pass and kept in ok meanwhile, since later passes change what it was settled by: the number behind its
// last page among all that are asked for (kMost for more: there are fewer pages), and whether it takes no page, or cannot be met.
constexpr int kMost = (1 << 30) - 1, kNoPage = 1 << 30, kRefused = INT_MIN;
__device__ __forceinline__ bool is_met(int settled, int free) { return !(settled & kRefused) && (settled & kNoPage || (settled & kMost) <= free); }

// Inclusive sum over the block's threads in order; total: of all of them.
__device__ __forceinline__ int block_scan(int v, int* red, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += o;
    }
    __syncthreads();  // the last call's readers
    if (lane == 31) red[warp] = v;
    __syncthreads();
    int t = red[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, t, d);
        if (lane >= d) t += o;
    }
    total = __shfl_sync(0xffffffffu, t, 31);
    const int before = __shfl_sync(0xffffffffu, t, (warp + 31) & 31);
    return v + (warp ? before : 0);
}

// fork: dst[i] becomes a row like src[i]; append: room for tokens behind row dst[i]. Requests' pages are numbered in order, the free pages too, and
// page number r goes to the request that holds number r. A request whose last number is past the free pages gets none.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) pages_kernel(const __grid_constant__ PagesArgs a, bool fork) {
    __shared__ int red[32], free_here;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank()), tid = threadIdx.x;
    const long long first = rank * kThreads + tid, step = kCluster * kThreads;
    if (fork) {
        release_rows(a, first, step);
        __threadfence();
        cluster.sync();
    }
    // the requests' numbers (first block), and each block's share of the pages: those that are free
    const int share = (a.n_pages + kCluster - 1) / kCluster, lo = min(rank * share, a.n_pages), hi = min(lo + share, a.n_pages);
    if (rank == 0) {
        int before = 0;
        for (int i0 = 0; i0 < a.n; i0 += kThreads) {
            Want w{};
            const int i = i0 + tid;
            bool can = i < a.n && want_of(a, i, fork, w);
            if (!fork) can = keep_own(a, can, w);
            const int pages = can ? w.behind - w.first : 0;
            int total;
            const int end = block_scan(pages, red, total) + before;
            if (i < a.n) a.ok[i] = min(end, kMost) | (can ? pages ? 0 : kNoPage : kRefused);
            before += total;
        }
    }
    int count = 0;
    for (int p = lo + tid; p < hi; p += kThreads) count += __ldcg(a.refs + p) <= 0;
    int here;
    block_scan(count, red, here);
    if (tid == 0) free_here = here;
    __threadfence();
    cluster.sync();
    int before = 0, free = 0;
    for (int r = 0; r < kCluster; ++r) {
        const int n = *cluster.map_shared_rank(&free_here, r);
        if (r < rank) before += n;
        free += n;
    }
    const int asked = __ldcg(a.ok + a.n - 1) & kMost;
    // the requests' answers
    for (int p0 = lo; p0 < hi && before < asked; p0 += kThreads) {
        const int p = p0 + tid;
        const bool is_free = p < hi && __ldcg(a.refs + p) <= 0;
        int total;
        const int number = block_scan(is_free, red, total) + before - 1;
        before += total;
        if (!is_free || number >= asked) continue;
        int l = 0, h = a.n - 1;  // the first request that ends behind this number
        while (l < h) {
            const int m = (l + h) / 2;
            if ((__ldcg(a.ok + m) & kMost) > number) h = m; else l = m + 1;
        }
        const int end = __ldcg(a.ok + l) & kMost;
        if (end > free) continue;
        Want w;
        want_of(a, l, fork, w);
        a.table[static_cast<long long>(w.row) * a.max_pages + w.behind - (end - number)] = p;
        a.refs[p] = 1;
        if (fork) a.copy_to[l] = p;
    }
    __threadfence();
    cluster.sync();
    if (fork) {  // the full pages are shared
        const long long entries = static_cast<long long>(a.n) * a.max_pages;
        for (long long e = first; e < entries; e += step) {
            const int i = static_cast<int>(e / a.max_pages), j = static_cast<int>(e - static_cast<long long>(i) * a.max_pages);
            Want w;
            if (!is_met(__ldcg(a.ok + i), free) || !want_of(a, i, true, w) || j >= w.first) continue;
            const int p = a.table[static_cast<long long>(a.src[i]) * a.max_pages + j];
            if (!is_page(a, p)) continue;
            a.table[static_cast<long long>(w.row) * a.max_pages + j] = p;
            atomicAdd(a.refs + p, 1);
        }
        cluster.sync();  // ok holds what was settled up to here: other threads look there for what their entries' requests get
    }
    for (long long i = first; i < a.n; i += step) {
        Want w;
        const bool can = is_met(__ldcg(a.ok + i), free) && want_of(a, static_cast<int>(i), fork, w);
        long long len = can ? length_of(a, fork ? a.src[i] : w.row) : -1;
        if (fork) {
            const bool copied = can && w.behind > w.first;
            a.copy_from[i] = copied ? a.table[static_cast<long long>(a.src[i]) * a.max_pages + w.first] : -1;
            if (!copied) a.copy_to[i] = -1;
        } else if (can) {
            len += a.tokens ? a.tokens[i] : a.every;
        }
        a.ok[i] = static_cast<int>(len);
    }
    cluster.sync();  // no length is set before the last one has been read
    for (long long i = first; i < a.n; i += step) {
        const int len = a.ok[i];
        const int row = a.dst[i];
        if (len >= 0) a.lengths[row] = len;
        a.ok[i] = len >= 0;
        if (a.active) a.active[i] = len >= 0 ? row : -1;
    }
}

__global__ void __launch_bounds__(256) release_kernel(const __grid_constant__ PagesArgs a) {
    release_rows(a, blockIdx.x * 256LL + threadIdx.x, gridDim.x * 256LL);
}

// ---------------------------------------------------------------------------------------------------------------------------------

constexpr int kPools = 32;      // pools of one launch
constexpr int kPiece = 32768;   // bytes that a block copies at a time
constexpr int kCopyThreads = 256;

struct CopyArgs {
    unsigned char* pool[kPools];
    long long bytes[kPools];
    int pieces[kPools + 1];  // pieces of a row in the pools before
    const int *from, *to;
    int n, n_rows, pools;
};

template <typename V>
__device__ __forceinline__ void copy_piece(unsigned char* to, const unsigned char* from, int bytes) {
    constexpr int kFlight = 8;
    const int n = bytes / static_cast<int>(sizeof(V));
    const V* s = reinterpret_cast<const V*>(from);
    V* d = reinterpret_cast<V*>(to);
    for (int i0 = threadIdx.x; i0 < n; i0 += kFlight * kCopyThreads) {
        V v[kFlight];
#pragma unroll
        for (int u = 0; u < kFlight; ++u)
            if (i0 + u * kCopyThreads < n) v[u] = __ldcs(s + i0 + u * kCopyThreads);
#pragma unroll
        for (int u = 0; u < kFlight; ++u)
            if (i0 + u * kCopyThreads < n) __stcs(d + i0 + u * kCopyThreads, v[u]);
    }
}

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyArgs a) {
    const long long units = static_cast<long long>(a.pieces[a.pools]) * a.n;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const int piece = static_cast<int>(u / a.n), i = static_cast<int>(u - static_cast<long long>(piece) * a.n);
        const int from = __ldg(a.from + i), to = __ldg(a.to + i);
        if (from < 0 || from >= a.n_rows || to < 0 || to >= a.n_rows || from == to) continue;
        int k = 0;
        while (a.pieces[k + 1] <= piece) ++k;
        const long long row = a.bytes[k], at = static_cast<long long>(piece - a.pieces[k]) * kPiece;
        const int bytes = static_cast<int>(row - at < kPiece ? row - at : kPiece);
        unsigned char* d = a.pool[k] + to * row + at;
        const unsigned char* s = a.pool[k] + from * row + at;
        const unsigned odd = static_cast<unsigned>(reinterpret_cast<uintptr_t>(a.pool[k])) | static_cast<unsigned>(row);
        if (!(odd & 15)) copy_piece<uint4>(d, s, bytes);
        else if (!(odd & 3)) copy_piece<unsigned>(d, s, bytes);
        else copy_piece<unsigned char>(d, s, bytes);
    }
}

gdn2_status pages_check(const PagesArgs& a) {
    if (a.n < 0 || a.n_slots < 0 || a.n_pages < 0 || a.max_pages <= 0 || a.page <= 0) return GDN2_ERR_INVALID_ARG;
    if (a.page > 65536 || static_cast<long long>(a.max_pages) * a.page >= (1LL << 30) || a.n_pages >= kMost || a.n >= (1 << 24) ||
        static_cast<long long>(a.n) * a.max_pages >= (1LL << 31) - 1)
        return GDN2_ERR_UNSUPPORTED;
    if (a.n == 0) return GDN2_OK;
    if (!a.table || !a.lengths || !a.refs || !a.dst) return GDN2_ERR_INVALID_ARG;
    for (const void* p : {(const void*)a.table, (const void*)a.lengths, (const void*)a.refs, (const void*)a.src, (const void*)a.dst,
                          (const void*)a.tokens, (const void*)a.copy_from, (const void*)a.copy_to, (const void*)a.ok, (const void*)a.active})
        if (!aligned_to(p, 4)) return GDN2_ERR_MISALIGNED;
    return GDN2_OK;
}

}  // namespace
}  // namespace gdn2

using namespace gdn2;

extern "C" {

gdn2_status gdn2_pages_fork_active(int32_t* table, int32_t* lengths, int32_t* refs, const int32_t* src, const int32_t* dst,
                                   int32_t* copy_from, int32_t* copy_to, int32_t* ok, int32_t* active, int n, int n_slots, int n_pages,
                                   int max_pages, int page, void* stream) {
    PagesArgs a{table, lengths, refs, src, dst, nullptr, copy_from, copy_to, ok, active, n, 0, n_slots, n_pages, max_pages, page};
    const gdn2_status st = pages_check(a);
    if (st != GDN2_OK || n == 0) return st;
    if (!src || !copy_from || !copy_to || !ok) return GDN2_ERR_INVALID_ARG;
    pages_kernel<<<kCluster, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(a, true);
    return cudaGetLastError() == cudaSuccess ? GDN2_OK : GDN2_ERR_CUDA;
}

gdn2_status gdn2_pages_fork(int32_t* table, int32_t* lengths, int32_t* refs, const int32_t* src, const int32_t* dst, int32_t* copy_from,
                            int32_t* copy_to, int32_t* ok, int n, int n_slots, int n_pages, int max_pages, int page, void* stream) {
    return gdn2_pages_fork_active(table, lengths, refs, src, dst, copy_from, copy_to, ok, nullptr, n, n_slots, n_pages, max_pages, page, stream);
}

gdn2_status gdn2_pages_append_active(int32_t* table, int32_t* lengths, int32_t* refs, const int32_t* slots, const int32_t* tokens, int every,
                                     int32_t* ok, int32_t* active, int n, int n_slots, int n_pages, int max_pages, int page, void* stream) {
    PagesArgs a{table, lengths, refs, nullptr, slots, tokens, nullptr, nullptr, ok, active, n, every, n_slots, n_pages, max_pages, page};
    const gdn2_status st = pages_check(a);
    if (st != GDN2_OK) return st;
    if (!tokens && every < 0) return GDN2_ERR_INVALID_ARG;
    if (n == 0) return GDN2_OK;
    if (!ok) return GDN2_ERR_INVALID_ARG;
    pages_kernel<<<kCluster, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(a, false);
    return cudaGetLastError() == cudaSuccess ? GDN2_OK : GDN2_ERR_CUDA;
}

gdn2_status gdn2_pages_append(int32_t* table, int32_t* lengths, int32_t* refs, const int32_t* slots, const int32_t* tokens, int every,
                              int32_t* ok, int n, int n_slots, int n_pages, int max_pages, int page, void* stream) {
    return gdn2_pages_append_active(table, lengths, refs, slots, tokens, every, ok, nullptr, n, n_slots, n_pages, max_pages, page, stream);
}

gdn2_status gdn2_pages_release(int32_t* table, int32_t* lengths, int32_t* refs, const int32_t* slots, int n, int n_slots, int n_pages,
                               int max_pages, void* stream) {
    PagesArgs a{table, lengths, refs, nullptr, slots, nullptr, nullptr, nullptr, nullptr, nullptr, n, 0, n_slots, n_pages, max_pages, 1};
    const gdn2_status st = pages_check(a);
    if (st != GDN2_OK || n == 0) return st;
    const long long blocks = (static_cast<long long>(n) * max_pages + 255) / 256;
    release_kernel<<<static_cast<unsigned>(blocks < 1216 ? blocks : 1216), 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return cudaGetLastError() == cudaSuccess ? GDN2_OK : GDN2_ERR_CUDA;
}

gdn2_status gdn2_pages_copy(void* const* pools, const long long* row_bytes, int n_pools, const int32_t* from, const int32_t* to, int n,
                            int n_rows, void* stream) {
    if (n_pools < 0 || n < 0 || n_rows < 0 || (n_pools && (!pools || !row_bytes))) return GDN2_ERR_INVALID_ARG;
    for (int k = 0; k < n_pools; ++k) {
        if (row_bytes[k] < 0 || (n_rows && row_bytes[k] && !pools[k])) return GDN2_ERR_INVALID_ARG;
        if (row_bytes[k] >= (1LL << 40)) return GDN2_ERR_UNSUPPORTED;
    }
    if (n == 0 || n_rows == 0 || n_pools == 0) return GDN2_OK;
    if (!from || !to) return GDN2_ERR_INVALID_ARG;
    if (!aligned_to(from, 4) || !aligned_to(to, 4)) return GDN2_ERR_MISALIGNED;
    for (int k0 = 0; k0 < n_pools; k0 += kPools) {
        CopyArgs a{};
        a.from = from;
        a.to = to;
        a.n = n;
        a.n_rows = n_rows;
        a.pools = n_pools - k0 < kPools ? n_pools - k0 : kPools;
        long long pieces = 0;
        for (int k = 0; k < a.pools; ++k) {
            a.pool[k] = static_cast<unsigned char*>(pools[k0 + k]);
            a.bytes[k] = row_bytes[k0 + k];
            pieces += (a.bytes[k] + kPiece - 1) / kPiece;
            if (pieces >= (1LL << 31)) return GDN2_ERR_UNSUPPORTED;
            a.pieces[k + 1] = static_cast<int>(pieces);
        }
        // a block per piece: 64 x 2 rows of 2 MB take 80 us (79 at the copy rate), 90 with four resident blocks per SM that walk over them
        const long long units = pieces * n, most = 1 << 20;
        if (units == 0) continue;
        copy_kernel<<<static_cast<unsigned>(units < most ? units : most), kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
        if (cudaGetLastError() != cudaSuccess) return GDN2_ERR_CUDA;
    }
    return GDN2_OK;
}

}  // extern "C"
