// sv_cache.cu -- the paged cache's upkeep: sv_cache_resize, sv_cache_fork and
// sv_cache_commit.
//
// Page accounting is one kernel of one thread-block cluster: give back, count
// the free pages, hand them out in increasing order of their id.  The answer
// does not depend on the order of any atomic: reference counts are sums, and
// a page's place in the hand-out is its rank among the free pages.  The
// copies are plain streams of 16-byte words, bound by memory.
//
// Measured on the device.  Page accounting of 64 slots 7 to 10 us, a chain of
// dependent loads and barriers; compaction of 64 trees through 32 layers (23
// MB) 12 us; 64 forks through 32 layers, 111 MB: 12 us of accounting and 22 us
// of copies, 5 TB/s.  The host's part of a call from Python is about 9 us, so
// that eager steps are bound by it and captured ones are not: resize, commit
// and resize take 35 us eagerly, 23 us (64 trees) and 10 us (2 trees) replayed.
#include <cstdint>

#include <cuda_runtime.h>

#include "sv_tree.h"
#include "sv_tree_common.cuh"

namespace sv {
namespace {

constexpr int kPoolThreads = 1024;
constexpr int kPoolWarps = kPoolThreads / 32;
constexpr int kPoolMaxCluster = 8;

struct PoolShared {
    int32_t base[SV_MAX_SLOTS + 1];  // pages wanted before each slot (or fork)
    int32_t warp[kPoolWarps];
    int64_t free_of[kPoolMaxCluster];  // free pages of each CTA's share
    uint32_t src_set[SV_MAX_SLOTS / 32], dst_set[SV_MAX_SLOTS / 32], dst_twice[SV_MAX_SLOTS / 32];
};

// Exclusive scan of one value per thread over the block; *total: the sum.
__device__ int block_scan(int v, int* total, int32_t* warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    __syncthreads();  // the sums of the call before are read
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int w = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += x;
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    *total = warp_sums[kPoolWarps - 1];
    return incl - v + (warp ? warp_sums[warp - 1] : 0);
}

// Pages that a slot's row lists, or -1 when the row is not valid (an entry
// outside [-1, pages), or a page behind a -1).  One warp.
__device__ int held_pages(const int32_t* row, int max_pages, int pages) {
    const int lane = threadIdx.x & 31;
    int held = 0;
    bool over = false, bad = false;
    for (int i0 = 0; i0 < max_pages; i0 += 32) {
        const int i = i0 + lane;
        const int e = i < max_pages ? row[i] : -1;
        const uint32_t has = __ballot_sync(0xffffffffu, e >= 0);
        bad |= __any_sync(0xffffffffu, e < -1 || e >= pages);
        const int n = __popc(has);
        bad |= (over && n > 0) || has != (n == 32 ? 0xffffffffu : (1u << n) - 1u);
        over |= n < 32;
        held += n;
    }
    return bad ? -1 : held;
}

__device__ void give_back(int32_t* row, int from, int to, int32_t* refcount) {
    for (int i = from + static_cast<int>(threadIdx.x & 31); i < to; i += 32) {
        atomicSub(refcount + row[i], 1);
        row[i] = -1;
    }
}

// base[i] = wants before entry i, base[n] = all; wants(i) from the statuses.
template <typename Wants>
__device__ int scan_wants(PoolShared& sh, int n, Wants wants) {
    int all = 0;
    for (int i0 = 0; i0 < n; i0 += kPoolThreads) {
        const int i = i0 + static_cast<int>(threadIdx.x);
        int total;
        const int before = block_scan(i < n ? wants(i) : 0, &total, sh.warp);
        if (i < n) sh.base[i] = all + before;
        all += total;
    }
    if (threadIdx.x == 0) sh.base[n] = all;
    __syncthreads();
    return all;
}

// Free pages of this CTA's share of [0, pages), told to the whole cluster.
// Returns the free pages of all; *before: those of the shares before.
__device__ int64_t count_free(PoolShared& sh, const int32_t* refcount, int pages, int lo, int hi, int64_t* before) {
    const uint32_t rank = cluster_ctarank(), C = cluster_nctarank();
    int n = 0;
    for (int p = lo + static_cast<int>(threadIdx.x); p < hi; p += kPoolThreads) n += __ldcg(refcount + p) == 0;
    int total;
    block_scan(n, &total, sh.warp);
    if (threadIdx.x < C) st_cluster_u64(&sh.free_of[rank], threadIdx.x, static_cast<uint64_t>(total));
    cluster_barrier();
    int64_t all = 0;
    *before = 0;
    for (uint32_t r = 0; r < C; ++r) {
        if (r == rank) *before = all;
        all += sh.free_of[r];
    }
    return all;
}

// Hands the free pages of this CTA's share out: take(entry, k, page) for the
// free page of rank base[entry] + k, as long as ranks are below `limit`.
template <typename Take>
__device__ void hand_out(PoolShared& sh, int32_t* refcount, int lo, int hi, int64_t rank, int64_t limit, int n,
                         Take take) {
    for (int p0 = lo; p0 < hi && rank < limit; p0 += kPoolThreads) {
        const int p = p0 + static_cast<int>(threadIdx.x);
        const bool is_free = p < hi && __ldcg(refcount + p) == 0;
        int total;
        const int64_t r = rank + block_scan(is_free, &total, sh.warp);
        if (is_free && r < limit) {
            int a = 0, z = n;  // the last entry with base <= r
            while (z - a > 1) {
                const int m = (a + z) / 2;
                if (sh.base[m] <= r) a = m;
                else z = m;
            }
            refcount[p] = 1;
            take(a, static_cast<int>(r - sh.base[a]), p);
        }
        rank += total;
    }
}

__device__ void share_of(int pages, int* lo, int* hi) {
    const int C = static_cast<int>(cluster_nctarank()), r = static_cast<int>(cluster_ctarank());
    const int each = (pages + C - 1) / C;
    *lo = r * each < pages ? r * each : pages;
    *hi = *lo + each < pages ? *lo + each : pages;
}

__global__ void __launch_bounds__(kPoolThreads)
resize_kernel(int32_t* table, int64_t stride, int slots, int max_pages, const int32_t* lens, int page_size,
              int32_t* refcount, int pages, int32_t* status) {
    extern __shared__ __align__(16) unsigned char smem[];
    PoolShared& sh = *reinterpret_cast<PoolShared*>(smem);
    const int C = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
    const int warp = rank * kPoolWarps + static_cast<int>(threadIdx.x >> 5);
    const bool lead = (threadIdx.x & 31) == 0;
    grid_dependency_wait();
    auto need_of = [&](int s) { return static_cast<int>((int64_t(lens[s]) + page_size - 1) / page_size); };
    for (int s = warp; s < slots; s += C * kPoolWarps) {
        int32_t* row = table + s * stride;
        const int held = held_pages(row, max_pages, pages);
        const bool ok = lens[s] >= 0 && need_of(s) <= max_pages && held >= 0;
        if (ok && held > need_of(s)) give_back(row, need_of(s), held, refcount);
        if (lead) status[s] = !ok ? -1 : held < need_of(s) ? need_of(s) - held : 0;
    }
    cluster_barrier();
    const int all = scan_wants(sh, slots, [&](int s) {
        const int w = __ldcg(status + s);
        return w > 0 ? w : 0;
    });
    if (all == 0) return;  // the statuses are final
    int lo, hi;
    share_of(pages, &lo, &hi);
    int64_t before;
    const int64_t free_all = count_free(sh, refcount, pages, lo, hi, &before);
    // slots are served in order as long as the running sum fits
    int a = 0, z = slots + 1;
    while (z - a > 1) {
        const int m = (a + z) / 2;
        if (sh.base[m] <= free_all) a = m;
        else z = m;
    }
    const int64_t limit = sh.base[a];
    hand_out(sh, refcount, lo, hi, before, limit, slots, [&](int s, int k, int page) {
        const int wants = sh.base[s + 1] - sh.base[s];
        table[s * stride + need_of(s) - wants + k] = page;
    });
    for (int s = rank * kPoolThreads + static_cast<int>(threadIdx.x); s < slots; s += C * kPoolThreads) {
        const int wants = sh.base[s + 1] - sh.base[s];
        if (wants > 0) status[s] = sh.base[s + 1] <= free_all ? 0 : -1;
    }
}

__global__ void __launch_bounds__(kPoolThreads)
fork_kernel(int32_t* table, int64_t stride, int slots, int max_pages, int32_t* lens, int page_size,
            int32_t* refcount, int pages, const int32_t* src, const int32_t* dst, int forks, int32_t* status) {
    extern __shared__ __align__(16) unsigned char smem[];
    PoolShared& sh = *reinterpret_cast<PoolShared*>(smem);
    const int C = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
    const int warp = rank * kPoolWarps + static_cast<int>(threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < SV_MAX_SLOTS / 32; i += kPoolThreads)
        sh.src_set[i] = sh.dst_set[i] = sh.dst_twice[i] = 0;
    __syncthreads();
    grid_dependency_wait();
    for (int f = threadIdx.x; f < forks; f += kPoolThreads) {
        const int s = src[f], d = dst[f];
        if (s >= 0 && s < slots) atomicOr(&sh.src_set[s / 32], 1u << (s % 32));
        if (d >= 0 && d < slots) {
            const uint32_t bit = 1u << (d % 32);
            if (atomicOr(&sh.dst_set[d / 32], bit) & bit) atomicOr(&sh.dst_twice[d / 32], bit);
        }
    }
    __syncthreads();
    // give back what the destinations hold; status: 1 = wants a page
    for (int f = warp; f < forks; f += C * kPoolWarps) {
        const int s = src[f], d = dst[f];
        int st = -1;
        if (s >= 0 && s < slots && d >= 0 && d < slots && !((sh.dst_twice[d / 32] | sh.src_set[d / 32]) >> (d % 32) & 1u)) {
            const int len = lens[s];
            const int held = held_pages(table + s * stride, max_pages, pages);
            const int old = held_pages(table + d * stride, max_pages, pages);
            const int64_t need = (int64_t(len) + page_size - 1) / page_size;
            if (len >= 0 && need <= held && old >= 0) {
                give_back(table + d * stride, 0, old, refcount);
                st = len % page_size != 0;
            }
        }
        if (lane == 0) status[f] = st;
    }
    cluster_barrier();
    const int all = scan_wants(sh, forks, [&](int f) { return __ldcg(status + f) > 0 ? 1 : 0; });
    int64_t free_all = 0, before = 0;
    int lo = 0, hi = 0;
    if (all > 0) {
        share_of(pages, &lo, &hi);
        free_all = count_free(sh, refcount, pages, lo, hi, &before);
        const int64_t limit = all < free_all ? all : free_all;
        hand_out(sh, refcount, lo, hi, before, limit, forks, [&](int f, int, int page) {
            table[dst[f] * stride + lens[src[f]] / page_size] = page;
        });
    }
    for (int f = warp; f < forks; f += C * kPoolWarps) {
        const int wants = sh.base[f + 1] - sh.base[f];
        // what this warp wrote above, or what the scan has seen
        const int st = wants > 0 ? (sh.base[f + 1] <= free_all ? 0 : -2) : __ldcg(status + f);
        const int s = src[f], d = dst[f];
        __syncwarp();
        if (st == 0) {
            const int full = lens[s] / page_size;
            for (int i = lane; i < full; i += 32) {
                const int page = table[s * stride + i];
                table[d * stride + i] = page;
                atomicAdd(refcount + page, 1);
            }
        }
        if (lane == 0) {
            status[f] = st;
            if (st != -1) lens[d] = st == 0 ? lens[s] : 0;
        }
    }
}

struct CopyParams {
    char* base[2];  // keys, values
    int64_t layer, page, row, head;  // strides in bytes
    int32_t layers, pages, page_size, heads, head_words;  // 16-byte words per head
};

// Byte offset of word w of a row.
__device__ __forceinline__ int64_t word_offset(const CopyParams& c, int w) {
    return (w / c.head_words) * c.head + int64_t(w % c.head_words) * 16;
}

constexpr int kCopyThreads = 256;

// One CTA copies the ragged page of one fork in one layer.  Rows are split
// over the threads in 16-byte words; `solid` pages are one run of bytes.
__global__ void __launch_bounds__(kCopyThreads)
fork_copy_kernel(CopyParams c, const int32_t* table, int64_t stride, const int32_t* lens, const int32_t* src,
                 const int32_t* dst, const int32_t* status, int solid) {
    grid_dependency_wait();
    const int f = blockIdx.x, layer = blockIdx.y;
    if (status[f] != 0) return;
    const int len = lens[src[f]], rag = len % c.page_size;
    if (rag == 0) return;
    const int64_t from = table[src[f] * stride + len / c.page_size], to = table[dst[f] * stride + len / c.page_size];
    const int words = c.heads * c.head_words, n = rag * words;
    for (int kv = 0; kv < 2; ++kv) {
        const char* a = c.base[kv] + layer * c.layer + from * c.page;
        char* b = c.base[kv] + layer * c.layer + to * c.page;
        if (solid) {
            const uint4* x = reinterpret_cast<const uint4*>(a);
            uint4* y = reinterpret_cast<uint4*>(b);
            for (int i = threadIdx.x; i < n; i += 4 * kCopyThreads) {
                uint4 w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (i + k * kCopyThreads < n) w[k] = x[i + k * kCopyThreads];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (i + k * kCopyThreads < n) y[i + k * kCopyThreads] = w[k];
            }
        } else {
            for (int i = threadIdx.x; i < n; i += kCopyThreads) {
                const int64_t at = (i / words) * c.row + word_offset(c, i % words);
                *reinterpret_cast<uint4*>(b + at) = *reinterpret_cast<const uint4*>(a + at);
            }
        }
    }
}

// Compaction.  A thread owns one 16-byte column (layer, keys or values, word
// of the row) of one request and moves it down row by row.  Destinations lie
// below their sources and the sources increase, so a row is always read
// before anything is written over it; eight rows are in flight at a time.
__global__ void __launch_bounds__(kCopyThreads)
commit_kernel(CopyParams c, const int32_t* table, int64_t stride, int max_pages, const int32_t* lens,
              const int32_t* path, int64_t path_stride, int width, int32_t* out_lens) {
    __shared__ int64_t from[SV_MAX_NODES], to[SV_MAX_NODES];
    __shared__ int32_t ids[SV_MAX_NODES], n_sh, first_sh, bad_sh;
    const int b = blockIdx.x;
    if (threadIdx.x == 0) {
        n_sh = first_sh = width;
        bad_sh = 0;
    }
    grid_dependency_wait();
    for (int i = threadIdx.x; i < width; i += kCopyThreads) ids[i] = path[b * path_stride + i];
    const int len = lens[b];
    __syncthreads();
    for (int i = threadIdx.x; i < width; i += kCopyThreads) {
        if (ids[i] < 0) atomicMin(&n_sh, i);
        if (ids[i] != i) atomicMin(&first_sh, i);
    }
    __syncthreads();
    const int n = n_sh, first = first_sh < n ? first_sh : n;
    const int64_t rows = int64_t(max_pages) * c.page_size;
    for (int i = threadIdx.x; i < n; i += kCopyThreads) {
        bool bad = len < 0 || (i > 0 && ids[i] <= ids[i - 1]) || int64_t(len) + ids[i] >= rows;
        if (!bad && i >= first) {
            // increasing from >= 0, so ids[i] >= i (a row that is not is found at its own i)
            const int64_t s = int64_t(len) + ids[i], d = int64_t(len) + i;
            const int ps = d < rows ? table[b * stride + s / c.page_size] : -1;
            const int pd = d < rows ? table[b * stride + d / c.page_size] : -1;
            bad = ps < 0 || ps >= c.pages || pd < 0 || pd >= c.pages;
            from[i] = ps * c.page + (s % c.page_size) * c.row;
            to[i] = pd * c.page + (d % c.page_size) * c.row;
        }
        if (bad) bad_sh = 1;
    }
    if (len < 0) bad_sh = 1;
    __syncthreads();
    if (blockIdx.y == 0 && threadIdx.x == 0) out_lens[b] = bad_sh ? -1 : len + n;
    if (bad_sh) return;
    const int words = c.heads * c.head_words;
    const int64_t column = int64_t(blockIdx.y) * kCopyThreads + threadIdx.x;
    const int64_t plane = column / words;
    if (plane >= 2 * int64_t(c.layers)) return;
    char* at = (plane & 1 ? c.base[1] : c.base[0]) + (plane >> 1) * c.layer + word_offset(c, static_cast<int>(column % words));
    for (int i0 = first; i0 < n; i0 += 8) {
        uint4 w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i0 + k < n) w[k] = *reinterpret_cast<const uint4*>(at + from[i0 + k]);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i0 + k < n) *reinterpret_cast<uint4*>(at + to[i0 + k]) = w[k];
    }
}

bool overlap(const int32_t* a, int64_t n, const int32_t* b, int64_t m) { return a < b + m && b < a + n; }

bool cache_ok(const sv_cache* c, CopyParams* out, sv_status* why) {
    *why = SV_EINVAL;
    if (!c || !c->k || !c->v || c->layers < 1 || c->pages < 1 || c->page_size < 1 || c->heads < 1 ||
        c->head_dim < 1)
        return false;
    if (c->dtype != SV_F32 && c->dtype != SV_BF16 && c->dtype != SV_F16) {
        *why = SV_EUNSUPPORTED;
        return false;
    }
    const int64_t es = c->dtype == SV_F32 ? 4 : 2;
    if (c->layer_stride < 0 || c->page_stride < 0 || c->row_stride < 0 || c->head_stride < 0) return false;
    if (!tree_aligned16(c->k) || !tree_aligned16(c->v) ||
        ((c->layer_stride | c->page_stride | c->row_stride | c->head_stride | int64_t(c->head_dim)) * es) % 16 != 0)
        return false;
    if (int64_t(c->page_size) * c->heads * (c->head_dim * es / 16) > 0x40000000 || c->layers > 65535) {
        *why = SV_EUNSUPPORTED;
        return false;
    }
    *out = CopyParams{{static_cast<char*>(c->k), static_cast<char*>(c->v)},
                      c->layer_stride * es, c->page_stride * es, c->row_stride * es, c->head_stride * es,
                      c->layers, c->pages, c->page_size, c->heads, static_cast<int32_t>(c->head_dim * es / 16)};
    return true;
}

template <auto kKernel, typename... Args>
cudaError_t launch_pool(int64_t entries, int pages, cudaStream_t st, const Args&... args) {
    // one CTA while its 1024 threads see each entry a few times; the cluster's
    // barriers cost about a microsecond
    const int cluster = entries + pages > 16 * kPoolThreads ? kPoolMaxCluster : 1;
    const size_t smem = sizeof(PoolShared);
    TreeDevice dev;
    cudaError_t e = tree_device(&dev);
    if (e == cudaSuccess) e = set_once<kKernel>(dev, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    return launch_dependent(kKernel, dim3(static_cast<unsigned>(cluster)), kPoolThreads, smem, cluster, st, args...);
}

}  // namespace
}  // namespace sv

extern "C" sv_status sv_cache_resize(int32_t* page_table, int64_t table_stride, int32_t slots, int32_t max_pages,
                                     const int32_t* lens, int32_t page_size, int32_t* refcount, int32_t pages,
                                     int32_t* out_status, void* stream) {
    using namespace sv;
    if (table_stride == 0) table_stride = max_pages;
    if (slots < 0 || max_pages < 1 || page_size < 1 || pages < 1 || table_stride < max_pages) return SV_EINVAL;
    if (slots == 0) return SV_OK;
    if (!page_table || !lens || !refcount || !out_status || overlap(lens, slots, out_status, slots)) return SV_EINVAL;
    if (slots > SV_MAX_SLOTS || int64_t(slots) * max_pages > 0x7fffffff) return SV_EUNSUPPORTED;
    const cudaError_t e = launch_pool<&resize_kernel>(int64_t(slots) * max_pages, pages, static_cast<cudaStream_t>(stream),
                                      page_table, table_stride, slots, max_pages, lens, page_size, refcount, pages,
                                      out_status);
    return e == cudaSuccess ? SV_OK : SV_ECUDA;
}

extern "C" sv_status sv_cache_fork(const sv_cache* cache, int32_t* page_table, int64_t table_stride, int32_t slots,
                                   int32_t max_pages, int32_t* lens, int32_t* refcount, const int32_t* src,
                                   const int32_t* dst, int32_t forks, int32_t* out_status, void* stream) {
    using namespace sv;
    CopyParams c;
    sv_status why;
    if (!cache_ok(cache, &c, &why)) return why;
    if (table_stride == 0) table_stride = max_pages;
    if (slots < 1 || max_pages < 1 || forks < 0 || table_stride < max_pages) return SV_EINVAL;
    if (forks == 0) return SV_OK;
    if (!page_table || !lens || !refcount || !src || !dst || !out_status) return SV_EINVAL;
    if (overlap(src, forks, out_status, forks) || overlap(dst, forks, out_status, forks) ||
        overlap(lens, slots, out_status, forks) || overlap(lens, slots, src, forks) || overlap(lens, slots, dst, forks))
        return SV_EINVAL;  // read again after they are written
    if (slots > SV_MAX_SLOTS || forks > SV_MAX_SLOTS) return SV_EUNSUPPORTED;
    auto st = static_cast<cudaStream_t>(stream);
    cudaError_t e = launch_pool<&fork_kernel>(2 * int64_t(forks) * max_pages, c.pages, st, page_table, table_stride,
                                slots, max_pages, lens, c.page_size, refcount, c.pages, src, dst, forks, out_status);
    if (e != cudaSuccess) return SV_ECUDA;
    const int solid = c.head == int64_t(c.head_words) * 16 && c.row == c.heads * c.head;
    e = launch_dependent(fork_copy_kernel, dim3(forks, c.layers), kCopyThreads, 0, 1, st, c,
                         static_cast<const int32_t*>(page_table), table_stride, static_cast<const int32_t*>(lens), src,
                         dst, static_cast<const int32_t*>(out_status), solid);
    return e == cudaSuccess ? SV_OK : SV_ECUDA;
}

extern "C" sv_status sv_cache_commit(const sv_cache* cache, const int32_t* page_table, int64_t table_stride,
                                     int32_t B, int32_t max_pages, const int32_t* lens, const int32_t* path,
                                     int64_t path_stride, int32_t width, int32_t* out_lens, void* stream) {
    using namespace sv;
    CopyParams c;
    sv_status why;
    if (!cache_ok(cache, &c, &why)) return why;
    if (table_stride == 0) table_stride = max_pages;
    if (path_stride == 0) path_stride = width;
    if (B < 0 || max_pages < 1 || width < 1 || table_stride < max_pages || path_stride < width) return SV_EINVAL;
    if (B == 0) return SV_OK;  // (an empty tensor's pointer may be null)
    if (!page_table || !lens || !path || !out_lens) return SV_EINVAL;
    if (overlap(lens, B, out_lens, B)) return SV_EINVAL;  // read by one CTA, written by another
    if (width > SV_MAX_NODES) return SV_EUNSUPPORTED;
    const int64_t columns = 2 * int64_t(c.layers) * c.heads * c.head_words;
    const int64_t y = (columns + kCopyThreads - 1) / kCopyThreads;
    if (y > 65535) return SV_EUNSUPPORTED;
    const cudaError_t e = launch_dependent(commit_kernel, dim3(B, static_cast<unsigned>(y)), kCopyThreads, 0, 1,
                                           static_cast<cudaStream_t>(stream), c, page_table, table_stride, max_pages,
                                           lens, path, path_stride, width, out_lens);
    return e == cudaSuccess ? SV_OK : SV_ECUDA;
}
