// sv_tree_attention.cu -- sv_tree_attention: the drafted nodes' keys and
// values go to a paged cache, and every node attends to the cached prefix and
// to its own ancestors.
//
// tree_prepare_kernel checks each request, works out every node's ancestor
// set and writes the new rows; tree_attend_kernel (sv_tree_attend.cuh) does
// the attention and tree_join_kernel joins what it had to cut.
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "sv_tree.h"
#include "sv_tree_attend.cuh"
#include "sv_tree_common.cuh"

namespace sv {
namespace {

constexpr int kPrepThreads = 256;
static_assert(kPrepThreads >= SV_MAX_NODES, "one thread per node");

// Whether one of two packed values is infinite or NaN (all exponent bits set).
template <typename T>
__device__ __forceinline__ bool not_finite(uint32_t w) {
    constexpr uint32_t e = Half<T>::kExp2;
    return (w & e & 0xffff0000u) == (e & 0xffff0000u) || (w & e & 0xffffu) == (e & 0xffffu);
}

// Checks request blockIdx.x, finds each node's ancestors by pointer jumping
// (log2 rounds), and copies its new rows; blockIdx.y shares out the copies.
template <typename T>
__global__ void __launch_bounds__(kPrepThreads) tree_prepare_kernel(const AttnParams a) {
    __shared__ uint32_t bits[2][SV_MAX_NODES][kMaskWords];
    __shared__ int32_t up[2][SV_MAX_NODES];
    const int b = blockIdx.x, tid = threadIdx.x, N = a.N;
    grid_dependency_wait();
    grid_launch_dependents();
    const int len = a.lens[b], count = a.counts ? a.counts[b] : N;
    const bool count_ok = count >= 0 && count <= N;
    const int64_t rows = int64_t(len) + count;
    bool bad = !count_ok || len < 0 || rows > int64_t(a.max_pages) * a.page_size;
    if (!bad && tid < count) {
        const int p = tid == 0 ? 0 : a.parents ? a.parents[int64_t(b) * N + tid] : tid - 1;
        if (p < 0 || (tid > 0 && p >= tid)) bad = true;
        up[0][tid] = bad ? 0 : p;
        for (int w = 0; w < kMaskWords; ++w) bits[0][tid][w] = tid / 32 == w ? 1u << (tid % 32) : 0u;
    }
    if (!bad) {
        const int n = static_cast<int>((rows + a.page_size - 1) / a.page_size);
        for (int i = tid; i < n; i += kPrepThreads) {
            const int id = a.table[b * a.table_stride + i];
            if (id < 0 || id >= a.pages) bad = true;
        }
    }
    bad = __syncthreads_or(bad);
    const int words = a.heads * a.head_dim / 8;  // 16-byte words of a key row
    if (bad) {
        if (blockIdx.y == 0) {
            if (tid == 0) a.ok[b] = 0;
            if (count_ok) {
                const int per = a.q_heads * a.head_dim / 8;
                const uint4 nan{Half<T>::kNan2, Half<T>::kNan2, Half<T>::kNan2, Half<T>::kNan2};
                for (int64_t i = tid; i < int64_t(count) * per; i += kPrepThreads) {
                    const int w = static_cast<int>(i % per) * 8;
                    *reinterpret_cast<uint4*>(a.out + b * a.ob + (i / per) * a.on + (w / a.head_dim) * a.oh +
                                              (w % a.head_dim) * 2) = nan;
                }
            }
        }
        return;
    }
    if (blockIdx.y == 0) {
        int cur = 0;
        for (int reach = 1; reach < count; reach *= 2) {
            if (tid < count) {
                const int p = up[cur][tid];
                for (int w = 0; w < kMaskWords; ++w) bits[cur ^ 1][tid][w] = bits[cur][tid][w] | bits[cur][p][w];
                up[cur ^ 1][tid] = up[cur][p];
            }
            cur ^= 1;
            __syncthreads();
        }
        if (tid < count)
            for (int w = 0; w < kMaskWords; ++w)
                a.masks[(int64_t(b) * N + tid) * kMaskWords + w] = bits[cur][tid][w];
        if (tid == 0) a.ok[b] = 1;
    }
    // one warp per node
    const int lane = tid & 31, warps = gridDim.y * (kPrepThreads / 32);
    for (int n = blockIdx.y * (kPrepThreads / 32) + tid / 32; n < count; n += warps) {
        const int t = len + n;
        const int64_t page = a.table[b * a.table_stride + t / a.page_size];
        const int64_t to = page * a.page_stride + (t % a.page_size) * a.row_stride;
        bool odd = false;
        for (int i = lane; i < words; i += 32) {
            const int w = i * 8, h = w / a.head_dim, d = (w % a.head_dim) * 2;
            const uint4 k = *reinterpret_cast<const uint4*>(a.k + b * a.kb + n * a.kn + h * a.kh + d);
            const uint4 v = *reinterpret_cast<const uint4*>(a.v + b * a.vb + n * a.vn + h * a.vh + d);
            *reinterpret_cast<uint4*>(a.kc + to + h * a.head_stride + d) = k;
            *reinterpret_cast<uint4*>(a.vc + to + h * a.head_stride + d) = v;
            odd |= not_finite<T>(v.x) || not_finite<T>(v.y) || not_finite<T>(v.z) || not_finite<T>(v.w);
        }
        odd = __any_sync(0xffffffffu, odd);
        if (lane == 0) a.odd[int64_t(b) * N + n] = odd;
    }
}

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

sv_status attention_ok(const sv_tree_attention_shape* s, const sv_cache* c) {
    if (!s || !c || s->B < 0 || s->N < 1 || s->q_heads < 1 || s->max_pages < 1) return SV_EINVAL;
    if (c->pages < 1 || c->page_size < 1 || c->heads < 1 || c->head_dim < 1) return SV_EINVAL;
    if (s->q_heads % c->heads != 0 || (s->table_stride != 0 && s->table_stride < s->max_pages)) return SV_EINVAL;
    const int64_t strides = c->page_stride | c->row_stride | c->head_stride | s->q_stride_b | s->q_stride_n |
                            s->q_stride_h | s->k_stride_b | s->k_stride_n | s->k_stride_h | s->v_stride_b |
                            s->v_stride_n | s->v_stride_h | s->o_stride_b | s->o_stride_n | s->o_stride_h;
    if (strides < 0 || strides % 8 != 0) return SV_EINVAL;
    if (c->dtype != SV_BF16 && c->dtype != SV_F16) return SV_EUNSUPPORTED;
    if (c->layers != 1 || s->N > SV_MAX_NODES || s->q_heads / c->heads > 64) return SV_EUNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128) return SV_EUNSUPPORTED;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) return SV_EUNSUPPORTED;
    if (int64_t(s->max_pages) * c->page_size > 0x40000000 || s->B > 0xffff || s->q_heads > 0x4000)
        return SV_EUNSUPPORTED;
    // tiles of one request, and units of the batch, are counted in 32 bits
    const int64_t units = int64_t(c->heads) * ((int64_t(s->N) * (s->q_heads / c->heads) + kUnitRows - 1) / kUnitRows);
    if (units * (int64_t(s->max_pages) * c->page_size / kTile + 1) > 0x7fffffff || units * s->B > 0x7fffffff)
        return SV_EUNSUPPORTED;
    return SV_OK;
}

// The workspace: what the preparation finds, then the parts of cut units.
struct AttnWorkspace {
    size_t ok, masks, odd, ml, o, total;
    int slot_rows;
};

AttnWorkspace workspace_layout(const sv_tree_attention_shape& s, const sv_cache& c) {
    AttnWorkspace w{};
    const int64_t most = int64_t(s.N) * (s.q_heads / c.heads);
    w.slot_rows = static_cast<int>(most < kUnitRows ? (most + 31) / 32 * 32 : kUnitRows);
    const size_t slots = 2 * size_t(kAttendMaxCtas) * w.slot_rows;
    size_t at = 0;
    w.ok = at;  at += align256(size_t(s.B) * 4);
    w.masks = at; at += align256(size_t(s.B) * s.N * kMaskWords * 4);
    w.odd = at;   at += align256(size_t(s.B) * s.N * 4);
    w.ml = at;    at += align256(slots * sizeof(float2));
    w.o = at;     at += align256(slots * c.head_dim * 4);
    w.total = at;
    return w;
}

// A cache as a 4-d tensor (column, head, row of a page, page); a box is the
// 64 columns of one head in one page, 128-byte swizzled.
bool cache_map(CUtensorMap* map, void* base, const sv_cache& c) {
    using Encode = decltype(&cuTensorMapEncodeTiled);
    static const Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<Encode>(f);
    }();
    if (!encode) return false;
    const cuuint64_t dims[4] = {cuuint64_t(c.head_dim), cuuint64_t(c.heads), cuuint64_t(c.page_size),
                                cuuint64_t(c.pages)};
    const cuuint64_t some = cuuint64_t(c.head_dim) * 2;  // the stride of a dimension of size one is not used
    const cuuint64_t strides[3] = {c.heads > 1 ? cuuint64_t(c.head_stride) * 2 : some,
                                   c.page_size > 1 ? cuuint64_t(c.row_stride) * 2 : some,
                                   c.pages > 1 ? cuuint64_t(c.page_stride) * 2 : some};
    const cuuint32_t box[4] = {64, 1, cuuint32_t(c.page_size), 1}, one[4] = {1, 1, 1, 1};
    return encode(map, c.dtype == SV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, base,
                  dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D>
cudaError_t run(const AttnParams& a, const sv_cache& c, cudaStream_t st) {
    TreeDevice dev;
    cudaError_t e = tree_device(&dev);
    if (e != cudaSuccess) return e;
    CUtensorMap kmap, vmap;
    if (!cache_map(&kmap, c.k, c) || !cache_map(&vmap, c.v, c)) return cudaErrorInvalidValue;
    const int splits = (a.N + kPrepThreads / 32 - 1) / (kPrepThreads / 32);
    e = launch_dependent(tree_prepare_kernel<T>, dim3(a.B, splits), kPrepThreads, 0, 1, st, a);
    if (e != cudaSuccess) return e;
    constexpr auto k = &tree_attend_kernel<T, D>;
    e = set_once<k>(dev, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(AttendSmem<D>::bytes()));
    if (e != cudaSuccess) return e;
    const int ctas = dev.sm_count < kAttendMaxCtas ? dev.sm_count : kAttendMaxCtas;
    e = launch_dependent(k, dim3(ctas), kAttendThreads, AttendSmem<D>::bytes(), 1, st, a, kmap, vmap);
    if (e != cudaSuccess) return e;
    const int units = a.heads * ((a.N * a.group + kUnitRows - 1) / kUnitRows);
    dim3 grid(static_cast<unsigned>(a.B * units), a.slot_rows / 32);
    constexpr int kCols = D / 4 / kJoinWarps;  // of a warp, where a CTA has all columns
    // Few units: their many parts are spread over more CTAs (two requests with one key head over
    // 12600 rows, 50 parts each: 72 us without, 27 with; many units, which have few parts: 93 us
    // for a batch of chains without, 100 with, 191 and 197 for long trees).
    if (int64_t(grid.x) * grid.y <= 2 * ctas) {
        grid.z = kCols;
        return launch_dependent(tree_join_kernel<T, D, 1>, grid, kJoinThreads, 0, 1, st, a, units, ctas);
    }
    return launch_dependent(tree_join_kernel<T, D, kCols>, grid, kJoinThreads, 0, 1, st, a, units, ctas);
}

}  // namespace
}  // namespace sv

extern "C" size_t sv_tree_attention_workspace_bytes(const sv_tree_attention_shape* shape, const sv_cache* cache) {
    return sv::attention_ok(shape, cache) == SV_OK ? sv::workspace_layout(*shape, *cache).total : 0;
}

extern "C" sv_status sv_tree_attention(const sv_tree_attention_shape* s, const sv_cache* cache, const void* q,
                                       const void* k, const void* v, const int32_t* page_table, const int32_t* lens,
                                       const int32_t* parents, const int32_t* counts, float scale, void* out,
                                       void* workspace, size_t workspace_bytes, void* stream) {
    using namespace sv;
    if (const sv_status why = attention_ok(s, cache); why != SV_OK) return why;
    if (s->B == 0) return SV_OK;  // (an empty tensor's pointer may be null)
    if (!q || !k || !v || !page_table || !lens || !out || !workspace || !cache->k || !cache->v) return SV_EINVAL;
    if (!std::isfinite(scale) || workspace_bytes < workspace_layout(*s, *cache).total) return SV_EINVAL;
    for (const void* p : {q, k, v, static_cast<const void*>(out), static_cast<const void*>(cache->k),
                          static_cast<const void*>(cache->v), static_cast<const void*>(workspace)})
        if (!tree_aligned16(p)) return SV_EINVAL;
    const AttnWorkspace w = workspace_layout(*s, *cache);
    char* ws = static_cast<char*>(workspace);
    AttnParams a{static_cast<char*>(cache->k), static_cast<char*>(cache->v), cache->page_stride * 2,
                 cache->row_stride * 2, cache->head_stride * 2, cache->pages, cache->page_size, cache->heads,
                 cache->head_dim, s->B, s->N, s->q_heads, s->q_heads / cache->heads, s->max_pages,
                 s->table_stride ? s->table_stride : s->max_pages,
                 s->q_stride_b * 2, s->q_stride_n * 2, s->q_stride_h * 2, s->k_stride_b * 2, s->k_stride_n * 2,
                 s->k_stride_h * 2, s->v_stride_b * 2, s->v_stride_n * 2, s->v_stride_h * 2, s->o_stride_b * 2,
                 s->o_stride_n * 2, s->o_stride_h * 2, static_cast<const char*>(q), static_cast<const char*>(k),
                 static_cast<const char*>(v), static_cast<char*>(out), page_table, lens, parents, counts, scale,
                 w.slot_rows, reinterpret_cast<int32_t*>(ws + w.ok), reinterpret_cast<uint32_t*>(ws + w.masks),
                 reinterpret_cast<int32_t*>(ws + w.odd), reinterpret_cast<float2*>(ws + w.ml),
                 reinterpret_cast<float4*>(ws + w.o)};
    auto st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (cache->dtype == SV_BF16)
        e = cache->head_dim == 64 ? run<__nv_bfloat16, 64>(a, *cache, st) : run<__nv_bfloat16, 128>(a, *cache, st);
    else
        e = cache->head_dim == 64 ? run<__half, 64>(a, *cache, st) : run<__half, 128>(a, *cache, st);
    return e == cudaSuccess ? SV_OK : SV_ECUDA;
}
