// sv_tree_attention.cu -- sv_tree_attention: the drafted nodes' keys and
// values go to a paged cache, and every node attends to the cached prefix and
// to its own ancestors.
//
// Two kernels: tree_prepare_kernel checks each request, works out every
// node's ancestor set and writes the new rows; tree_attend_kernel computes
// one (request, node, query head) per warp.
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "sv_tree.h"
#include "sv_tree_common.cuh"

namespace sv {
namespace {

constexpr int kMaskWords = SV_MAX_NODES / 32;
constexpr int kPrepThreads = 256;
static_assert(kPrepThreads >= SV_MAX_NODES, "one thread per node");

struct AttnParams {
    char* kc;
    char* vc;
    int64_t page_stride, row_stride, head_stride;  // of the cache, in bytes
    int32_t pages, page_size, heads, head_dim;
    int32_t B, N, q_heads, max_pages;
    int64_t table_stride;
    int64_t qb, qn, qh, kb, kn, kh, vb, vn, vh, ob, on, oh;  // in bytes
    const char* q;
    const char* k;
    const char* v;
    char* out;
    const int32_t* table;
    const int32_t* lens;
    const int32_t* parents;
    const int32_t* counts;
    float scale;
    int32_t* rows;     // [B] cached rows lens + count of a request to compute, 0 = none
    uint32_t* masks;   // [B][N][kMaskWords] ancestors-or-self of each node
};

template <typename T>
struct Half;
template <>
struct Half<__nv_bfloat16> {
    __device__ static float to(__nv_bfloat16 x) { return __bfloat162float(x); }
    __device__ static __nv_bfloat16 from(float x) { return __float2bfloat16(x); }
    static constexpr uint32_t kNan2 = 0x7fc07fc0u;
};
template <>
struct Half<__half> {
    __device__ static float to(__half x) { return __half2float(x); }
    __device__ static __half from(float x) { return __float2half(x); }
    static constexpr uint32_t kNan2 = 0x7e007e00u;
};

// Checks request blockIdx.x, finds each node's ancestors by pointer jumping
// (log2 rounds), and copies its new rows; blockIdx.y shares out the copies.
template <typename T>
__global__ void __launch_bounds__(kPrepThreads) tree_prepare_kernel(const AttnParams a) {
    __shared__ uint32_t bits[2][SV_MAX_NODES][kMaskWords];
    __shared__ int32_t up[2][SV_MAX_NODES];
    const int b = blockIdx.x, tid = threadIdx.x, N = a.N;
    grid_dependency_wait();
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
            if (tid == 0) a.rows[b] = 0;
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
        if (tid == 0) a.rows[b] = count > 0 ? static_cast<int>(rows) : 0;
    }
    for (int i = blockIdx.y * kPrepThreads + tid; i < 2 * count * words; i += gridDim.y * kPrepThreads) {
        const bool value = i >= count * words;
        const int j = value ? i - count * words : i;
        const int n = j / words, w = (j % words) * 8, h = w / a.head_dim, d = (w % a.head_dim) * 2;
        const int t = len + n;
        const int64_t page = a.table[b * a.table_stride + t / a.page_size];
        const int64_t to = page * a.page_stride + (t % a.page_size) * a.row_stride + h * a.head_stride + d;
        const char* from = value ? a.v + b * a.vb + n * a.vn + h * a.vh + d : a.k + b * a.kb + n * a.kn + h * a.kh + d;
        *reinterpret_cast<uint4*>((value ? a.vc : a.kc) + to) = *reinterpret_cast<const uint4*>(from);
    }
}

constexpr int kAttendWarps = 8;

// One warp per (request, node, query head), a position at a time; running
// maximum and sum in 32 bits.
template <typename T, int D>
__global__ void __launch_bounds__(kAttendWarps * 32) tree_attend_kernel(const AttnParams a) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t item = int64_t(blockIdx.x) * kAttendWarps + (threadIdx.x >> 5);
    grid_dependency_wait();
    if (item >= int64_t(a.B) * a.N * a.q_heads) return;
    const int h = static_cast<int>(item % a.q_heads), n = static_cast<int>(item / a.q_heads % a.N);
    const int b = static_cast<int>(item / a.q_heads / a.N);
    const int rows = a.rows[b], len = a.lens[b];
    if (n >= rows - len || rows == 0) return;
    const int kvh = h / (a.q_heads / a.heads);
    const float c = a.scale * kLog2e;
    float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
    const T* qp = reinterpret_cast<const T*>(a.q + b * a.qb + n * a.qn + h * a.qh) + lane * E;
    for (int e = 0; e < E; ++e) q[e] = Half<T>::to(qp[e]);
    const uint32_t* mask = a.masks + (int64_t(b) * a.N + n) * kMaskWords;
    for (int t = 0; t < rows; ++t) {
        if (t >= len && !(mask[(t - len) / 32] >> ((t - len) % 32) & 1u)) continue;
        const int64_t at = int64_t(a.table[b * a.table_stride + t / a.page_size]) * a.page_stride +
                           (t % a.page_size) * a.row_stride + kvh * a.head_stride;
        const T* kp = reinterpret_cast<const T*>(a.kc + at) + lane * E;
        const T* vp = reinterpret_cast<const T*>(a.vc + at) + lane * E;
        float s = 0.f;
        for (int e = 0; e < E; ++e) s += q[e] * Half<T>::to(kp[e]);
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= c;
        const float m2 = fmaxf(m, s), f = ex2_approx(m - m2), p = ex2_approx(s - m2);
        l = l * f + p;
        m = m2;
        for (int e = 0; e < E; ++e) o[e] = o[e] * f + p * Half<T>::to(vp[e]);
    }
    T* op = reinterpret_cast<T*>(a.out + b * a.ob + n * a.on + h * a.oh) + lane * E;
    for (int e = 0; e < E; ++e) op[e] = Half<T>::from(o[e] / l);
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
    return SV_OK;
}

size_t masks_bytes(const sv_tree_attention_shape& s) { return align256(size_t(s.B) * s.N * kMaskWords * 4); }
size_t workspace_for(const sv_tree_attention_shape& s) { return align256(size_t(s.B) * 4) + masks_bytes(s); }

template <typename T, int D>
cudaError_t run(const AttnParams& a, cudaStream_t st) {
    const int words = a.heads * a.head_dim / 8;
    const int copies = 2 * a.N * words / (8 * kPrepThreads) + 1;
    cudaError_t e = launch_dependent(tree_prepare_kernel<T>, dim3(a.B, copies < 32 ? copies : 32), kPrepThreads, 0, 1,
                                     st, a);
    if (e != cudaSuccess) return e;
    const int64_t items = int64_t(a.B) * a.N * a.q_heads;
    return launch_dependent(tree_attend_kernel<T, D>, dim3(static_cast<unsigned>((items + kAttendWarps - 1) / kAttendWarps)),
                            kAttendWarps * 32, 0, 1, st, a);
}

}  // namespace
}  // namespace sv

extern "C" size_t sv_tree_attention_workspace_bytes(const sv_tree_attention_shape* shape, const sv_cache* cache) {
    return sv::attention_ok(shape, cache) == SV_OK ? sv::workspace_for(*shape) : 0;
}

extern "C" sv_status sv_tree_attention(const sv_tree_attention_shape* s, const sv_cache* cache, const void* q,
                                       const void* k, const void* v, const int32_t* page_table, const int32_t* lens,
                                       const int32_t* parents, const int32_t* counts, float scale, void* out,
                                       void* workspace, size_t workspace_bytes, void* stream) {
    using namespace sv;
    if (const sv_status why = attention_ok(s, cache); why != SV_OK) return why;
    if (!q || !k || !v || !page_table || !lens || !out || !workspace || !cache->k || !cache->v) return SV_EINVAL;
    if (!std::isfinite(scale) || workspace_bytes < workspace_for(*s)) return SV_EINVAL;
    for (const void* p : {q, k, v, static_cast<const void*>(out), static_cast<const void*>(cache->k),
                          static_cast<const void*>(cache->v), static_cast<const void*>(workspace)})
        if (!tree_aligned16(p)) return SV_EINVAL;
    if (s->B == 0) return SV_OK;
    AttnParams a{static_cast<char*>(cache->k), static_cast<char*>(cache->v), cache->page_stride * 2,
                 cache->row_stride * 2, cache->head_stride * 2, cache->pages, cache->page_size, cache->heads,
                 cache->head_dim, s->B, s->N, s->q_heads, s->max_pages,
                 s->table_stride ? s->table_stride : s->max_pages,
                 s->q_stride_b * 2, s->q_stride_n * 2, s->q_stride_h * 2, s->k_stride_b * 2, s->k_stride_n * 2,
                 s->k_stride_h * 2, s->v_stride_b * 2, s->v_stride_n * 2, s->v_stride_h * 2, s->o_stride_b * 2,
                 s->o_stride_n * 2, s->o_stride_h * 2, static_cast<const char*>(q), static_cast<const char*>(k),
                 static_cast<const char*>(v), static_cast<char*>(out), page_table, lens, parents, counts, scale,
                 static_cast<int32_t*>(workspace),
                 reinterpret_cast<uint32_t*>(static_cast<char*>(workspace) + align256(size_t(s->B) * 4))};
    auto st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (cache->dtype == SV_BF16)
        e = cache->head_dim == 64 ? run<__nv_bfloat16, 64>(a, st) : run<__nv_bfloat16, 128>(a, st);
    else
        e = cache->head_dim == 64 ? run<__half, 64>(a, st) : run<__half, 128>(a, st);
    return e == cudaSuccess ? SV_OK : SV_ECUDA;
}
