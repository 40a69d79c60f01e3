// sv_tree_attend.cuh -- the attention kernel of sv_tree_attention on the
// tensor cores, and the kernel that joins what several CTAs found.
//
// Mathematics.  For one request and key/value head, the rows of Q are its
// (node, query head of the group) pairs, up to 256 per unit of work, in tiles
// of 128.  Per tile of 128 cached rows: S = Q K^T, p = 2^(S c - m) with m a
// reference of each row (its maximum over the first tile of its run),
// O += P V, l += sum p.  The exponents' range leaves room above the reference
// and a weight's relative error does not depend on it, so the maximum is not
// followed: only when a tile's weights come to more than 2^15 is a new one
// looked for and O and l rescaled (scores past 2^22: far_exponents).  p is
// rounded to the cache's type for the second product.
//
// Roles (10 warps).  Warps 0-3 and 4-7 are two softmax groups, a thread per
// row of S (a lane of tensor memory).  Warp 8 loads K and V tiles by TMA, one
// box per page and 64 columns, into rings of shared memory.  Warp 9 issues
// the matrix instructions: S from shared memory, O from P in tensor memory
// (written over S) and V in shared memory.  With more than 128 rows the
// groups take one tile of rows each; with fewer they take the even and the
// odd cached tiles of the same rows, and their results are joined at the end,
// so that one group's exponentials overlap the other's products.
//
// Work split.  The cached tiles of all units form one line that is cut into
// equal runs, one per CTA (one CTA per SM), whatever the lengths of the
// requests.  A unit that lies in one run is finished there; the parts of
// one that is cut go to the workspace and are joined by
// tree_join_kernel in a fixed order.
//
// Bound.  Up to about 256 rows per head the cache's bytes: 64 KiB of K and V
// per tile take an SM's share of HBM some 1.5 us, the two products of 256
// rows about 1.1 us.  Measured, whole call: 64 chains of 9 nodes over 2000
// rows (360 MB, 8 key heads of 128, groups of 4) 94 us, 3.8 TB/s; 16 trees of
// 64 nodes over 8k to 16k rows (740 MB, 165 GFLOP) 194 us, 3.8 TB/s and 0.85
// PFLOP/s at 1.97 GHz, 227 us and 0.73 once the power limit of a long run of
// them holds the SM clock at 1.48; one token over 500 rows 12.4 us.  By length:
// 22 to 29 us a call and, for chains, 1.48 us a tile, which is the copy rate
// (6.3 TB/s over 32000 rows).  Units of 256 rows take 2.3 us a tile: 1510
// cycles for a group's weights, 750 until its products start, 1360 for the two
// of them; the tensor pipe is active 1940 cycles a tile, 60 %.
//
// What the registers decide.  A softmax thread holds 64 packed weights and 64
// scores; ten warps leave it 168 registers.  Spills go to L1, and shared
// memory leaves little of that: a build whose frames come to 100 bytes a
// thread takes 25 us longer.  So the weights' code is there once (masked
// scores are written back as -inf first), what runs once per unit is not
// unrolled, and the slow part of a wait is out of line.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "sv_tcgen05.cuh"
#include "sv_tree.h"
#include "sv_tree_common.cuh"

namespace sv {

constexpr int kTile = 128;                      // cached rows per step, and rows of Q per tile
constexpr int kUnitRows = 2 * kTile;            // rows of Q per unit of work
constexpr int kMaskWords = SV_MAX_NODES / 32;
constexpr int kAttendThreads = 320;
constexpr int kAttendMaxCtas = 160;

struct AttnParams {
    char* kc;
    char* vc;
    int64_t page_stride, row_stride, head_stride;  // of the cache, in bytes
    int32_t pages, page_size, heads, head_dim;
    int32_t B, N, q_heads, group, max_pages;  // group: query heads per key head
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
    int32_t slot_rows;  // rows of a partial result
    int32_t* ok;        // [B] the request passed all checks
    uint32_t* masks;    // [B][N][kMaskWords] ancestors-or-self of each node
    int32_t* odd;       // [B][N] the node's value row is not finite
    float2* part_ml;    // [2 CTAs][slot_rows] reference and sum,
    float4* part_o;     // [2 CTAs][head_dim / 4][slot_rows] and unnormalised result
};

template <typename T>
struct Half;
template <>
struct Half<__nv_bfloat16> {
    static constexpr uint32_t kNan2 = 0x7fc07fc0u, kExp2 = 0x7f807f80u, kType = 1;
    static constexpr int kExp2Degree = 3;
    static constexpr float kShift = 0.f;
    __device__ static uint32_t pack(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
};
template <>
struct Half<__half> {
    static constexpr uint32_t kNan2 = 0x7e007e00u, kExp2 = 0x7c007c00u, kType = 0;
    static constexpr int kExp2Degree = 4;
    // weights are kept 2^6 up, so that small ones do not fall among the
    // subnormals of a type whose least normal is 2^-14; 128 of them come to 2^13
    static constexpr float kShift = 6.f;
    __device__ static uint32_t pack(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
};

// 2^x for a pair on the multiply-add pipe: 2^n 2^f with n the nearest whole
// number and a minimax polynomial for 2^f on [-1/2, 1/2] that is 1 at 0,
// relative error 1.0e-04 (degree 3) or 2.8e-06 (degree 4), well inside half a step of
// the type that the weights are rounded to.  Below -127 it is exactly 0: there
// n = -127 takes the exponent of 1 to nothing.  The special-function unit does
// 16 a cycle and is the softmax's bottleneck; kExp2Every says which pairs it is
// spared: every 4th 95 us for a batch of chains and 194 for long trees, every
// 8th 97 and 196, every 3rd 99 and 197, every 2nd 109 and 214, none 115 and 213.
constexpr int kExp2Every = 4;
// What 128 weights may come to before their row gets a new reference: within
// the range of fp16, and far from where the products could overflow.
constexpr float kMostSum = 32768.f;
template <int kDegree>
__device__ __forceinline__ uint64_t exp2_pair(uint64_t x) {
    float a, b;
    f2_unpack(x, a, b);
    x = f2_pack(max_nan(a, -127.f), max_nan(b, -127.f));
    const uint64_t t = f2_add(x, f2_pack(12582912.f, 12582912.f));  // 1.5 2^23: the low bits are n
    const uint64_t f = f2_fma(f2_add(t, f2_pack(-12582912.f, -12582912.f)), f2_pack(-1.f, -1.f), x);
    uint64_t p;
    if constexpr (kDegree == 3) {
        p = f2_fma(f2_pack(0.05500893085f, 0.05500893085f), f, f2_pack(0.2422109594f, 0.2422109594f));
        p = f2_fma(p, f, f2_pack(0.6932829272f, 0.6932829272f));
        p = f2_fma(p, f, f2_pack(1.f, 1.f));
    } else {
        p = f2_fma(f2_pack(0.00958285307f, 0.00958285307f), f, f2_pack(0.05590642463f, 0.05590642463f));
        p = f2_fma(p, f, f2_pack(0.2402409861f, 0.2402409861f));
        p = f2_fma(p, f, f2_pack(0.6931241934f, 0.6931241934f));
        p = f2_fma(p, f, f2_pack(1.f, 1.f));
    }
    float pa, pb, ta, tb;
    f2_unpack(p, pa, pb);
    f2_unpack(t, ta, tb);
    return f2_pack(__uint_as_float(__float_as_uint(pa) + (__float_as_uint(ta) << 23)),
                   __uint_as_float(__float_as_uint(pb) + (__float_as_uint(tb) << 23)));
}

// ---------------------------------------------------------------------------
// The line of tiles.

__device__ __forceinline__ int groups_of(const AttnParams& a, int count) {
    return (count * (a.group) + kUnitRows - 1) / kUnitRows;
}
// Cached rows of request b with its nodes, 0 where there is nothing to do
// (what tree_prepare_kernel finds wrong beyond this is left to it).
__device__ __forceinline__ int rows_of(const AttnParams& a, int b, int* len) {
    const int count = a.counts ? a.counts[b] : a.N;
    *len = a.lens[b];
    const int64_t rows = int64_t(*len) + count;
    const bool fits = count > 0 && count <= a.N && *len >= 0 && rows <= int64_t(a.max_pages) * a.page_size;
    return fits ? static_cast<int>(rows) : 0;
}
// Tiles of request b's units.
__device__ __forceinline__ int64_t tiles_of(const AttnParams& a, int b) {
    int len;
    const int rows = rows_of(a, b, &len);
    if (rows == 0) return 0;
    return int64_t((rows + kTile - 1) / kTile) * a.heads * groups_of(a, rows - len);
}
// Sums of v over the threads before this one and over all (whole warps).
template <int kThreads>
__device__ int64_t scan_block(int64_t v, int64_t* total, int64_t* warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int64_t before = 0, all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += warp_sums[w];
        all += warp_sums[w];
    }
    *total = all;
    return before + incl - v;
}

struct Piece {
    int b, head, row0, rows_q, len, rows;  // rows: cached rows of the request
    int first, n, tiles;                   // tiles [first, first + n) of the unit's `tiles`
    bool split;                            // both groups on the same rows of Q
};

// Walks this CTA's run; every role has its own.
struct PieceIter {
    int b, rem;    // request, tile within the request
    int64_t left;  // tiles left in the run
    __device__ bool next(const AttnParams& a, Piece& p) {
        if (left <= 0) return false;
        int rows, len;
        while ((rows = rows_of(a, b, &len)) == 0) {
            ++b;
            rem = 0;
        }
        const int g = a.group, R = (rows - len) * g;
        const int groups = (R + kUnitRows - 1) / kUnitRows, tiles = (rows + kTile - 1) / kTile;
        const int unit = rem / tiles;
        p.b = b;
        p.head = unit / groups;
        p.row0 = (unit % groups) * kUnitRows;
        p.rows_q = R - p.row0 < kUnitRows ? R - p.row0 : kUnitRows;
        p.len = len;
        p.rows = rows;
        p.tiles = tiles;
        p.first = rem - unit * tiles;
        p.n = tiles - p.first < left ? tiles - p.first : static_cast<int>(left);
        p.split = p.rows_q <= kTile;
        rem += p.n;
        left -= p.n;
        if (rem == tiles * a.heads * groups) {
            ++b;
            rem = 0;
        }
        return true;
    }
};

// ---------------------------------------------------------------------------

// All of it stays below 196 KiB (164 KiB for D = 64), the step of the carve-out
// that leaves 60 KiB (92 KiB) of L1 for the page table, the masks, Q and the
// softmax warps' few spilled registers.  A third stage of K leaves 28 KiB and
// costs 7 % of a batch of chains (107 us against 100) although more is in flight.
template <int D>
struct AttendSmem {
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kKStages = D == 128 ? 2 : 4;
    static constexpr int kVStages = D == 128 ? 2 : 4;
    struct Ctrl {
        uint64_t kfull[kKStages], kempty[kKStages], vfull[kVStages], vempty[kVStages];
        uint64_t qfull[2], sfull[2], pfull[2], ofull[2];
        int64_t warp_sums[kAttendThreads / 32];
        int64_t left;
        float m1[kTile], l1[kTile];
        uint32_t odd[2][2][kTile / 32];  // [group][tile parity]: rows of V that are not finite
        uint32_t tmem;
        int32_t b0, rem0;
    };
    static_assert(kTileBytes % 1024 == 0, "the 128-byte swizzle repeats every 1024 bytes");
    static constexpr size_t bytes() { return size_t(2 + kKStages + kVStages) * kTileBytes + sizeof(Ctrl); }
};

// The 32 mask bits of cached rows a0 .. a0 + 31 of the tree (rows before the
// tree are seen by all).
__device__ __forceinline__ uint32_t mask_word(const uint32_t* mask, int a0) {
    if (a0 <= -32) return 0xffffffffu;
    if (a0 < 0) return ((1u << -a0) - 1u) | (mask[0] << -a0);
    const int w = a0 >> 5, s = a0 & 31;
    if (w >= kMaskWords) return 0u;
    return __funnelshift_r(mask[w], w + 1 < kMaskWords ? mask[w + 1] : 0u, s);
}

// Maximum of this row's 128 scores at `addr`.
__device__ __forceinline__ float tile_top(uint32_t addr) {
    float m = -INFINITY;
#pragma unroll 1
    for (int w = 0; w < 4; ++w) {
        uint32_t s[32];
        tmem_load(s, addr + 32 * w);
#pragma unroll
        for (int k = 0; k < 32; k += 2) m = max3(__uint_as_float(s[k]), __uint_as_float(s[k + 1]), m);
    }
    return m;
}

// A reference is its maximum's s c rounded to a float, the weights' exponents
// s c - ref are not: past kFar (2^22) the two differ by so much (1 at 2^23, 64
// at 2^29) that weights would leave the type's range.  A warp with such a row
// looks for the maximum of every tile, takes a reference that is not above it,
// and puts exponents of at most `most` in the scores' place.  Up to 2^26 the
// bound changes nothing; past it, it rounds scores by less than two steps of a
// float of their size.
constexpr float kFar = 4194304.f;  // 2^22
constexpr float kFarRoom = 8.f;    // 2^(6 + 8) is in fp16's range
__device__ __noinline__ void far_exponents(uint32_t addr, float c, float ref, float most) {
#pragma unroll 1
    for (int w = 0; w < 4; ++w) {
        uint32_t s[32];
        tmem_load(s, addr + 32 * w);
#pragma unroll
        for (int k = 0; k < 32; ++k) {
            const float x = fmaf(__uint_as_float(s[k]), c, -ref);
            s[k] = __float_as_uint(x > most ? most : x);  // (NaN stays)
        }
        tmem_store(addr + 32 * w, s);
    }
    tmem_wait_st();
}

// Weights 2^(s c - ref) of the row's 128 scores, packed in pairs; returns
// their sum (NaN or past kMostSum where the reference is too low for the type
// to hold them).  The next 32 scores are on their way while 32 are worked on,
// and nothing branches in between, so that the pairs overlap in the pipes.
template <typename T>
__device__ __forceinline__ float tile_weights(uint32_t addr, float c, float ref, uint32_t (&packed)[64]) {
    using H = Half<T>;
    const uint64_t cc = f2_pack(c, c), mm = f2_pack(-ref, -ref);
    uint64_t sum[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
    float top = -INFINITY;  // of the exponents that exp2_pair takes
    uint32_t s[2][32];
    tmem_start(s[0], addr);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        tmem_arrived(s[w & 1]);
        if (w < 3) tmem_start(s[(w + 1) & 1], addr + 32 * (w + 1));
        uint32_t(&v)[32] = s[w & 1];
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
            const uint64_t x2 = f2_fma(f2_pack(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), cc, mm);
            float x, y;
            f2_unpack(x2, x, y);
            if (k / 2 % kExp2Every == kExp2Every - 1) {
                top = max3(x, y, top);
                f2_unpack(exp2_pair<H::kExp2Degree>(x2), x, y);
            } else {
                x = ex2_approx(x);
                y = ex2_approx(y);
            }
            packed[16 * w + k / 2] = H::pack(x, y);
            sum[k / 2 & 1] = f2_add(sum[k / 2 & 1], f2_pack(x, y));
        }
    }
    float x, y;
    f2_unpack(f2_add(sum[0], sum[1]), x, y);
    return top > 64.f ? INFINITY : x + y;
}

template <typename T, int D>
__global__ void __launch_bounds__(kAttendThreads, 1)
tree_attend_kernel(const AttnParams a, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap) {
    using S = AttendSmem<D>;
    using H = Half<T>;
    constexpr int KS = S::kKStages, VS = S::kVStages, TB = S::kTileBytes;
    // tensor memory: scores (then weights) of the two groups, then their results
    auto s_at = [](int t) { return static_cast<uint32_t>(t * kTile); };
    auto o_at = [](int t) { return static_cast<uint32_t>(2 * kTile + t * D); };
    extern __shared__ __align__(1024) unsigned char qs[];  // two tiles of Q, then K, V and the rest
    unsigned char* ks = qs + 2 * TB;
    unsigned char* vs = ks + KS * TB;
    auto& ctl = *reinterpret_cast<typename S::Ctrl*>(vs + VS * TB);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;  // uniform

    if (warp == 8 && lane == 0) {
        for (int i = 0; i < KS; ++i) {
            mbar_init(&ctl.kfull[i], 1);
            mbar_init(&ctl.kempty[i], 1);
        }
        for (int i = 0; i < VS; ++i) {
            mbar_init(&ctl.vfull[i], 1);
            mbar_init(&ctl.vempty[i], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&ctl.qfull[t], kTile / 32);
            mbar_init(&ctl.sfull[t], 1);
            mbar_init(&ctl.pfull[t], kTile / 32);
            mbar_init(&ctl.ofull[t], 1);
        }
        fence_mbar_init();
        tma_prefetch_map(&kmap);
        tma_prefetch_map(&vmap);
    }
    if (warp == 9) tmem_alloc(&ctl.tmem, 512);
    if (tid == 0) ctl.left = 0;
    grid_launch_dependents();
    // The kernel before this one (tree_prepare_kernel) lets this one start once all work before it
    // is done: the inputs and the cached prefix can be read.  What it writes itself, the new rows
    // and the checks, is waited for where it is read.
    auto reads_new_rows = [](const Piece& p, int tile) { return (tile + 1) * kTile > p.len; };

    // this CTA's run of tiles
    {
        const int each = (a.B + kAttendThreads - 1) / kAttendThreads;
        const int lo = tid * each < a.B ? tid * each : a.B, hi = lo + each < a.B ? lo + each : a.B;
        int64_t mine = 0, total;
        for (int b = lo; b < hi; ++b) mine += tiles_of(a, b);
        int64_t at = scan_block<kAttendThreads>(mine, &total, ctl.warp_sums);
        const int64_t per = (total + gridDim.x - 1) / gridDim.x;
        const int64_t start = per * blockIdx.x;
        if (mine > 0 && at <= start && start < at + mine) {
            for (int b = lo; b < hi; ++b) {
                const int64_t n = tiles_of(a, b);
                if (start < at + n) {
                    ctl.b0 = b;
                    ctl.rem0 = static_cast<int>(start - at);
                    ctl.left = total - start < per ? total - start : per;
                    break;
                }
                at += n;
            }
        }
    }
    tcgen05_fence_before();
    __syncthreads();
    tcgen05_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, ctl.tmem, 0);
    PieceIter it{ctl.b0, ctl.rem0, ctl.left};
    Piece p{};

    if (warp == 8) {
        // ---- loads: a box per page and 64 columns
        constexpr int kPages = kTile / 16;  // pages of a tile, at most
        uint32_t kn = 0, vn = 0;            // tiles issued
        bool ok = true;
        const int per_tile = kTile / a.page_size;
        auto wait_new_rows = [] {
            grid_dependency_wait();
            asm volatile("fence.proxy.async;" ::: "memory");
        };
        struct Ids {
            int id[kPages];  // -1: past the request
        };
        auto fetch = [&](int tile) {
            Ids x;
            const int32_t* ids = a.table + p.b * a.table_stride + tile * per_tile;
#pragma unroll
            for (int i = 0; i < kPages; ++i)
                x.id[i] = i < per_tile && (tile * per_tile + i) * a.page_size < p.rows ? ids[i] : -1;
            return x;
        };
        auto load = [&](const CUtensorMap* map, unsigned char* ring, uint64_t* full, uint64_t* empty, uint32_t stages,
                        uint32_t& n, const Ids& ids) {
            const uint32_t s = n % stages;
            ok = ok && (n < stages || mbar_wait_short(empty + s, (n / stages - 1) & 1));
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) return;
            unsigned char* dst = ring + s * TB;
            if (elect_one()) {
                int pages = 0;
#pragma unroll
                for (int i = 0; i < kPages; ++i) pages += ids.id[i] >= 0;
                mbar_arrive_expect_tx(full + s, static_cast<uint32_t>(pages * a.page_size * D * 2));
#pragma unroll
                for (int i = 0; i < kPages; ++i)
                    if (ids.id[i] >= 0) {
#pragma unroll
                        for (int x = 0; x < D; x += 64)
                            tma_load_4d(dst + (x / 64) * (kTile * 128) + i * a.page_size * 128, map, x, p.head, 0,
                                        ids.id[i], full + s);
                    }
            }
            __syncwarp();
            ++n;
        };
        while (ok && it.next(a, p)) {
            Ids id = fetch(p.first), next = id;
            if (p.n > 1) next = fetch(p.first + 1);
            if (reads_new_rows(p, p.first)) wait_new_rows();
            load(&kmap, ks, ctl.kfull, ctl.kempty, KS, kn, id);
            for (int i = 0; i < p.n && ok; ++i) {
                Ids after = next;
                if (i + 2 < p.n) after = fetch(p.first + i + 2);
                if (i + 1 < p.n) {
                    if (reads_new_rows(p, p.first + i + 1)) wait_new_rows();
                    load(&kmap, ks, ctl.kfull, ctl.kempty, KS, kn, next);
                }
                load(&vmap, vs, ctl.vfull, ctl.vempty, VS, vn, id);
                id = next;
                next = after;
            }
        }
        // a wait ran out: nothing may be in flight when the CTA ends
        if (!ok) {
            for (uint32_t i = kn > KS ? kn - KS : 0; i < kn; ++i)
                mbar_wait_short(&ctl.kfull[i % KS], (i / KS) & 1);
            for (uint32_t i = vn > VS ? vn - VS : 0; i < vn; ++i)
                mbar_wait_short(&ctl.vfull[i % VS], (i / VS) & 1);
        }
    } else if (warp == 9) {
        // ---- matrix products
        {
            uint32_t kn = 0, vn = 0, qn[2] = {0, 0}, pn[2] = {0, 0};
            bool ok = true;
            const uint32_t qaddr = smem_u32(qs), kaddr = smem_u32(ks), vaddr = smem_u32(vs);
            auto wait = [&](uint64_t* bar, uint32_t n) {
                ok = ok && mbar_wait_short(bar, n & 1);
                ok = __all_sync(0xffffffffu, ok);
                tcgen05_fence_after();
            };
            // (advancing an operand adds to its address field, in units of 16 bytes)
            auto qk = [&](int t, int qtile) {  // S[t] = Q[qtile] K^T, K the tile `kn`
                const uint64_t q0 = smem_operand(qaddr + qtile * TB, 16, 1024);
                const uint64_t k0 = smem_operand(kaddr + (kn % KS) * TB, 16, 1024);
                const uint32_t d = tmem + s_at(t);
                if (elect_one()) {
#pragma unroll
                    for (int x = 0; x < D; x += 16) {
                        const uint32_t at = ((x / 64) * (kTile * 128) + (x % 64) * 2) >> 4;
                        mma_ss(d, q0 + at, k0 + at, mma_shape(H::kType, kTile, false), x > 0);
                    }
                    tcgen05_commit(&ctl.sfull[t]);
                }
                __syncwarp();
            };
            auto pv = [&](int t, bool add) {  // O[t] (+)= P[t] V, V the tile `vn`
                const uint64_t v0 = smem_operand(vaddr + (vn % VS) * TB, kTile * 128, 1024);
                const uint32_t d = tmem + o_at(t), w = tmem + s_at(t);
                if (elect_one()) {
#pragma unroll
                    for (int x = 0; x < kTile; x += 16)
                        mma_ts(d, w + x / 2, v0 + (x * 128 >> 4), mma_shape(H::kType, D, true), add || x > 0);
                }
                __syncwarp();
            };
            auto commit = [&](uint64_t* bar) {
                if (elect_one()) tcgen05_commit(bar);
                __syncwarp();
            };
            auto k_ready = [&] { wait(&ctl.kfull[kn % KS], kn / KS); };
            auto k_done = [&] {
                commit(&ctl.kempty[kn % KS]);
                ++kn;
            };
            while (ok && it.next(a, p)) {
                wait(&ctl.qfull[0], qn[0]++);
                if (!p.split) wait(&ctl.qfull[1], qn[1]++);
                // the first scores
                for (int t = 0; t < 2 && ok; ++t) {
                    if (p.split ? t < p.n : t == 0) k_ready();
                    if (!ok || (p.split && t >= p.n)) break;
                    qk(t, p.split ? 0 : t);
                    if (p.split || t == 1) k_done();
                }
                for (int i = 0; i < p.n && ok; ++i) {
                    wait(&ctl.vfull[vn % VS], vn / VS);
                    if (p.split) {
                        const int t = i & 1;
                        wait(&ctl.pfull[t], pn[t]++);
                        if (!ok) break;
                        pv(t, i >= 2);
                        commit(&ctl.vempty[vn % VS]);
                        ++vn;
                        if (i + 2 >= p.n) commit(&ctl.ofull[t]);
                        if (i + 2 < p.n) {
                            k_ready();
                            if (!ok) break;
                            qk(t, 0);
                            k_done();
                        }
                    } else {
                        for (int t = 0; t < 2 && ok; ++t) {
                            wait(&ctl.pfull[t], pn[t]++);
                            if (!ok) break;
                            pv(t, i > 0);
                            if (t == 1) commit(&ctl.vempty[vn % VS]);
                            if (i + 1 == p.n) {
                                commit(&ctl.ofull[t]);
                            } else {
                                if (t == 0) k_ready();
                                if (!ok) break;
                                qk(t, t);
                                if (t == 1) k_done();
                            }
                        }
                        ++vn;
                    }
                }
            }
        }
    } else {
        // ---- softmax: group t, row r (a lane of tensor memory)
        const int t = warp >> 2, r = tid & (kTile - 1);
        const uint32_t lanes = tmem + (uint32_t(warp & 3) << 21);
        const int g = a.group;
        const float c = fmaxf(fabsf(a.scale) * kLog2e, 1e-37f);
        const uint32_t sign = a.scale < 0.f ? 0x80008000u : 0u;
        uint32_t sn = 0, on = 0, vn = 0;
        bool ok = true;
        while (it.next(a, p)) {
            const int tile0 = p.split ? 0 : t * kTile;
            const int rows_here = p.rows_q - tile0;              // valid rows of this group's tile
            const bool live = (warp & 3) * 32 < rows_here;       // some row of this warp is valid
            const int row = p.row0 + tile0 + r, node = row / g, h = p.head * g + row % g;
            const bool valid = r < rows_here;
            if (t == 0 || !p.split) {
                // Q into shared memory, 128-byte swizzle; rows past the unit are zero
                unsigned char* dst = qs + t * TB + r * 128;
                const uint4* src = reinterpret_cast<const uint4*>(a.q + p.b * a.qb + node * a.qn + h * a.qh);
#pragma unroll
                for (int x = 0; x < D / 8; ++x) {
                    uint4 w{0, 0, 0, 0};
                    if (valid) {
                        w = __ldg(src + x);
                        w.x ^= sign;
                        w.y ^= sign;
                        w.z ^= sign;
                        w.w ^= sign;
                    }
                    *reinterpret_cast<uint4*>(dst + (x / 8) * (kTile * 128) + (((x % 8) ^ (r & 7)) * 16)) = w;
                }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.qfull[t]);
            }
            const uint32_t* mask = a.masks + (int64_t(p.b) * a.N + (valid ? node : 0)) * kMaskWords;
            float m = -INFINITY, l = 0.f;
            const int step = p.split ? 2 : 1, from = p.split ? t : 0;
            bool odd = false;
            for (int i = from; i < p.n; i += step) {
                const int pos0 = (p.first + i) * kTile;
                const bool tail = reads_new_rows(p, p.first + i);  // holds rows of the tree, or past it
                bool clear = false, bad = false;
                uint32_t see0, see1, see2, see3;                   // which columns this row sees, 32 to a word
                if (tail) {
                    // (what is read here is on its way while the scores are waited for)
                    grid_dependency_wait();
                    const int a0 = pos0 + r - p.len;
                    const bool past = pos0 + r >= p.rows;
                    bad = !past && a0 >= 0 && a.odd[int64_t(p.b) * a.N + a0] != 0;
                    clear = past || bad;
                    see0 = mask_word(mask, pos0 - p.len);
                    see1 = mask_word(mask, pos0 + 32 - p.len);
                    see2 = mask_word(mask, pos0 + 64 - p.len);
                    see3 = mask_word(mask, pos0 + 96 - p.len);
                }
                // (after a wait that ran out every barrier is still met, so that no thread waits for good)
                const int parity = sn & 1;
                ok = ok && mbar_wait_short(&ctl.sfull[t], parity);
                ++sn;
                if (tail) {
                    const uint32_t bits = __ballot_sync(0xffffffffu, bad);
                    if (lane == 0) ctl.odd[t][parity][warp & 3] = bits;
                    named_barrier_sync(1 + t, kTile);            // the group's bits are written
                }
                ok = __all_sync(0xffffffffu, ok);
                tcgen05_fence_after();
                if (live && ok) {
                    if (tail) {
                        // scores of what the row does not see become -inf, 32 columns at a time
#pragma unroll 1
                        for (int w = 0; w < 4; ++w) {
                            const uint32_t see = w < 2 ? (w == 0 ? see0 : see1) : (w == 2 ? see2 : see3);
                            odd |= (see & ctl.odd[t][parity][w]) != 0;
                            if (__all_sync(0xffffffffu, see == 0xffffffffu)) continue;
                            uint32_t x[32];
                            tmem_load(x, lanes + s_at(t) + 32 * w);
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (!(see >> k & 1u)) x[k] = 0xff800000u;
                            tmem_store(lanes + s_at(t) + 32 * w, x);
                        }
                        tmem_wait_st();
                    }
                    // Weights against the reference so far; only where some row of the warp rises
                    // too far over it for its weights to be held (and in the first tile of a
                    // piece) is the maximum looked for and the reference moved there.
                    uint32_t packed[64];
                    float part = 0.f;
                    // (a row without a reference, -inf, or one whose reference is far)
                    bool fresh = !__all_sync(0xffffffffu, fabsf(m) < kFar), far = false;
                    float ce = c, re = m;  // (chosen here and not at the call: 93.6 us for chains against 95.7)
                    for (;;) {
                        if (!fresh) {
                            part = tile_weights<T>(lanes + s_at(t), ce, re, packed);
                            // (a sum that is NaN is not mended by another reference)
                            if (!__any_sync(0xffffffffu, part > kMostSum) || far) break;
                        }
                        // rounded down, so that no reference lies above its maximum
                        const float top = __fadd_rd(__fmul_rd(tile_top(lanes + s_at(t)), c), -H::kShift);
                        if (!fresh && !__any_sync(0xffffffffu, top > m)) break;
                        const float f = top > m ? ex2_approx(m - top) : 1.f;  // 0 where there was nothing yet
                        if (top > m) m = top;
                        if (i != from) {
                            l *= f;
#pragma unroll 1
                            for (int x = 0; x < D; x += 32) {
                                uint32_t o[32];
                                tmem_load(o, lanes + o_at(t) + x);
#pragma unroll
                                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                                tmem_store(lanes + o_at(t) + x, o);
                            }
                        }
                        fresh = false;
                        far = __any_sync(0xffffffffu, m > -INFINITY && fabsf(m) >= kFar);
                        re = m == -INFINITY ? 0.f : m;  // (a row that sees nothing yet: all weights 0)
                        if (far) {
                            far_exponents(lanes + s_at(t), c, re, H::kShift + kFarRoom);
                            ce = 1.f;
                            re = 0.f;
                        }
                    }
                    l += part;
                    tmem_store(lanes + s_at(t), packed);         // over the scores
                    tmem_wait_st();
                }
                // V rows that nobody may see become zero before P V reads them: rows past the
                // request and rows of the tree that are not finite (they make NaN of the nodes
                // that see them, by `odd`).  The scores of this tile say that the products two tiles back
                // are done, so the V stage is in this tile's phase or the one before it.
                if (tail && (t == 0 || p.split)) {
                    const uint32_t n = vn + i;
                    ok = ok && mbar_wait_short(&ctl.vfull[n % VS], (n / VS) & 1);
                    const uint32_t rows = __ballot_sync(0xffffffffu, clear);
                    // (eight lanes to a row's 128 bytes: a thread per row would write to the same banks)
                    unsigned char* at = vs + (n % VS) * TB + (warp & 3) * (32 * 128) + lane * 16;
#pragma unroll 1
                    for (int x = 0; x < 8 && rows != 0; ++x) {
                        if (!(rows >> (4 * x + lane / 8) & 1u)) continue;
#pragma unroll
                        for (int d = 0; d < D / 64; ++d)
                            *reinterpret_cast<uint4*>(at + x * (4 * 128) + d * (kTile * 128)) = uint4{0, 0, 0, 0};
                    }
                    fence_async_shared();
                }
                tcgen05_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.pfull[t]);
            }
            vn += p.n;
            if (odd || !ok) l = NAN;
            const bool any = from < p.n;
            if (any) ok = ok && mbar_wait_short(&ctl.ofull[t], on++ & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) l = NAN;
            tcgen05_fence_after();
            float f0 = 1.f, f1 = 0.f;
            if (p.split) {
                // group 0 joins both groups' results
                if (t == 1) {
                    ctl.m1[r] = m;
                    ctl.l1[r] = l;
                }
                named_barrier_sync(3, 2 * kTile);
                tcgen05_fence_after();
                if (t == 0) {
                    const float mo = ctl.m1[r], lo = ctl.l1[r], M = fmaxf(m, mo);
                    const float ref = M == -INFINITY ? 0.f : M;
                    f0 = ex2_approx(m - ref);
                    f1 = ex2_approx(mo - ref);
                    l = l * f0 + lo * f1;
                    m = M;
                }
            }
            grid_dependency_wait();
            if (live && (t == 0 || !p.split)) {
                const bool good = valid && a.ok[p.b] != 0;
                const bool whole = p.n == p.tiles;
                const int64_t slot = 2 * int64_t(blockIdx.x) + (p.first == 0);
                const int slot_row = tile0 + r;
                const float inv = 1.f / l;
                char* dst = a.out + p.b * a.ob + node * a.on + h * a.oh;
                const bool both = p.split && p.n > 1;
#pragma unroll 1
                for (int x = 0; x < D; x += 32) {
                    uint32_t o[32];
                    tmem_load(o, lanes + o_at(t) + x);
                    if (p.split) {
                        uint32_t o1[32];
                        if (both) tmem_load(o1, lanes + o_at(1) + x);
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            float y = __uint_as_float(o[k]) * f0;
                            if (both) y = fmaf(__uint_as_float(o1[k]), f1, y);
                            o[k] = __float_as_uint(y);
                        }
                    }
                    if (good && whole) {
#pragma unroll
                        for (int k = 0; k < 32; k += 8) {
                            uint4 w;
                            uint32_t* wp = &w.x;
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                wp[e] = H::pack(__uint_as_float(o[k + 2 * e]) * inv, __uint_as_float(o[k + 2 * e + 1]) * inv);
                            *reinterpret_cast<uint4*>(dst + (x + k) * 2) = w;
                        }
                    } else if (good) {
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            a.part_o[(slot * (D / 4) + (x + k) / 4) * a.slot_rows + slot_row] =
                                float4{__uint_as_float(o[k]), __uint_as_float(o[k + 1]), __uint_as_float(o[k + 2]),
                                       __uint_as_float(o[k + 3])};
                    }
                    __syncwarp();
                }
                if (valid && !whole) a.part_ml[slot * a.slot_rows + slot_row] = float2{m, l};
            }
            tcgen05_fence_before();
            if (p.split) named_barrier_sync(3, 2 * kTile);       // O of group 1 and the exchange are read
        }
    }
    grid_dependency_wait();  // this grid ends after the one before it
    tcgen05_fence_before();
    __syncthreads();
    tcgen05_fence_after();
    if (warp == 9) {
        __syncwarp();
        tmem_free(tmem, 512);
    }
}

// Joins the parts of units that were cut: 32 rows of one unit per CTA, a lane
// per row, kCols columns of four per warp, the rest over blockIdx.z.  Usually
// there are two or three parts; few units over a long axis have many, and
// their CTAs are few: then a warp takes one column and loads eight parts at a
// time (sv_tree_attention.cu chooses).
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;

template <typename T, int D, int kCols>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const AttnParams a, int units, int ctas) {
    __shared__ int64_t sums[2][kJoinWarps];
    __shared__ float tops[kJoinWarps][32];
    const int b = blockIdx.x / units, unit = blockIdx.x % units;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int len;
    const int rows = rows_of(a, b, &len);
    if (rows == 0) {
        grid_dependency_wait();
        return;
    }
    const int g = a.group, R = (rows - len) * g;
    const int groups = (R + kUnitRows - 1) / kUnitRows, tiles = (rows + kTile - 1) / kTile;
    const int row0 = (unit % groups) * kUnitRows, r = blockIdx.y * 32 + lane;
    if (unit >= a.heads * groups || row0 + static_cast<int>(blockIdx.y) * 32 >= R) {
        grid_dependency_wait();
        return;
    }
    int64_t before = 0, all = 0;
    for (int i = tid; i < a.B; i += kJoinThreads) {
        const int64_t n = tiles_of(a, i);
        all += n;
        if (i < b) before += n;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, o);
        all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    if (lane == 0) {
        sums[0][warp] = before;
        sums[1][warp] = all;
    }
    __syncthreads();
    before = all = 0;
    for (int w = 0; w < kJoinWarps; ++w) {
        before += sums[0][w];
        all += sums[1][w];
    }
    const int64_t per = (all + ctas - 1) / ctas;
    const int64_t u0 = before + int64_t(unit) * tiles;
    const int c0 = static_cast<int>(u0 / per), c1 = static_cast<int>((u0 + tiles - 1) / per);
    grid_dependency_wait();
    if (c0 == c1 || a.ok[b] == 0) return;
    const bool in = row0 + r < R && r < kUnitRows;
    float M = -INFINITY;
    if (in)
#pragma unroll 4
        for (int c = c0 + warp; c <= c1; c += kJoinWarps)
            M = fmaxf(M, a.part_ml[(2 * int64_t(c) + (c == c0)) * a.slot_rows + r].x);
    tops[warp][lane] = M;
    __syncthreads();
    if (!in) return;
    for (int w = 0; w < kJoinWarps; ++w) M = fmaxf(M, tops[w][lane]);
    const float ref = M == -INFINITY ? 0.f : M;
    const int node = (row0 + r) / g, h = (unit / groups) * g + (row0 + r) % g;
    char* dst = a.out + b * a.ob + node * a.on + h * a.oh;
    const int col0 = (blockIdx.z * kJoinWarps + warp) * kCols;
    float4 o[kCols] = {};
    float l = 0.f;
#pragma unroll kCols == 1 ? 8 : 2
    for (int c = c0; c <= c1; ++c) {
        const int64_t slot = 2 * int64_t(c) + (c == c0);
        const float2 ml = a.part_ml[slot * a.slot_rows + r];
        const float f = ex2_approx(ml.x - ref);
        l += ml.y * f;
#pragma unroll
        for (int k = 0; k < kCols; ++k) {
            const float4 v = a.part_o[(slot * (D / 4) + col0 + k) * a.slot_rows + r];
            o[k].x = fmaf(v.x, f, o[k].x);
            o[k].y = fmaf(v.y, f, o[k].y);
            o[k].z = fmaf(v.z, f, o[k].z);
            o[k].w = fmaf(v.w, f, o[k].w);
        }
    }
    const float inv = 1.f / l;
#pragma unroll
    for (int k = 0; k < kCols; ++k)
        *reinterpret_cast<uint2*>(dst + (col0 + k) * 8) =
            uint2{Half<T>::pack(o[k].x * inv, o[k].y * inv), Half<T>::pack(o[k].z * inv, o[k].w * inv)};
}

}  // namespace sv
