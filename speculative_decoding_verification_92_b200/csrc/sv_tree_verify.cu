// sv_tree_verify.cu -- sv_tree_verify: lossless verification of a drafted
// token tree, one thread-block cluster per request.
//
// Mathematics.  The walk from the root visits one node per level.  At a node
// with target row z the weights are 2^((z_v - M) c), c = log2(e) / T, M the
// row's maximum; everything else is ratios of sums of weights.
//   ids only: the sum is taken over the tokens that are no child's (base), the
//     children's weights e_c apart.  The mass before child c is then
//     base + sum of e over the distinct children from c on: no subtraction,
//     so no cancellation when the children hold nearly all of it; and base is
//     the mass of the final draw.
//   draft logits: r rejected independent draws from q leave
//     max(0, p - l q) / n with l the sum of the n's before it (l, n = 0, 1 at
//     the start), because max(0, max(0, p - l q) / n - q) is
//     max(0, p - (l + n) q) / n.  A rejection therefore costs one pass that
//     sums max(0, p - l q), whatever was rejected before.
// Why 64 bits: the answer is a whole number.  A vocabulary of 150k tokens has
// CDF steps of 1e-8 and less; sums in 32 bits move the CDF by more than
// that, and one draw in some hundred would pick a neighbouring token.  An
// acceptance test is another matter: it compares u with a ratio of sums, so a
// first pass in 32 bits with a proven error bound (kFastError) settles nearly
// all of them, and only a test within the bound of its border, a rejection or
// a leaf (which need the exact sums for the draw) makes the pass in 64 bits.
//
// Bound.  Only rows on the accepted path are read, so a step is a chain of
// visits: load latency, the arithmetic of one row, one cluster barrier.  The
// CTAs of a cluster split the vocabulary; the more requests, the smaller the
// cluster, so that all of them run at once (cluster_for).  A warp owns one
// contiguous range of the row, which is the unit the final draw looks up.
//
// Measured on the device, V = 151936 in bf16.  A visit takes 3.7 us for one
// request and 8.8 us for 64 (their rows alone 3 us at copy rate); greedy 2.1
// and 5.9.  A leaf, which needs the 64-bit pass and the draw, 10 and 30 us, of
// them the draw 3 and 7.  128 trees of 40 nodes: 92 us; 64 trees of 13 nodes
// with draft logits in fp32 (V = 128256): 112 us.  Four CTAs per SM with 64
// registers against two with 128: 92 to 113 us and 112 to 134, although the
// leaf alone gains (30 to 26).  Batches loaded ahead of their use cost 10 us
// (spills).
#include <cmath>
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "sv_tree.h"
#include "sv_tree_common.cuh"

namespace sv {
namespace {

constexpr int kTvThreads = 256;
constexpr int kTvWarps = kTvThreads / 32;
constexpr int kTvMaxCluster = 16;
constexpr int64_t kL2Bytes = 126ll << 20;
constexpr int kTvCtasPerSm = 4;  // of a large batch; the clusters of a small one have two, with more registers

struct TreeVerifyParams {
    const void* target;
    const void* draft;
    const int32_t* tokens;
    const int32_t* parents;
    const int32_t* counts;
    const float* uniforms;
    double scale;  // log2(e) / T
    int32_t* out_len;
    int32_t* out_tok;
    int32_t* out_path;
    int32_t N, V, range;  // range: elements per warp, a multiple of a warp's vector step
    int64_t stride;
    bool ahead;  // rows come from DRAM and there is bandwidth to spare
};

struct Part {
    double s;  // sum of 2^((z - m) c)
    float m;   // its reference, -inf when it is empty
    int32_t i; // greedy: index of the maximum
};

// 2^(k/16), its bits less k << 48: adding (16 e + k) << 16 to the upper word
// then multiplies by 2^e.  Sixteen 64-bit entries lie in 32 banks once, so
// that no two lanes of a load are ever in conflict.
constexpr int kExp2Entries = 16;
__constant__ unsigned long long kExp2Table[kExp2Entries] = {
    0x3ff0000000000000ull, 0x3fefb5586cf9890full, 0x3fef72b83c7d517bull, 0x3fef387a6e756238ull,
    0x3fef06fe0a31b715ull, 0x3feedea64c123422ull, 0x3feebfdad5362a27ull, 0x3feeab07dd485429ull,
    0x3feea09e667f3bcdull, 0x3feea11473eb0187ull, 0x3feeace5422aa0dbull, 0x3feec49182a3f090ull,
    0x3feee89f995ad3adull, 0x3fef199bdd85529cull, 0x3fef5818dcfba487ull, 0x3fefa4afa2a490daull};

// Relative error of the 32-bit pass.  A weight 2^y has an error of 2^-21 from
// ex2 and of |y| 2^-22 ln2 from its argument (a rounded difference times a
// rounded scale): 6e-6 down to y = -30, and what lies lower weighs less than
// V 2^-30 altogether.  A lane adds at most 400 vectors, 2^-24 each; four
// joins (batch, lane, warp, CTA) rescale, 6e-6 each.
constexpr double kFastError = 1e-4;
constexpr float kFaint = -100.f;  // children below 2^-100 are left to the pass in 64 bits

struct TvShared {
    double tab[kExp2Entries];
    Part ex[2][kTvMaxCluster][2];    // [parity][rank][target, draft]: what the CTAs tell one another
    Part warp[2][kTvWarps];          // statistics of the warps' ranges
    double wp[kTvWarps];             // target sums of the warps' ranges, against the CTA's reference
    double wres[kTvWarps];           // residual sums of the warps' ranges
    double wscan[kTvWarps];
    double ce[SV_MAX_NODES], cq[SV_MAX_NODES];                    // the children's weights (draft logits)
    int32_t child[2][SV_MAX_NODES], ctok[2][SV_MAX_NODES], nchild[2];  // [parity of the level]
    int32_t par[SV_MAX_NODES], tok[SV_MAX_NODES];
    float u[SV_MAX_NODES];
    int32_t bad;
};

// ln2^k / k!, k = 5 .. 1.  From constant memory, where an operation can take
// them as they are; as literals each would be moved to registers first.
__constant__ double kExp2Poly[5] = {1.3333558146428443e-3, 9.6181291076284772e-3, 5.5504108664821580e-2,
                                    2.4022650695910072e-1, 6.9314718055994531e-1};

// 2^y, relative error below 2e-13: table of 2^(k/16) and the Taylor polynomial
// of degree 5 on |f| <= 1/32 (Tang's table-driven scheme; the remainder is
// (f ln2)^6 / 720).  A CDF that is off by 2e-13 moves a draw once in some ten
// million.  y in [-1000, 1000].
// In two factors: 2^n/16 with its exponent in place, and 2^f near 1 (a sum
// takes their product in one fused operation).
__device__ __forceinline__ void exp2_table(double y, const double* tab, double* b, double* q) {
    const double magic = 6755399441055744.0 / kExp2Entries;  // 1.5 2^52 / 16: rounds y to a multiple of 1/16
    const double t = y + magic;
    const double f = y - (t - magic);
    const int n = __double2loint(t);
    double p = kExp2Poly[0];
    p = fma(p, f, kExp2Poly[1]);
    p = fma(p, f, kExp2Poly[2]);
    p = fma(p, f, kExp2Poly[3]);
    p = fma(p, f, kExp2Poly[4]);
    *q = fma(p, f, 1.0);
    const double x = tab[n & (kExp2Entries - 1)];
    *b = __hiloint2double(__double2hiint(x) + (n << 16), __double2loint(x));
}

// Weight of z against the reference m: 0 where z is far below (or -inf).
__device__ __forceinline__ double bulk_weight(float z, float m, double c, float cf, const double* tab) {
    double b, q;
    exp2_table((static_cast<double>(z) - static_cast<double>(m)) * c, tab, &b, &q);
    return (z - m) * cf > -900.f ? b * q : 0.0;
}
// The same, not inlined: what runs once or twice per level waits for its
// instructions to be fetched more than for its arithmetic.
__device__ __noinline__ double weight(float z, float m, double c, float cf, const double* tab) {
    return bulk_weight(z, m, c, cf, tab);
}

__device__ __noinline__ double warp_sum(double v) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// s, held against the reference m, against the reference M >= m.
template <bool kExact>
__device__ __forceinline__ double rescale(double s, float m, float M, double c, float cf, const double* tab) {
    if (m == M) return s;  // also where both are -inf (s = 0)
    if (m == -INFINITY) return 0.0;
    return s * (kExact ? weight(m, M, c, cf, tab) : static_cast<double>(ex2_approx((m - M) * cf)));
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// A warp's range of a row, in batches of kUnroll 16-byte vectors per lane,
// kept as they were stored.  Element e of vector u is element
// base + u kStep + lane EV + e of the row; those at or past `hi` are -inf and
// are not loaded.
template <typename T, bool kVec, int kUnroll>
struct Batch {
    static constexpr int EV = Logit<T>::kPerVec;
    static constexpr int kStep = 32 * EV;              // elements of a warp's vector
    uint4 w[kUnroll];

    __device__ __forceinline__ void load(const void* row, int base, int hi, int lane) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int at = base + u * kStep;
            if (kVec && at + kStep <= hi) w[u] = __ldg(reinterpret_cast<const uint4*>(row) + at / EV + lane);
            else if (at < hi) w[u] = ragged(row, at + lane * EV, hi);
            else w[u] = uint4{kEmpty, kEmpty, kEmpty, kEmpty};
        }
    }
    static constexpr uint32_t kEmpty = EV == 4 ? 0xff800000u : 0xff80ff80u;
    // Elements [i, i + EV) of the row one by one, those from hi on as -inf.
    __device__ __noinline__ static uint4 ragged(const void* row, int i, int hi) {
        uint32_t x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int at = i + k * (EV / 4);
            if constexpr (EV == 4) {
                x[k] = at < hi ? __ldg(reinterpret_cast<const uint32_t*>(row) + at) : 0xff800000u;
            } else {
                const uint32_t lo = at < hi ? __ldg(reinterpret_cast<const unsigned short*>(row) + at) : 0xff80u;
                const uint32_t up = at + 1 < hi ? __ldg(reinterpret_cast<const unsigned short*>(row) + at + 1) : 0xff80u;
                x[k] = lo | up << 16;
            }
        }
        return uint4{x[0], x[1], x[2], x[3]};
    }
    // Takes the listed tokens out (few, and in few ranges).
    __device__ __forceinline__ void drop(const int32_t* tok, int n, int base, int lane) {
        for (int c = 0; c < n; ++c) {
            const int i = tok[c] - base - lane * EV;   // place behind this lane's first element
            if (i < 0) continue;
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                uint32_t x[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
                for (int e = 0; e < EV; ++e) {
                    if (i != u * kStep + e) continue;
                    if (EV == 4) x[e] = 0xff800000u;
                    else x[e / 2] = e % 2 ? (x[e / 2] & 0xffffu) | 0xff800000u : (x[e / 2] & 0xffff0000u) | 0xff80u;
                }
                w[u] = uint4{x[0], x[1], x[2], x[3]};
            }
        }
    }
    __device__ __forceinline__ float top() const {
        if constexpr (EV == 8) {  // two elements per instruction
            uint32_t m = w[0].x;
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                m = bf16x2_max(bf16x2_max(bf16x2_max(w[u].x, w[u].y), bf16x2_max(w[u].z, w[u].w)), m);
            return fmaxf(bf16_lo(m), bf16_hi(m));
        } else {
            float m = -INFINITY;
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                float f[EV];
                Logit<T>::unpack(w[u], f);
                m = fmaxf(m, fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3])));
            }
            return m;
        }
    }
};

// Statistics of a row's range [lo, hi) without the n listed tokens: reference
// and sum of the whole warp (every lane has them), in 64 bits (kExact) or to
// kFastError.  m is the reference to start from, the same in every lane, warp
// and CTA (some logit of the row; -inf: none).  The exponents' range leaves
// room above it, so it moves only past 2^600 (2^60 in 32 bits): nothing waits
// for a running maximum, and sums nearly always join without being rescaled.
template <typename T, bool kVec, bool kExact>
__device__ __forceinline__ Part range_stats(const void* row, int lo, int hi, const int32_t* drop, int n, float m,
                                            double c, const double* tab) {
    constexpr int kUnroll = kExact ? 2 : 4;  // 64 bits are bound by their arithmetic
    constexpr float kRoom = kExact ? 600.f : 60.f;
    using Sum = std::conditional_t<kExact, double, float>;
    using B = Batch<T, kVec, kUnroll>;
    const int lane = threadIdx.x & 31;
    const float cf = static_cast<float>(c);
    bool any = false;
    for (int k = lane; k < n; k += 32) any |= drop[k] >= lo && drop[k] < hi;
    any = __any_sync(0xffffffffu, any);
    float ref, least;
    double md, mc;
    bool near = false;
    auto refer = [&] {
        ref = m == -INFINITY ? 0.f : m;
        md = static_cast<double>(ref);
        mc = md * c;
        near = fabs(mc) < 4096.0;
        // Below 2^-900: nothing.  Rounded up, so that a logit is let in only where its exponent is
        // at least -900: at small temperatures one step of a float below the reference can be
        // past all that exp2_table holds.
        least = fmaxf(__fsub_ru(ref, 900.f / cf), -3.402823466e38f);
    };
    refer();
    Sum s[2] = {0, 0};
    for (int base = lo; base < hi; base += kUnroll * B::kStep) {
        B b;
        b.load(row, base, hi, lane);
        if (any) b.drop(drop, n, base, lane);
        const float bm = b.top();
        if ((bm - m) * cf > kRoom) {
            const Sum f = m == -INFINITY ? Sum(0) : Sum(rescale<kExact>(1.0, m, bm, c, cf, tab));
            s[0] *= f;
            s[1] *= f;
            m = bm;
            refer();
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (base + u * B::kStep >= hi) break;
            float z[B::EV];
            Logit<T>::unpack(b.w[u], z);
            if constexpr (kExact) {
                // one operation for y where rounding m c (the same for all) is below 2^-41, else two
                auto add = [&](auto y) {
#pragma unroll
                    for (int k = 0; k < B::EV; ++k) {
                        double x, q;
                        exp2_table(y(static_cast<double>(z[k])), tab, &x, &q);
                        if (z[k] >= least) s[k & 1] = fma(x, q, s[k & 1]);  // (q is NaN for -inf)
                    }
                };
                if (near) add([&](double v) { return fma(v, c, -mc); });
                else add([&](double v) { return (v - md) * c; });
            } else {
                float a[2] = {0.f, 0.f};
#pragma unroll
                for (int k = 0; k < B::EV; ++k) a[k & 1] += ex2_approx((z[k] - ref) * cf);
                s[u & 1] += a[0] + a[1];
            }
        }
    }
    Sum all = s[0] + s[1];
    float M = __shfl_sync(0xffffffffu, m, 0);
    if (!__all_sync(0xffffffffu, m == M)) {
        M = warp_max(m);
        all = static_cast<Sum>(rescale<kExact>(all, m, M, c, cf, tab));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    return Part{static_cast<double>(all), M, 0};
}

// Greedy: maximum and its lowest index.
template <typename T, bool kVec>
__device__ __forceinline__ Part range_argmax(const void* row, int lo, int hi) {
    using B = Batch<T, kVec, 4>;
    const int lane = threadIdx.x & 31;
    VI best{-INFINITY, 0x7fffffff};
    for (int base = lo; base < hi; base += 4 * B::kStep) {
        B b;
        b.load(row, base, hi, lane);
        const float bm = b.top();
        if (bm > best.v || base == lo) {  // the first place where it stands
            int at = 0x7fffffff;
#pragma unroll
            for (int u = 3; u >= 0; --u) {
                float z[B::EV];
                Logit<T>::unpack(b.w[u], z);
#pragma unroll
                for (int k = B::EV - 1; k >= 0; --k)
                    if (z[k] == bm) at = base + u * B::kStep + lane * B::EV + k;
            }
            best = VI{bm, at};
        }
    }
    best = warp_merge_vi(best);
    return Part{0.0, best.v, best.i};
}

// sum over [lo, hi) of max(0, p - l q)
template <typename T, bool kVec>
__device__ __forceinline__ double range_residual(const void* zr, const void* yr, int lo, int hi, float Mp, float Mq,
                                                 double ip, double lq, double c, const double* tab) {
    using B = Batch<T, kVec, 1>;
    const int lane = threadIdx.x & 31;
    const float cf = static_cast<float>(c);
    double s = 0.0;
    for (int base = lo; base < hi; base += B::kStep) {
        B a, b;
        a.load(zr, base, hi, lane);
        b.load(yr, base, hi, lane);
        float z[B::EV], y[B::EV];
        Logit<T>::unpack(a.w[0], z);
        Logit<T>::unpack(b.w[0], y);
#pragma unroll
        for (int k = 0; k < B::EV; ++k)
            s += fmax(0.0, bulk_weight(z[k], Mp, c, cf, tab) * ip - bulk_weight(y[k], Mq, c, cf, tab) * lq);
    }
    return warp_sum(s);
}

// The entry that holds `want` when n <= 32 weights (one per lane, 0 beyond)
// stand in a row: the first whose running sum exceeds it, else the last with
// weight, -1 when there is none.  *want becomes what is left within it.
__device__ __noinline__ int pick_entry(double w, int n, double* want, bool* passed = nullptr) {
    const int lane = threadIdx.x & 31;
    double incl = w;
    for (int o = 1; o < n; o <<= 1) {
        const double x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    const uint32_t has = __ballot_sync(0xffffffffu, lane < n && w > 0.0);
    const uint32_t hit = __ballot_sync(0xffffffffu, lane < n && w > 0.0 && incl > *want);
    const int at = hit ? __ffs(hit) - 1 : has ? 31 - __clz(has) : -1;
    const double before = __shfl_sync(0xffffffffu, incl, at > 0 ? at - 1 : 0);
    if (at > 0) *want -= before;
    if (passed) *passed = hit != 0;
    return at;
}

// Every CTA of a cluster, and after an exchange every warp of a CTA, takes
// the same decisions from the same numbers; nothing has to be told twice.
template <typename T, bool kVec, bool kGreedy, int kCtasPerSm>
__global__ void __launch_bounds__(kTvThreads, kCtasPerSm) tree_verify_kernel(const TreeVerifyParams prm) {
    __shared__ TvShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = static_cast<int>(cluster_ctarank()), C = static_cast<int>(cluster_nctarank());
    const int b = blockIdx.x / C;
    const int N = prm.N, V = prm.V;
    const double c = prm.scale;
    const float cf = static_cast<float>(c);

    if (tid < kExp2Entries) sh.tab[tid] = __longlong_as_double(kExp2Table[tid]);
    if (tid == 0) sh.bad = 0;
    cluster_barrier();  // every CTA of the cluster runs before any writes to another's shared memory
    grid_dependency_wait();
    const int count = prm.counts ? prm.counts[b] : N;
    for (int i = tid; i < N; i += kTvThreads) {
        const int p = i == 0 ? -1 : prm.parents ? prm.parents[int64_t(b) * N + i] : i - 1;
        const int t = i == 0 ? 0 : prm.tokens[int64_t(b) * N + i];
        sh.par[i] = p;
        sh.tok[i] = t;
        if (!kGreedy) sh.u[i] = prm.uniforms[int64_t(b) * N + i];
        if (i > 0 && i < count && (p < 0 || p >= i || t < 0 || t >= V)) sh.bad = 1;
    }
    if (tid == 0 && (count < 0 || count > N)) sh.bad = 1;
    __syncthreads();
    int32_t* out_tok = prm.out_tok + int64_t(b) * N;
    int32_t* out_path = prm.out_path + int64_t(b) * N;
    if (sh.bad || count == 0) {  // the same in every CTA of the cluster
        if (rank == 0) {
            for (int i = tid; i < N; i += kTvThreads) out_tok[i] = out_path[i] = -1;
            if (tid == 0) prm.out_len[b] = sh.bad ? -1 : 0;
        }
        return;
    }

    const int64_t lo64 = (int64_t(rank) * kTvWarps + warp) * prm.range;
    const int lo = static_cast<int>(lo64 < V ? lo64 : V);
    const int hi = lo + prm.range < V ? lo + prm.range : V;
    int node = 0, j = 0, parity = 0;

    // One part per lane: their common reference, and the lane's sum against it.
    auto common = [&](const Part& r, bool exact, float* M) {
        *M = __shfl_sync(0xffffffffu, r.m, 0);
        if (__all_sync(0xffffffffu, r.m == *M)) return r.s;
        *M = warp_max(r.m);
        return exact ? rescale<true>(r.s, r.m, *M, c, cf, sh.tab) : rescale<false>(r.s, r.m, *M, c, cf, sh.tab);
    };
    // What the warps found, merged and told to every CTA: warp 0 the target's
    // row, warp 1 the draft's.
    auto exchange = [&](int which, bool exact) {
        Part r = sh.warp[which][lane % kTvWarps];
        if (kGreedy) {
            VI v{r.m, r.i};
#pragma unroll
            for (int o = kTvWarps / 2; o > 0; o >>= 1)
                v = vi_better(v, VI{__shfl_xor_sync(0xffffffffu, v.v, o), __shfl_xor_sync(0xffffffffu, v.i, o)});
            r = Part{0.0, v.v, v.i};
        } else {
            float M;
            double s = common(r, exact, &M);
            if (which == 0 && lane < kTvWarps) sh.wp[lane] = s;
#pragma unroll
            for (int o = kTvWarps / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            r.s = s;
            r.m = M;
        }
        if (lane < C) {
            Part* at = &sh.ex[parity][rank][which];
            st_cluster_u64(&at->s, lane, __double_as_longlong(r.s));
            st_cluster_u64(&at->m, lane, uint64_t(__float_as_uint(r.m)) | uint64_t(static_cast<uint32_t>(r.i)) << 32);
        }
    };
    // The row's reference M and sum; *mine: the weight of CTA lane % C in it.
    auto row_sum = [&](int which, bool exact, float* M, double* mine) {
        double s = common(sh.ex[parity][lane & (C - 1)][which], exact, M);
        *mine = s;
        for (int o = C >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        return s;
    };

    for (;;) {
        const int lv = j & 1;  // the lists of a level live until the next one's are read
        const char* zr = reinterpret_cast<const char*>(prm.target) +
                         (int64_t(b) * N + node) * prm.stride * Logit<T>::kSize;
        const char* yr = reinterpret_cast<const char*>(prm.draft) +
                         (int64_t(b) * N + node) * prm.stride * Logit<T>::kSize;
        if (warp == 0) {  // the node's children, in order
            int n = 0;
            for (int i0 = 0; i0 < count; i0 += 32) {
                const int i = i0 + lane;
                const bool is = i > 0 && i < count && sh.par[i] == node;
                const uint32_t mask = __ballot_sync(0xffffffffu, is);
                if (is) {
                    const int k = n + __popc(mask & ((1u << lane) - 1u));
                    sh.child[lv][k] = i;
                    sh.ctok[lv][k] = sh.tok[i];
                }
                n += __popc(mask);
            }
            if (lane == 0) sh.nchild[lv] = n;
        }
        __syncthreads();
        const int nchild = sh.nchild[lv];
        const int32_t *child = sh.child[lv], *ctok = sh.ctok[lv];
        if (kCtasPerSm == 2 && prm.ahead && nchild > 0) {
            // the first child is the likeliest to be taken: its rows start on their way to L2
            const int64_t next = (int64_t(child[0]) - node) * prm.stride * Logit<T>::kSize;
            const int64_t from = lo * int64_t(Logit<T>::kSize), to = hi * int64_t(Logit<T>::kSize);
            for (int64_t i = from + lane * 128; i < to; i += 32 * 128) {
                prefetch_l2(zr + next + i);
                if (prm.draft) prefetch_l2(yr + next + i);
            }
        }
        int acc = -1;
        if constexpr (kGreedy) {
            const Part r = range_argmax<T, kVec>(zr, lo, hi);
            if (lane == 0) sh.warp[0][warp] = r;
            __syncthreads();
            if (warp == 0) exchange(0, false);
            cluster_barrier();
            VI g{sh.ex[parity][lane & (C - 1)][0].m, sh.ex[parity][lane & (C - 1)][0].i};
            for (int o = C >> 1; o > 0; o >>= 1)
                g = vi_better(g, VI{__shfl_xor_sync(0xffffffffu, g.v, o), __shfl_xor_sync(0xffffffffu, g.i, o)});
            parity ^= 1;
            for (int k0 = 0; k0 < nchild && acc < 0; k0 += 32) {
                const uint32_t hit = __ballot_sync(0xffffffffu, k0 + lane < nchild && ctok[k0 + lane] == g.i);
                if (hit) acc = k0 + __ffs(hit) - 1;
            }
            if (acc < 0) {
                if (rank == 0 && tid == 0) out_tok[j] = g.i < V ? g.i : 0;
                break;
            }
        } else {
            const bool use_q = prm.draft != nullptr && nchild > 0;
            const bool ids_only = prm.draft == nullptr;
            // The children's logits: lane k has child k's, in every warp (the few past 32 are read
            // again where they are needed).  The largest is the reference to start from; a leaf
            // takes the largest of the row's first 32.
            const bool mine_q = use_q && lane < nchild;
            const float cz = lane < nchild ? Logit<T>::load(zr, ctok[lane])
                                           : nchild == 0 && lane < V ? Logit<T>::load(zr, lane) : -INFINITY;
            const float cy = mine_q ? Logit<T>::load(yr, ctok[lane]) : -INFINITY;
            float Mp = cz, Mq = cy, Mcta = 0.f;
            for (int k = lane + 32; k < nchild; k += 32) Mp = fmaxf(Mp, Logit<T>::load(zr, ctok[k]));
            Mp = warp_max(Mp);
            if (use_q) Mq = warp_max(Mq);
            // First in 32 bits, then, where that does not settle it, in 64.
            double ip = 0.0, iq = 0.0, lam = 0.0, cta_p = 0.0, cta_r = 0.0;
            bool residual = false;
            for (bool exact = nchild == 0; acc < 0; exact = true) {
                for (int which = 0; which < (use_q ? 2 : 1); ++which) {
                    const char* row = which ? yr : zr;
                    const int ndrop = ids_only ? nchild : 0;
                    const float m = which ? Mq : Mp;
                    const Part r = exact ? range_stats<T, kVec, true>(row, lo, hi, ctok, ndrop, m, c, sh.tab)
                                         : range_stats<T, kVec, false>(row, lo, hi, ctok, ndrop, m, c, sh.tab);
                    if (lane == 0) sh.warp[which][warp] = r;
                }
                __syncthreads();
                if (warp < (use_q ? 2 : 1)) exchange(warp, exact);
                cluster_barrier();
                const double Sp = row_sum(0, exact, &Mp, &cta_p);
                Mcta = sh.ex[parity][rank][0].m;
                if (ids_only) {
                    // The mass before child k is what is not tried yet: base and the children from k
                    // on.  Children in lanes, chunks from the last to the first; -2: too near to tell.
                    const double above = exact ? 1.0 : 1.0 + kFastError, below = exact ? 1.0 : 1.0 - kFastError;
                    double rest = Sp;
                    for (int k0 = (nchild - 1) & ~31; k0 >= 0 && nchild > 0; k0 -= 32) {
                        const int k = k0 + lane, n = nchild - k0 < 32 ? nchild - k0 : 32;
                        const bool has = k < nchild;
                        const int t = has ? ctok[k] : -1;
                        bool again = false;  // a sibling's token again: nothing of it is left
                        for (int e = 0; e + 1 < n; ++e) {
                            const int other = __shfl_sync(0xffffffffu, t, e);
                            again |= lane > e && other == t;
                        }
                        for (int e = 0; e < k0; ++e) again |= ctok[e] == t;
                        double w = 0.0;
                        bool faint = false;  // too small for 32 bits
                        if (has && !again) {
                            const float z = k0 == 0 ? cz : Logit<T>::load(zr, t);
                            w = exact ? weight(z, Mp, c, cf, sh.tab) : static_cast<double>(ex2_approx((z - Mp) * cf));
                            faint = !exact && (z - Mp) * cf < kFaint;
                        }
                        double from = w;  // of the children from k on, in this chunk
                        for (int o = 1; o < n; o <<= 1) {
                            const double x = __shfl_down_sync(0xffffffffu, from, o);
                            if (lane + o < 32) from += x;
                        }
                        const double x = has ? static_cast<double>(sh.u[child[k]]) * (rest + from) : 0.0;
                        const uint32_t yes = __ballot_sync(0xffffffffu, has && x * above < w);
                        const uint32_t may = __ballot_sync(0xffffffffu, has && (x * below < w || faint));
                        if (may) acc = yes && __ffs(yes) == __ffs(may) ? k0 + __ffs(yes) - 1 : -2;
                        rest += __shfl_sync(0xffffffffu, from, 0);
                    }
                } else if (use_q) {
                    double cta_q;
                    const double Sq = row_sum(1, exact, &Mq, &cta_q);
                    if (!exact) {
                        // the first child's test: u q < p
                        const double x = static_cast<double>(sh.u[child[0]]) * ex2_approx((cy - Mq) * cf) * Sp;
                        const bool yes = x * (1.0 + 4.0 * kFastError) < ex2_approx((cz - Mp) * cf) * Sq &&
                                         (cy - Mq) * cf >= kFaint && (cz - Mp) * cf >= kFaint;
                        if (__shfl_sync(0xffffffffu, int(yes), 0)) acc = 0;
                    } else {
                        ip = 1.0 / Sp;
                        iq = 1.0 / Sq;
                        for (int k = tid; k < nchild; k += kTvThreads) {
                            sh.ce[k] = weight(Logit<T>::load(zr, ctok[k]), Mp, c, cf, sh.tab) * ip;
                            sh.cq[k] = weight(Logit<T>::load(yr, ctok[k]), Mq, c, cf, sh.tab) * iq;
                        }
                        __syncthreads();
                        double nrm = 1.0;
                        for (int k = 0; k < nchild; ++k) {
                            const double p = sh.ce[k], q = sh.cq[k];
                            if (static_cast<double>(sh.u[child[k]]) * nrm * q < fmax(0.0, p - lam * q)) {
                                acc = k;
                                break;
                            }
                            lam += nrm;
                            parity ^= 1;
                            const double w = range_residual<T, kVec>(zr, yr, lo, hi, Mp, Mq, ip, lam * iq, c, sh.tab);
                            if (lane == 0) sh.wres[warp] = w;
                            __syncthreads();
                            if (warp == 0) {
                                double t = sh.wres[lane % kTvWarps];
#pragma unroll
                                for (int o = kTvWarps / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
                                if (lane < C) st_cluster_u64(&sh.ex[parity][rank][0].s, lane, __double_as_longlong(t));
                            }
                            cluster_barrier();
                            cta_r = nrm = sh.ex[parity][lane & (C - 1)][0].s;
                            for (int o = C >> 1; o > 0; o >>= 1) nrm += __shfl_xor_sync(0xffffffffu, nrm, o);
                            residual = nrm > 0.0;
                        }
                    }
                }
                parity ^= 1;
                if (exact) break;
            }
            if (acc < 0) {
                // The final draw: CTA, then warp, then element (a residual without mass falls back to p).
                const double cta = lane < C ? (residual ? cta_r : cta_p) : 0.0;
                double W = cta;
                for (int o = kTvMaxCluster / 2; o > 0; o >>= 1) W += __shfl_xor_sync(0xffffffffu, W, o);
                double rest = static_cast<double>(sh.u[0]) * __shfl_sync(0xffffffffu, W, 0);
                const int owner = pick_entry(cta, C, &rest);
                if (owner < 0 && rank == 0 && tid == 0) out_tok[j] = nchild > 0 ? ctok[0] : 0;
                if (owner != rank) break;
                const double f = residual ? 1.0 : rescale<true>(1.0, Mcta, Mp, c, cf, sh.tab);
                const int from = pick_entry(lane < kTvWarps ? (residual ? sh.wres[lane] : sh.wp[lane]) * f : 0.0,
                                            kTvWarps, &rest);
                const int64_t rlo64 = (int64_t(rank) * kTvWarps + from) * prm.range;
                const int rlo = static_cast<int>(rlo64 < V ? rlo64 : V);
                const int rhi = rlo + prm.range < V ? rlo + prm.range : V;
                // thread i sums elements [i each, (i + 1) each) of the range
                const int each = (rhi - rlo + kTvThreads - 1) / kTvThreads;
                const int v0 = rlo + tid * each, v1 = v0 + each < rhi ? v0 + each : rhi;
                auto draw_weight = [&](int v) {
                    double w = weight(Logit<T>::load(zr, v), Mp, c, cf, sh.tab);
                    if (residual) w = fmax(0.0, w * ip - weight(Logit<T>::load(yr, v), Mq, c, cf, sh.tab) * (lam * iq));
                    if (ids_only)
                        for (int k = 0; k < nchild; ++k)
                            if (ctok[k] == v) w = 0.0;
                    return w;
                };
                double mine = 0.0;
#pragma unroll 1
                for (int v = v0; v < v1; ++v) mine += draw_weight(v);
                const double sum = warp_sum(mine);
                if (lane == 0) sh.wscan[warp] = sum;
                __syncthreads();
                const int at = pick_entry(lane < kTvWarps ? sh.wscan[lane] : 0.0, kTvWarps, &rest);
                if (at < 0 && tid == 0) out_tok[j] = rlo < V ? rlo : V - 1;
                if (warp == at) {
                    // that thread's elements, a lane each
                    const int src = pick_entry(mine, 32, &rest);
                    int t = rlo;
                    const int p0 = __shfl_sync(0xffffffffu, v0, src), p1 = __shfl_sync(0xffffffffu, v1, src);
#pragma unroll 1
                    for (int v = p0; v < p1; v += 32) {
                        const double w = v + lane < p1 ? draw_weight(v + lane) : 0.0;
                        const double all = warp_sum(w);
                        double left = rest;
                        bool passed;
                        const int i = pick_entry(w, 32, &left, &passed);
                        if (i >= 0) t = v + i;
                        if (passed) break;
                        rest -= all;
                    }
                    if (lane == 0) out_tok[j] = t;
                }
                break;
            }
        }
        node = child[acc];
        if (rank == 0 && tid == 0) {
            out_tok[j] = sh.tok[node];
            out_path[j + 1] = node;
        }
        ++j;
    }
    if (rank == 0) {
        for (int i = tid; i < N; i += kTvThreads) {
            if (i > j) out_tok[i] = out_path[i] = -1;
        }
        if (tid == 0) {
            out_path[0] = 0;
            prm.out_len[b] = j;
        }
    }
}

// CTAs per request: as many as let all requests run at once, no more than
// the row has 4 KiB pieces for.
int cluster_for(int B, int V, int es, int sms) {
    int c = kTvMaxCluster;
    while (c > 1 && (int64_t(B) * c > kTvCtasPerSm * int64_t(sms) || int64_t(c / 2) * 4096 >= int64_t(V) * es)) c /= 2;
    return c;
}

template <typename T, bool kVec, bool kGreedy>
cudaError_t launch(TreeVerifyParams prm, int B, cudaStream_t st) {
    TreeDevice dev;
    cudaError_t e = tree_device(&dev);
    if (e != cudaSuccess) return e;
    const int C = cluster_for(B, prm.V, Logit<T>::kSize, dev.sm_count);
    const bool roomy = int64_t(B) * C <= 2 * int64_t(dev.sm_count);
    constexpr auto few = &tree_verify_kernel<T, kVec, kGreedy, 2>, many = &tree_verify_kernel<T, kVec, kGreedy, kTvCtasPerSm>;
    const auto k = roomy ? few : many;
    if (C > 8) {
        e = roomy ? set_once<few>(dev, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)
                  : set_once<many>(dev, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    // Few requests over logits that L2 cannot hold: 12 chains of 39 nodes (V = 146376, fp32, with
    // draft logits) 268 us with rows brought ahead, 305 without; where L2 holds them it costs 0.5 us
    // in 13 to 2 in 26, and a large batch has no bandwidth left for it (92 us to 96).
    prm.ahead = roomy && int64_t(B) * prm.N * prm.stride * Logit<T>::kSize * (prm.draft ? 2 : 1) > kL2Bytes;
    const int step = Batch<T, kVec, 1>::kStep;  // a warp's vector
    const int64_t warps = int64_t(C) * kTvWarps;
    prm.range = static_cast<int>(((prm.V + warps - 1) / warps + step - 1) / step * step);
    return launch_dependent(k, dim3(static_cast<unsigned>(int64_t(B) * C)), kTvThreads, 0, C, st, prm);
}

}  // namespace
}  // namespace sv

extern "C" sv_status sv_tree_verify(const sv_tree_shape* s, const void* target, const void* draft,
                                    const int32_t* tokens, const int32_t* parents, const int32_t* counts,
                                    const float* uniforms, double temperature, int32_t greedy,
                                    int32_t* out_accept_len, int32_t* out_tokens, int32_t* out_path, void* stream) {
    using namespace sv;
    if (!s || s->B < 0 || s->N < 1 || s->V < 1) return SV_EINVAL;
    if (s->dtype != SV_F32 && s->dtype != SV_BF16) return SV_EUNSUPPORTED;
    if (s->N > SV_MAX_NODES || s->V > SV_MAX_V) return SV_EUNSUPPORTED;
    const int64_t stride = s->row_stride ? s->row_stride : s->V;
    if (stride < s->V) return SV_EINVAL;
    if (s->B == 0) return SV_OK;  // (an empty tensor's pointer may be null)
    if (!target || !tokens || !out_accept_len || !out_tokens || !out_path) return SV_EINVAL;
    if (!greedy && (!uniforms || !(temperature > 0.0) || !std::isfinite(temperature) ||
                    !std::isnormal(static_cast<float>(1.4426950408889634 / temperature))))
        return SV_EINVAL;
    if (int64_t(s->B) * kTvMaxCluster > 0x7fffffff) return SV_EUNSUPPORTED;
    const int es = s->dtype == SV_BF16 ? 2 : 4;
    const bool vec = tree_aligned16(target) && (greedy || tree_aligned16(draft)) && stride * es % 16 == 0;
    TreeVerifyParams prm{target, greedy ? nullptr : draft, tokens, parents, counts, uniforms,
                         greedy ? 1.0 : 1.4426950408889634 / temperature, out_accept_len, out_tokens, out_path,
                         s->N, s->V, 0, stride, false};
    auto st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (s->dtype == SV_BF16) {
        using T = bf16_bits;
        e = greedy ? (vec ? launch<T, true, true>(prm, s->B, st) : launch<T, false, true>(prm, s->B, st))
                   : (vec ? launch<T, true, false>(prm, s->B, st) : launch<T, false, false>(prm, s->B, st));
    } else {
        using T = float;
        e = greedy ? (vec ? launch<T, true, true>(prm, s->B, st) : launch<T, false, true>(prm, s->B, st))
                   : (vec ? launch<T, true, false>(prm, s->B, st) : launch<T, false, false>(prm, s->B, st));
    }
    return e == cudaSuccess ? SV_OK : SV_ECUDA;
}
