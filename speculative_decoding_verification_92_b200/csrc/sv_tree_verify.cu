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
// that, and one draw in some hundred would pick a neighbouring token.
//
// Bound.  Only rows on the accepted path are read, so a step is a chain of
// visits: load latency, the arithmetic of one row, one cluster barrier.  The
// CTAs of a cluster split the vocabulary; the more requests, the smaller the
// cluster, so that all of them run at once (cluster_for).  A warp owns one
// contiguous range of the row, which is the unit the final draw looks up.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "sv_tree.h"
#include "sv_tree_common.cuh"

namespace sv {
namespace {

constexpr int kTvThreads = 256;
constexpr int kTvWarps = kTvThreads / 32;
constexpr int kTvMaxCluster = 16;
constexpr int kTvUnroll = 4;  // 16-byte loads in flight per lane

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
};

struct Part {
    double s;  // sum of 2^((z - m) c)
    float m;   // its reference, -inf when it is empty
    int32_t i; // greedy: index of the maximum
};

struct TvShared {
    double tab[32];                       // 2^(k/32)
    Part ex[2][kTvMaxCluster][2];         // [parity][rank][target, draft]: what the CTAs tell one another
    Part warp[2][kTvWarps];               // statistics of the warps' ranges
    double wres[kTvWarps];                // residual sums of the warps' ranges
    double cta_p[kTvMaxCluster];          // weight of each CTA: of the row,
    double cta_r[kTvMaxCluster];          // of the residual
    double ce[SV_MAX_NODES], cq[SV_MAX_NODES];
    float cz[SV_MAX_NODES], cy[SV_MAX_NODES];
    int32_t par[SV_MAX_NODES], tok[SV_MAX_NODES];
    int32_t child[SV_MAX_NODES], ctok[SV_MAX_NODES];
    double S[2], wscan[kTvWarps];
    float M[2], u[SV_MAX_NODES];
    int32_t nchild, accepted, bad, pick;
};

// 2^y for y <= 0 or moderately above, relative error about 2^-52: table of
// 2^(k/32) and a polynomial on |f| <= 1/64 (Tang's table-driven scheme; its
// remainder (f ln2)^6 / 720 is below 2e-15).  y in [-1000, 1000].
__device__ __forceinline__ double exp2_table(double y, const double* tab) {
    const double magic = 6755399441055744.0 / 32.0;  // 1.5 * 2^52 / 32: rounds y to a multiple of 1/32
    const double t = y + magic;
    const double f = y - (t - magic);
    const int n = __double2loint(t);
    double p = 1.3333558146428443e-3;                // ln2^k / k!, k = 5 .. 1
    p = fma(p, f, 9.6181291076284772e-3);
    p = fma(p, f, 5.5504108664821580e-2);
    p = fma(p, f, 2.4022650695910072e-1);
    p = fma(p, f, 6.9314718055994531e-1);
    const double b = tab[n & 31];
    const double r = fma(b * f, p, b);
    return __hiloint2double(__double2hiint(r) + ((n >> 5) << 20), __double2loint(r));
}

// Weight of z against the reference m: 0 where z is far below (or -inf).
__device__ __forceinline__ double weight(float z, float m, double c, float cf, const double* tab) {
    const double y = (static_cast<double>(z) - static_cast<double>(m)) * c;
    const double w = exp2_table(y, tab);
    return (z - m) * cf > -900.f ? w : 0.0;
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// One batch of a warp's range: kTvUnroll vectors per lane from element `base`
// on, as fp32; elements at or past `hi` are -inf and are not read.  Element
// j of vector u is element index(base, u, lane) + j of the row (kVec), or the
// lane-interleaved order for rows without 16-byte alignment.
template <typename T, bool kVec>
struct Batch {
    static constexpr int EV = Logit<T>::kPerVec;
    static constexpr int kElems = EV * kTvUnroll;      // per lane
    static constexpr int kStep = 32 * kElems;          // per warp
    float z[kElems];

    __device__ __forceinline__ static int index(int base, int k, int lane) {
        return kVec ? base + (k / EV) * (32 * EV) + lane * EV + k % EV : base + k * 32 + lane;
    }
    // Whether vector u of this batch lies (for some lane) before `hi`.
    __device__ __forceinline__ static bool live(int base, int u, int hi) { return base + u * 32 * EV < hi; }
    __device__ __forceinline__ void load(const void* row, int base, int hi, int lane) {
        uint4 w[kTvUnroll];
        const uint4* p = reinterpret_cast<const uint4*>(row) + base / EV + lane;
#pragma unroll
        for (int u = 0; u < kTvUnroll; ++u)
            if (kVec && live(base, u + 1, hi + 1)) w[u] = __ldg(p + u * 32);
#pragma unroll
        for (int u = 0; u < kTvUnroll; ++u) {
            if (kVec && live(base, u + 1, hi + 1)) {
                float f[EV];
                Logit<T>::unpack(w[u], f);
#pragma unroll
                for (int e = 0; e < EV; ++e) z[u * EV + e] = f[e];
            } else {
#pragma unroll
                for (int e = 0; e < EV; ++e) {
                    const int i = index(base, u * EV + e, lane);
                    z[u * EV + e] = i < hi ? Logit<T>::load(row, i) : -INFINITY;
                }
            }
        }
    }
    // Takes the listed tokens out (one of `n` at a time; rare).
    __device__ __forceinline__ void drop(const int32_t* tok, int n, int base, int lane) {
        for (int c = 0; c < n; ++c) {
            const int t = tok[c];
            if (t < base || t >= base + kStep) continue;
#pragma unroll
            for (int k = 0; k < kElems; ++k)
                if (index(base, k, lane) == t) z[k] = -INFINITY;
        }
    }
};

// Statistics of a row's range [lo, hi) without the n listed tokens: reference
// and sum of the whole warp (every lane has them).
template <typename T, bool kVec>
__device__ Part range_stats(const void* row, int lo, int hi, const int32_t* drop, int n, double c, const double* tab) {
    using B = Batch<T, kVec>;
    const int lane = threadIdx.x & 31;
    const float cf = static_cast<float>(c);
    bool any = false;
    for (int k = lane; k < n; k += 32) any |= drop[k] >= lo && drop[k] < hi;
    any = __any_sync(0xffffffffu, any);
    float m = -INFINITY;
    double s = 0.0;
    for (int base = lo; base < hi; base += B::kStep) {
        B b;
        b.load(row, base, hi, lane);
        if (any) b.drop(drop, n, base, lane);
        float bm = b.z[0];
#pragma unroll
        for (int k = 1; k < B::kElems; ++k) bm = fmaxf(bm, b.z[k]);
        if (bm > m) {
            s = m == -INFINITY ? 0.0 : s * weight(m, bm, c, cf, tab);
            m = bm;
        }
        if (m != -INFINITY) {
#pragma unroll
            for (int u = 0; u < kTvUnroll; ++u) {
                if (!B::live(base, u, hi)) break;
                double a[2] = {0.0, 0.0};
#pragma unroll
                for (int e = 0; e < B::EV; ++e) a[e & 1] += weight(b.z[u * B::EV + e], m, c, cf, tab);
                s += a[0] + a[1];
            }
        }
    }
    const float M = warp_max(m);
    if (m != -INFINITY) s *= weight(m, M, c, cf, tab);
    return Part{warp_sum(s), M, 0};
}

// Greedy: maximum and its lowest index.
template <typename T, bool kVec>
__device__ Part range_argmax(const void* row, int lo, int hi) {
    using B = Batch<T, kVec>;
    const int lane = threadIdx.x & 31;
    VI best{-INFINITY, 0x7fffffff};
    for (int base = lo; base < hi; base += B::kStep) {
        B b;
        b.load(row, base, hi, lane);
#pragma unroll
        for (int k = 0; k < B::kElems; ++k) best = vi_better(best, VI{b.z[k], B::index(base, k, lane)});
    }
    best = warp_merge_vi(best);
    return Part{0.0, best.v, best.i};
}

// sum over [lo, hi) of max(0, p - l q)
template <typename T, bool kVec>
__device__ double range_residual(const void* zr, const void* yr, int lo, int hi, float Mp, float Mq, double ip,
                                 double lq, double c, const double* tab) {
    using B = Batch<T, kVec>;
    const int lane = threadIdx.x & 31;
    const float cf = static_cast<float>(c);
    double s = 0.0;
    for (int base = lo; base < hi; base += B::kStep) {
        B a, b;
        a.load(zr, base, hi, lane);
        b.load(yr, base, hi, lane);
#pragma unroll
        for (int u = 0; u < kTvUnroll; ++u) {
            if (!B::live(base, u, hi)) break;
#pragma unroll
            for (int k = u * B::EV; k < (u + 1) * B::EV; ++k)
                s += fmax(0.0, weight(a.z[k], Mp, c, cf, tab) * ip - weight(b.z[k], Mq, c, cf, tab) * lq);
        }
    }
    return warp_sum(s);
}

template <typename T, bool kVec, bool kGreedy>
__global__ void __launch_bounds__(kTvThreads) tree_verify_kernel(const TreeVerifyParams prm) {
    __shared__ TvShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_ctarank(), C = cluster_nctarank();
    const int b = blockIdx.x / C;
    const int N = prm.N, V = prm.V;
    const double c = prm.scale;
    const float cf = static_cast<float>(c);

    if (tid < 32) sh.tab[tid] = exp2(tid / 32.0);
    if (tid == 0) sh.bad = 0;
    cluster_barrier();  // every CTA of the cluster runs before any writes to another's shared memory
    grid_dependency_wait();
    const int count = prm.counts ? prm.counts[b] : N;
    if (count < 0 || count > N) {
        if (tid == 0) sh.bad = 1;
    } else {
        for (int i = tid; i < count; i += kTvThreads) {
            const int p = i == 0 ? -1 : prm.parents ? prm.parents[int64_t(b) * N + i] : i - 1;
            const int t = i == 0 ? 0 : prm.tokens[int64_t(b) * N + i];
            sh.par[i] = p;
            sh.tok[i] = t;
            if (!kGreedy) sh.u[i] = prm.uniforms[int64_t(b) * N + i];
            if (i > 0 && (p < 0 || p >= i || t < 0 || t >= V)) sh.bad = 1;
        }
    }
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

    // What each warp found, merged per CTA and told to every CTA.
    auto exchange = [&](int which) {
        if (warp == 0 && lane < static_cast<int>(C)) {
            Part r = sh.warp[which][0];
            if (kGreedy) {
                for (int w = 1; w < kTvWarps; ++w) {
                    const VI v = vi_better(VI{r.m, r.i}, VI{sh.warp[which][w].m, sh.warp[which][w].i});
                    r.m = v.v;
                    r.i = v.i;
                }
            } else {
                for (int w = 1; w < kTvWarps; ++w) r.m = fmaxf(r.m, sh.warp[which][w].m);
                r.s = 0.0;
                for (int w = 0; w < kTvWarps; ++w)
                    if (sh.warp[which][w].m != -INFINITY)
                        r.s += sh.warp[which][w].s * weight(sh.warp[which][w].m, r.m, c, cf, sh.tab);
            }
            Part* at = &sh.ex[parity][rank][which];
            st_cluster_u64(&at->s, lane, __double_as_longlong(r.s));
            st_cluster_u64(&at->m, lane,
                           uint64_t(__float_as_uint(r.m)) | uint64_t(static_cast<uint32_t>(r.i)) << 32);
        }
    };

    for (;;) {
        const char* zr = reinterpret_cast<const char*>(prm.target) +
                         (int64_t(b) * N + node) * prm.stride * Logit<T>::kSize;
        const char* yr = reinterpret_cast<const char*>(prm.draft) +
                         (int64_t(b) * N + node) * prm.stride * Logit<T>::kSize;
        // the node's children, in order
        if (warp == 0) {
            int n = 0;
            for (int i0 = 0; i0 < count; i0 += 32) {
                const int i = i0 + lane;
                const bool is = i > 0 && i < count && sh.par[i] == node;
                const uint32_t mask = __ballot_sync(0xffffffffu, is);
                if (is) {
                    const int k = n + __popc(mask & ((1u << lane) - 1u));
                    sh.child[k] = i;
                    sh.ctok[k] = sh.tok[i];
                }
                n += __popc(mask);
            }
            if (lane == 0) sh.nchild = n;
        }
        __syncthreads();
        const int nchild = sh.nchild;
        const bool use_q = !kGreedy && prm.draft != nullptr && nchild > 0;
        const bool ids_only = !kGreedy && prm.draft == nullptr;
        if (kGreedy) {
            const Part r = range_argmax<T, kVec>(zr, lo, hi);
            if (lane == 0) sh.warp[0][warp] = r;
        } else {
            for (int k = tid; k < nchild; k += kTvThreads) {
                sh.cz[k] = Logit<T>::load(zr, sh.ctok[k]);
                if (use_q) sh.cy[k] = Logit<T>::load(yr, sh.ctok[k]);
            }
            const Part r = range_stats<T, kVec>(zr, lo, hi, sh.ctok, ids_only ? nchild : 0, c, sh.tab);
            if (lane == 0) sh.warp[0][warp] = r;
            if (use_q) {
                const Part q = range_stats<T, kVec>(yr, lo, hi, sh.ctok, 0, c, sh.tab);
                if (lane == 0) sh.warp[1][warp] = q;
            }
        }
        __syncthreads();
        exchange(0);
        if (use_q) exchange(1);
        cluster_barrier();

        if (kGreedy) {
            VI g{sh.ex[parity][0][0].m, sh.ex[parity][0][0].i};
            for (int r = 1; r < static_cast<int>(C); ++r)
                g = vi_better(g, VI{sh.ex[parity][r][0].m, sh.ex[parity][r][0].i});
            int next = -1;
            for (int k = 0; k < nchild && next < 0; ++k)
                if (sh.ctok[k] == g.i) next = sh.child[k];
            parity ^= 1;
            if (next < 0) {
                if (rank == 0 && tid == 0) out_tok[j] = g.i < V ? g.i : 0;
                break;
            }
            if (rank == 0 && tid == 0) {
                out_tok[j] = sh.tok[next];
                out_path[j + 1] = next;
            }
            node = next;
            ++j;
            __syncthreads();
            continue;
        }

        // row sums, and the children's weights against the row's reference
        if (warp < (use_q ? 2 : 1)) {
            Part r{0.0, -INFINITY, 0};
            if (lane < static_cast<int>(C)) r = sh.ex[parity][lane][warp];
            float M = r.m;
            if (warp == 0 && ids_only)
                for (int k = lane; k < nchild; k += 32) M = fmaxf(M, sh.cz[k]);
            M = warp_max(M);
            const double s = r.m == -INFINITY ? 0.0 : r.s * weight(r.m, M, c, cf, sh.tab);
            if (warp == 0 && lane < kTvMaxCluster) sh.cta_p[lane] = s;
            const double S = warp_sum(s);
            if (lane == 0) {
                sh.M[warp] = M;
                sh.S[warp] = S;
            }
            for (int k = lane; k < nchild; k += 32) {
                bool again = false;  // an earlier sibling's token: nothing of it is left
                if (ids_only)
                    for (int e = 0; e < k; ++e) again |= sh.ctok[e] == sh.ctok[k];
                const double w = again ? 0.0 : weight(warp == 0 ? sh.cz[k] : sh.cy[k], M, c, cf, sh.tab);
                if (warp == 0) sh.ce[k] = w;
                else sh.cq[k] = w;
            }
            __syncwarp();
            if (warp == 0 && ids_only && lane == 0) {
                // the mass before child k is what is not tried yet: base and the children from k on
                double rest = S;
                int acc = -1;
                for (int k = nchild - 1; k >= 0; --k) {
                    rest += sh.ce[k];
                    if (static_cast<double>(sh.u[sh.child[k]]) * rest < sh.ce[k]) acc = k;
                }
                sh.accepted = acc;
            }
        }
        __syncthreads();
        const float Mp = sh.M[0], Mq = sh.M[1];
        const double ip = 1.0 / sh.S[0], iq = use_q ? 1.0 / sh.S[1] : 0.0;
        parity ^= 1;
        int acc = ids_only ? sh.accepted : -1;
        double lam = 0.0;
        bool residual = false;
        if (use_q) {
            double nrm = 1.0;
            for (int k = 0; k < nchild; ++k) {
                const double p = sh.ce[k] * ip, q = sh.cq[k] * iq;
                if (static_cast<double>(sh.u[sh.child[k]]) * nrm * q < fmax(0.0, p - lam * q)) {
                    acc = k;
                    break;
                }
                lam += nrm;
                const double w = range_residual<T, kVec>(zr, yr, lo, hi, Mp, Mq, ip, lam * iq, c, sh.tab);
                if (lane == 0) sh.wres[warp] = w;
                __syncthreads();
                if (warp == 0 && lane < static_cast<int>(C)) {
                    double t = 0.0;
                    for (int i = 0; i < kTvWarps; ++i) t += sh.wres[i];
                    st_cluster_u64(&sh.ex[parity][rank][0].s, lane, __double_as_longlong(t));
                }
                cluster_barrier();
                nrm = 0.0;
                for (uint32_t r = 0; r < C; ++r) nrm += sh.ex[parity][r][0].s;
                residual = nrm > 0.0;
                if (residual && tid < static_cast<int>(C)) sh.cta_r[tid] = sh.ex[parity][tid][0].s;
                parity ^= 1;
            }
            __syncthreads();
        }
        if (acc >= 0) {
            node = sh.child[acc];
            if (rank == 0 && tid == 0) {
                out_tok[j] = sh.tok[node];
                out_path[j + 1] = node;
            }
            ++j;
            __syncthreads();  // the lists are rebuilt
            continue;
        }

        // The final draw: CTA, then warp, then element.
        // (a residual without mass falls back to p)
        const double* cta_w = residual ? sh.cta_r : sh.cta_p;
        double W = 0.0;
        for (uint32_t r = 0; r < C; ++r) W += cta_w[r];
        const double want = static_cast<double>(sh.u[0]) * W;
        double before = 0.0, rest = 0.0;
        int owner = -1;
        {
            double cum = 0.0;
            for (int r = 0; r < static_cast<int>(C); ++r) {
                const double w = cta_w[r];
                if (w > 0.0) {
                    owner = r;
                    before = cum;
                }
                cum += w;
                if (cum > want) break;
            }
            rest = want - before;
        }
        if (owner < 0 && rank == 0 && tid == 0) out_tok[j] = nchild > 0 ? sh.ctok[0] : 0;
        if (owner != static_cast<int>(rank)) break;
        int from = 0;
        {
            double cum = 0.0, left = 0.0;
            for (int w = 0; w < kTvWarps; ++w) {
                double x;
                if (residual) x = sh.wres[w];
                else x = sh.warp[0][w].m == -INFINITY ? 0.0
                                                      : sh.warp[0][w].s * weight(sh.warp[0][w].m, Mp, c, cf, sh.tab);
                if (x > 0.0) {
                    from = w;
                    left = cum;
                }
                cum += x;
                if (cum > rest) break;
            }
            rest -= left;
        }
        const int64_t rlo64 = (int64_t(rank) * kTvWarps + from) * prm.range;
        const int rlo = static_cast<int>(rlo64 < V ? rlo64 : V);
        const int rhi = rlo + prm.range < V ? rlo + prm.range : V;
        const int each = (rhi - rlo + kTvThreads - 1) / kTvThreads;
        auto draw_weight = [&](int v) {
            double w = weight(Logit<T>::load(zr, v), Mp, c, cf, sh.tab);
            if (residual) return fmax(0.0, w * ip - weight(Logit<T>::load(yr, v), Mq, c, cf, sh.tab) * (lam * iq));
            if (ids_only)
                for (int k = 0; k < nchild; ++k)
                    if (sh.ctok[k] == v) w = 0.0;
            return w;
        };
        const int v0 = rlo + tid * each, v1 = v0 + each < rhi ? v0 + each : rhi;
        double mine = 0.0;
        for (int v = v0; v < v1; ++v) mine += draw_weight(v);
        double incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        if (lane == 31) sh.wscan[warp] = incl;
        if (tid == 0) sh.pick = 0x7fffffff;
        __syncthreads();
        for (int w = 0; w < warp; ++w) incl += sh.wscan[w];
        // the first thread whose running sum passes; else the last with weight
        if (mine > 0.0 && incl > rest) atomicMin(&sh.pick, tid);
        __syncthreads();
        if (sh.pick == 0x7fffffff) {
            __syncthreads();
            if (tid == 0) sh.pick = -1;
            __syncthreads();
            if (mine > 0.0) atomicMax(&sh.pick, tid);
            __syncthreads();
        }
        if (tid == sh.pick) {
            double run = incl - mine;
            int t = v0;
            for (int v = v0; v < v1; ++v) {
                const double w = draw_weight(v);
                run += w;
                if (w > 0.0) {
                    t = v;
                    if (run > rest) break;
                }
            }
            out_tok[j] = t;
        }
        break;
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

// CTAs per request: as many as let all requests run at once (two CTAs per
// SM), no more than the row has 4 KiB pieces for.
int cluster_for(int B, int V, int es, int sms) {
    int c = kTvMaxCluster;
    while (c > 1 && (int64_t(B) * c > 2 * int64_t(sms) || int64_t(c / 2) * 4096 >= int64_t(V) * es)) c /= 2;
    return c;
}

template <typename T, bool kVec, bool kGreedy>
cudaError_t launch(TreeVerifyParams prm, int B, cudaStream_t st) {
    auto k = tree_verify_kernel<T, kVec, kGreedy>;
    TreeDevice dev;
    cudaError_t e = tree_device(&dev);
    if (e != cudaSuccess) return e;
    const int C = cluster_for(B, prm.V, Logit<T>::kSize, dev.sm_count);
    if (C > 8) {
        e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    const int step = Batch<T, kVec>::kStep / kTvUnroll;  // a warp's vector step
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
    if (!target || !tokens || !out_accept_len || !out_tokens || !out_path) return SV_EINVAL;
    if (!greedy && (!uniforms || !(temperature > 0.0) || !std::isfinite(temperature) ||
                    !std::isfinite(1.4426950408889634 / temperature)))
        return SV_EINVAL;
    if (s->B == 0) return SV_OK;
    if (int64_t(s->B) * kTvMaxCluster > 0x7fffffff) return SV_EUNSUPPORTED;
    const int es = s->dtype == SV_BF16 ? 2 : 4;
    const bool vec = tree_aligned16(target) && (greedy || tree_aligned16(draft)) && stride * es % 16 == 0;
    TreeVerifyParams prm{target, greedy ? nullptr : draft, tokens, parents, counts, uniforms,
                         greedy ? 1.0 : 1.4426950408889634 / temperature, out_accept_len, out_tokens, out_path,
                         s->N, s->V, 0, stride};
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
