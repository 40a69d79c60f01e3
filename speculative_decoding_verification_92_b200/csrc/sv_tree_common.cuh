// sv_tree_common.cuh -- what the kernels of the tree operators share: cluster
// barriers and distributed-shared-memory stores, programmatic launches, and
// the host-side facts of the current device.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "sv_common.cuh"

namespace sv {

__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;"); }

__device__ __forceinline__ uint32_t cluster_ctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_nctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// All threads of all CTAs of the cluster; orders shared-memory accesses.
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 8 bytes into the shared memory of CTA `rank` of the cluster, at the place
// that `p` has in this CTA.
__device__ __forceinline__ void st_cluster_u64(void* p, uint32_t rank, uint64_t v) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// ---------------------------------------------------------------------------
// Host side.  (Internal linkage: what a copy of the library remembers about
// its kernels does not hold for another copy in the same process.)
namespace {

constexpr int kKnownDevices = 64;  // facts of devices past these are asked for in every call

struct TreeDevice {
    int index = 0, sm_count = 0;
};

inline cudaError_t tree_device(TreeDevice* d) {
    static std::atomic<int> sms[kKnownDevices];
    cudaError_t e = cudaGetDevice(&d->index);
    if (e != cudaSuccess) return e;
    const bool known = d->index < kKnownDevices;
    d->sm_count = known ? sms[d->index].load(std::memory_order_relaxed) : 0;
    if (d->sm_count > 0) return cudaSuccess;
    e = cudaDeviceGetAttribute(&d->sm_count, cudaDevAttrMultiProcessorCount, d->index);
    if (e == cudaSuccess && known) sms[d->index].store(d->sm_count, std::memory_order_relaxed);
    return e;
}

// The current context's id, which no later context has again; 0 where the
// driver cannot tell.
inline unsigned long long tree_context() {
    using GetCurrent = int (*)(void**);
    using GetId = int (*)(void*, unsigned long long*);
    auto entry = [](const char* name) {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        return cudaGetDriverEntryPoint(name, &f, cudaEnableDefault, &q) == cudaSuccess &&
                       q == cudaDriverEntryPointSuccess ? f : nullptr;
    };
    static const GetCurrent get_current = reinterpret_cast<GetCurrent>(entry("cuCtxGetCurrent"));
    static const GetId get_id = reinterpret_cast<GetId>(entry("cuCtxGetId"));
    void* context = nullptr;
    unsigned long long id = 0;
    if (!get_current || !get_id || get_current(&context) != 0 || !context || get_id(context, &id) != 0) return 0;
    return id;
}

// Sets an attribute that kernel `kKernel` needs, once per device and context
// (attributes live in the context).
template <auto kKernel>
cudaError_t set_once(const TreeDevice& d, cudaFuncAttribute attribute, int value) {
    static std::atomic<unsigned long long> set_in[kKnownDevices];
    const unsigned long long context = d.index < kKnownDevices ? tree_context() : 0;
    if (context != 0 && set_in[d.index].load(std::memory_order_relaxed) == context) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kKernel, attribute, value);
    if (e == cudaSuccess && context != 0) set_in[d.index].store(context, std::memory_order_relaxed);
    return e;
}

// Launch as a programmatic dependent of the work before it (the kernel waits
// with grid_dependency_wait), in clusters of `cluster` CTAs.
template <typename Kernel, typename... Args>
cudaError_t launch_dependent(Kernel k, dim3 grid, int threads, size_t smem, int cluster, cudaStream_t st,
                             const Args&... args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k, args...);
}

}  // namespace

inline bool tree_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace sv
