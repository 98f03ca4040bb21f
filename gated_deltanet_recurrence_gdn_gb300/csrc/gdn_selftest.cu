// gdn_selftest.cu -- device self-test of the bounded waits (gdn_selftest.h).
//
// One CTA waits, through the control block the pipelined kernels use (Ctl),
// on an mbarrier phase and on a release/acquire counter in shared memory.
// Either the CTA completes both itself before waiting (the waits must
// succeed, no error recorded), or nothing ever completes them (each wait
// must give up after its poll limit and record a timeout in the device error
// word).  No fault, trap or unbounded loop is involved: the failure is a
// phase that nobody completes, and the kernel always returns.
#include <cuda_runtime.h>

#include "gdn.h"
#include "gdn_selftest.h"
#include "gdn_internal.h"
#include "gdn_kv_attn.cuh"
#include "tc_common.cuh"

namespace gdn {
namespace {

constexpr long long kMaxSelftestLimit = 1LL << 22;

// whether each wait succeeded (1) or gave up (0), for the host to read back
__device__ int g_selftest_out[2];

__global__ void __launch_bounds__(32, 1)
k_wait_selftest(int complete, uint32_t limit, int *err, int *out) {
    __shared__ uint64_t bar[1];
    __shared__ uint32_t counter;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        ptx::mbar_init(bar, 1);
        counter = 0;
        abort_flag = 0;
        ptx::fence_mbar_init();
    }
    __syncthreads();
    if (threadIdx.x != 0) return;
    if (complete) {
        ptx::mbar_arrive(bar);              // the one expected arrival: phase 0 completes
        ptx::st_release_cta(&counter, 1u);
    }
    const tcx::Ctl ctl{bar, &abort_flag, err, limit};
    const bool bar_ok = ctl.wait(0, 0);
    abort_flag = 0;                         // let the second wait run as well
    const bool flag_ok = ctl.flag(&counter, 1u);
    out[0] = bar_ok ? 1 : 0;
    out[1] = flag_ok ? 1 : 0;
}

constexpr int kRingThreads = 256;
constexpr int kRingStages = 3, kRingWords = 1024;
constexpr int kRingAt = 128, kRingSmem = kRingAt + kRingStages * kRingWords * 4;
__device__ int g_ring_out[3];
__device__ __align__(16) uint32_t g_ring_src[kRingWords];

// The attention kernels' waits (kv::Waits), by eight warps on a phase that the CTA
// completes itself or that nothing completes, and once more on the same phase: how
// many threads found it complete each time.  Before that two copies are sent into a
// ring, which nobody waits for but its drain: how many of their words are there then.
__global__ void __launch_bounds__(kRingThreads, 1)
k_ring_selftest(int complete, uint32_t limit, int *err, int *out) {
    // the barriers of the ring, then the phase that is waited for; the ring
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(smem), *bar = full + kRingStages;
    uint32_t *ring = reinterpret_cast<uint32_t *>(smem + kRingAt);
    __shared__ uint32_t armed[kRingStages];
    __shared__ int abort_flag;
    for (int i = threadIdx.x; i < kRingWords; i += kRingThreads) {
        g_ring_src[i] = 0x9e3779b9u * (uint32_t)(i + 1);
        for (int s = 0; s < kRingStages; ++s) ring[s * kRingWords + i] = 0;
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < kRingStages; ++s) {
            ptx::mbar_init(full + s, 1);
            armed[s] = 0;
        }
        ptx::mbar_init(bar, 1);
        abort_flag = 0;
        ptx::fence_mbar_init();
    }
    ptx::fence_proxy_async_global();
    ptx::fence_proxy_async_smem();
    __syncthreads();
    if (complete && threadIdx.x == 0) ptx::mbar_arrive(bar);
    if (threadIdx.x == 0 || threadIdx.x == 64) {        // stages 0 and 2
        const int s = threadIdx.x / 32;
        armed[s] = 1;
        ptx::mbar_arrive_expect_tx(full + s, kRingWords * 4);
        kv::bulk_load(ptx::smem_u32(ring + s * kRingWords), g_ring_src, kRingWords * 4, full + s);
    }
    __syncwarp();
    const kv::Waits waits{&abort_flag, err, limit};
    const bool first = waits.on(bar, 0), second = waits.on(bar, 0);
    const int n_first = __syncthreads_count(first), n_second = __syncthreads_count(second);
    if (threadIdx.x >= 32) return;
    kv::drain_ring<kRingStages>(full, armed);
    int there = 0;
    for (int i = threadIdx.x; i < kRingStages * kRingWords; i += 32)
        there += ring[i] == 0x9e3779b9u * (uint32_t)(i % kRingWords + 1);
    there = __reduce_add_sync(0xffffffffu, there);
    if (threadIdx.x == 0) {
        out[0] = n_first;
        out[1] = n_second;
        out[2] = there;
    }
}

}  // namespace
}  // namespace gdn

extern "C" gdn_status gdn_selftest_wait(int complete, long long limit, int *waits_ok,
                                        void *stream) {
    if ((complete != 0 && complete != 1) || limit < 1 || limit > gdn::kMaxSelftestLimit)
        return GDN_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int *err = gdn::device_error_word();
    int *out = nullptr;
    if (!err || cudaGetSymbolAddress(reinterpret_cast<void **>(&out), gdn::g_selftest_out) !=
                    cudaSuccess)
        return GDN_ERR_CUDA;
    gdn::k_wait_selftest<<<1, 32, 0, st>>>(complete, static_cast<uint32_t>(limit), err, out);
    gdn::count_launch();
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    int host[2] = {0, 0};
    if (cudaMemcpyAsync(host, out, sizeof(host), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return GDN_ERR_CUDA;
    if (waits_ok) {
        waits_ok[0] = host[0];
        waits_ok[1] = host[1];
    }
    return GDN_OK;
}

extern "C" gdn_status gdn_selftest_ring(int complete, long long limit, int *result,
                                        void *stream) {
    if ((complete != 0 && complete != 1) || limit < 1 || limit > gdn::kMaxSelftestLimit || !result)
        return GDN_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int *err = gdn::device_error_word();
    int *out = nullptr;
    if (!err || cudaGetSymbolAddress(reinterpret_cast<void **>(&out), gdn::g_ring_out) !=
                    cudaSuccess)
        return GDN_ERR_CUDA;
    gdn::k_ring_selftest<<<1, gdn::kRingThreads, gdn::kRingSmem, st>>>(
        complete, static_cast<uint32_t>(limit), err, out);
    gdn::count_launch();
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    if (cudaMemcpyAsync(result, out, sizeof(gdn::g_ring_out), cudaMemcpyDeviceToHost, st) !=
            cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return GDN_ERR_CUDA;
    return GDN_OK;
}
