// host.h -- what the library's translation units share on the host: error
// text, device facts, tensor maps and the test knobs (defined in
// tcgemm_host.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <mutex>

#include "../../include/tcgemm.h"

namespace tcg {
namespace host {

struct Device {
    int num_sms = 0;
    int max_smem_optin = 0;
};

constexpr int kMaxExtent = 0x7FFFFFFF - 4095;   // rows or columns: an index rounded up to a tile or a step still fits an int

// A workspace, from its start: the status words, then what every call finds
// zero and leaves zero (the arrival counters of tiles whose K is shared, the
// balance loss's totals), then what a call may leave anything in (partial
// sums).  Each has a range of its own, the same for every entry point, so one
// workspace serves them in any order.
constexpr size_t kWorkspaceHeader = 256;   // status word and diagnostics
constexpr size_t kCounterBytes = 8192;
constexpr int kMaxBalanceExperts = 1024;
constexpr size_t kBalanceAt = kWorkspaceHeader + kCounterBytes;
constexpr size_t kBalanceBytes = static_cast<size_t>(kMaxBalanceExperts) * 28 + 256;
constexpr size_t kScratchAt = kBalanceAt + kBalanceBytes;
static_assert(kBalanceAt % 256 == 0 && kScratchAt % 256 == 0, "ranges start on 256 bytes");

// What has to be set up once on each device, a kernel's attributes: f() runs in
// the first call made with that device current, and its outcome is that
// device's for good.
constexpr int kMaxDevices = 64;
class OncePerDevice {
public:
    template <typename F>
    cudaError_t operator()(F f) {
        int dev = 0;
        const cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
        std::call_once(once_[dev], [&] { err_[dev] = f(); });
        return err_[dev];
    }

private:
    std::once_flag once_[kMaxDevices];
    cudaError_t err_[kMaxDevices] = {};
};

// The current device; TCG_ERR_ARCH when it is not sm_103.
tcg_status device(Device& out);
// The text of tcg_last_error, and the code to return.
tcg_status fail(tcg_status st, const char* text);
tcg_status fail_launch(const char* what, cudaError_t e);
// 2-D tensor map of an 8-bit matrix (inner contiguous bytes per row, outer
// rows ld bytes apart), 128-byte swizzled boxes; cached as tcg_gemm's are.
tcg_status map_bytes(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer, uint64_t ld,
                     uint32_t box_inner, uint32_t box_outer);
// Launch with leave to start while the kernel ahead ends; the kernel calls
// wait_for_kernel_ahead() before it reads or writes anything.
template <typename P>
cudaError_t launch_early(void (*kernel)(P), dim3 grid, unsigned threads, cudaStream_t stream, const P& p, size_t smem = 0) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}
__device__ __forceinline__ void wait_for_kernel_ahead() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // and the next one may do the same
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Test knobs of tcg_debug_set.
long long wait_timeout_ns();
int fault_inject();

}  // namespace host
}  // namespace tcg
