// ccc_waits.cu -- the bounded waits inside the mixer's kernels as a caller
// sees them (include/ccc.h): how long they last, and how many have been given
// up on this device.
//
// A kernel whose wait runs out ends like any other, so nothing on the host
// tells of it.  Each of its CTAs that gave up adds one to a counter in device
// memory, which only ever grows: the common case costs nothing, there is
// nothing to clear in front of a launch, and no call can hide another's.
#include <atomic>
#include <mutex>

#include "ccc.h"
#include "ccc_checks.h"
#include "ccc_symbol.h"
#include "ccc_waits.h"

namespace ccc {

namespace {

__device__ unsigned int g_given_up;

SymbolAddress g_address;
std::atomic<int64_t> g_limit{CCC_WAIT_LIMIT_DEFAULT};

// Driver entry points, fetched through the runtime so the library needs no
// link against the driver library.
using CtxGetCurrentFn = CUresult (*)(CUcontext *);
using CtxGetIdFn = CUresult (*)(CUcontext, unsigned long long *);

std::once_flag g_entry_once;
CtxGetCurrentFn g_ctx_get_current = nullptr;
CtxGetIdFn g_ctx_get_id = nullptr;

void load_entry_points() {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
        g_ctx_get_current = reinterpret_cast<CtxGetCurrentFn>(f);
    f = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
        g_ctx_get_id = reinterpret_cast<CtxGetIdFn>(f);
}

}  // namespace

unsigned long long current_context_id() {
    std::call_once(g_entry_once, load_entry_points);
    if (!g_ctx_get_current || !g_ctx_get_id) return 0;
    CUcontext ctx = nullptr;
    if (g_ctx_get_current(&ctx) != CUDA_SUCCESS || ctx == nullptr) return 0;
    unsigned long long id = 0;
    if (g_ctx_get_id(ctx, &id) != CUDA_SUCCESS) return 0;
    return id;
}

Waits current_waits() { return Waits{static_cast<unsigned int *>(g_address.find(&g_given_up)), g_limit.load(std::memory_order_relaxed)}; }

}  // namespace ccc

using namespace ccc;

extern "C" {

int ccc_set_wait_limit(int64_t clocks) {
    if (clocks < 0) return CCC_ERR_SHAPE;
    g_limit.store(clocks, std::memory_order_relaxed);
    return CCC_OK;
}

int ccc_wait_status(uint32_t *status, void *cuda_stream) {
    if (!status) return CCC_ERR_NULL;
    if (!aligned(status, 4)) return CCC_ERR_ALIGN;
    const void *counter = g_address.find(&g_given_up);
    if (!counter) return CCC_ERR_CUDA;
    return cudaMemcpyAsync(status, counter, sizeof(uint32_t), cudaMemcpyDeviceToDevice, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess
               ? CCC_OK
               : CCC_ERR_CUDA;
}

}  // extern "C"
