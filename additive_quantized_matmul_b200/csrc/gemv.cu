// Decode-time product y = diag(s) W x for batch 1..16 (sm_100a): aq_gemv,
// aq_gemv_ordered and aq_gemv_noalloc.  The kernels are in gemv_kernels.cuh,
// the launch plans in gemv_plan.cuh.
#include <mutex>

#include <cuda.h>  // driver types only; the calls are fetched at run time

#include "gemv_plan.cuh"

namespace aqh {
using namespace aqk;

size_t gemv_workspace_bytes(const Geom &g, int batch) { return plan_gemv(g, batch).ws_bytes; }

static GemvOut plain_out(const void *packed, const uint16_t *cb, const uint16_t *scales, uint16_t *y)
{
    return GemvOut{{{reinterpret_cast<const uint8_t *>(packed), reinterpret_cast<const uint4 *>(cb), scales}}, y};
}

cudaError_t launch_gemv(const Geom &g, const void *packed, const uint16_t *cb,
                        const uint16_t *scales, const uint16_t *x, int batch, uint16_t *y,
                        void *ws, cudaStream_t s, bool pdl)
{
    return launch_plan(g, plan_gemv(g, batch), plain_out(packed, cb, scales, y), x, batch, ws, s, pdl);
}

// ---------------------------------------------------------------------------
// Decode-time product without caller-provided workspace.
//
// The split-K partial sums, arrival counters and status word live in one
// file-scope device array (every GPU that loads this library holds it until
// the process exits).  Host code must not hand the array's name to a kernel:
// on the host it is only a stand-in, so its device address is looked up
// with cudaGetSymbolAddress, the device current, once per device and context.  All
// calls share the array, so calls that overlap on the GPU race; each call
// clears the status word and counters (cudaMemsetAsync on its stream) before
// its kernel starts.
// ---------------------------------------------------------------------------
static __device__ __align__(256) unsigned char g_gemv_scratch[AQ_GEMV_NOALLOC_SCRATCH_BYTES];

namespace {

// The array's device address belongs to one CUDA context.  It is looked up
// once per context (the runtime's primary context of a device, or another
// context the caller made current) and kept with the context's id, which
// the driver never reuses within a process: after cudaDeviceReset, or under
// a different current context, the next call looks the address up again
// instead of using a stale one.  The driver calls are fetched at run time,
// so the library does not link the driver library itself.
using CtxGetCurrentFn = CUresult (*)(CUcontext *);
using CtxGetIdFn = CUresult (*)(CUcontext, unsigned long long *);

// Id of the calling thread's current context, or 0 if there is none (or the
// driver lacks the calls).
unsigned long long current_context_id()
{
    static CtxGetCurrentFn get_current = nullptr;
    static CtxGetIdFn get_id = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            get_current = reinterpret_cast<CtxGetCurrentFn>(f);
        f = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            get_id = reinterpret_cast<CtxGetIdFn>(f);
        cudaGetLastError();  // a failed query leaves no sticky error behind
    });
    if (!get_current || !get_id) return 0;
    CUcontext ctx = nullptr;
    if (get_current(&ctx) != CUDA_SUCCESS || !ctx) return 0;
    unsigned long long id = 0;
    return get_id(ctx, &id) == CUDA_SUCCESS ? id : 0;
}

constexpr int kMaxDevices = 64;
struct ScratchAddr {
    unsigned long long ctx_id;  // 0: not looked up
    void *ptr;
};
std::mutex g_scratch_mutex;
ScratchAddr g_scratch_addr[kMaxDevices] = {};

cudaError_t scratch_for_current_context(void **out)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    const unsigned long long id = current_context_id();
    std::lock_guard<std::mutex> lock(g_scratch_mutex);
    ScratchAddr &a = g_scratch_addr[dev];
    if (id != 0 && a.ctx_id == id) {
        *out = a.ptr;
        return cudaSuccess;
    }
    // with this device current: the array's address in the current context
    // (this also makes the device's primary context current if none was)
    void *p = nullptr;
    e = cudaGetSymbolAddress(&p, g_gemv_scratch);
    if (e != cudaSuccess) return e;
    a.ctx_id = id != 0 ? id : current_context_id();
    a.ptr = p;
    *out = p;
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_gemv_noalloc(const Geom &g, const void *packed, const uint16_t *cb,
                                const uint16_t *scales, const uint16_t *x, int batch, uint16_t *y,
                                cudaStream_t s, bool *too_large)
{
    const GemvPlan p = plan_gemv(g, batch, AQ_GEMV_NOALLOC_SCRATCH_BYTES);
    *too_large = p.ws_bytes > AQ_GEMV_NOALLOC_SCRATCH_BYTES;
    if (*too_large) return cudaSuccess;
    void *scratch = nullptr;
    cudaError_t e = scratch_for_current_context(&scratch);
    if (e != cudaSuccess) return e;
    // status word and arrival counters must start at zero; the partials are
    // fully written before they are read
    const size_t clear = p.slots > 0 ? kWsData : kWsHeader;
    e = cudaMemsetAsync(scratch, 0, clear, s);
    if (e != cudaSuccess) return e;
    return launch_plan(g, p, plain_out(packed, cb, scales, y), x, batch, scratch, s, true);
}

}  // namespace aqh
