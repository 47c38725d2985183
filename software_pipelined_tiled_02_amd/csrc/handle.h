// handle.h -- what a gemm_handle_t points to, and how an entry point
// enqueues on the handle's device.
#ifndef PIPEGEMM_HANDLE_H
#define PIPEGEMM_HANDLE_H

#include <hip/hip_runtime.h>

#include "pipegemm.h"

struct gemm_handle_s {
    int device;
    int num_cus;
    int tile_override;  // GEMM_TILE_AUTO or a class
    void* scratch;      // this device's scratch array (gemm_run_splitk_noalloc)
};

namespace pg {

// Notes a failing call for gemm_last_hip_error; returns GEMM_ERR_HIP.
int hip_fail(hipError_t e);

// enqueue() with the handle's device current; the caller's device is put
// back, and a failure to do so is reported unless enqueue already failed.
template <typename F>
int on_device(gemm_handle_t h, F enqueue) {
    int cur = -1;
    hipError_t e = hipGetDevice(&cur);
    if (e != hipSuccess) return hip_fail(e);
    if (cur != h->device && (e = hipSetDevice(h->device)) != hipSuccess) return hip_fail(e);
    e = enqueue();
    if (cur != h->device) {
        const hipError_t r = hipSetDevice(cur);
        if (e == hipSuccess) e = r;
    }
    return e == hipSuccess ? GEMM_OK : hip_fail(e);
}

}  // namespace pg

#endif
