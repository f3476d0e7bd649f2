/*
 * nvfp4_testing.h -- test hooks of libnvfp4.so.  Not part of the stable ABI;
 * the test suite uses them to exercise the GEMM's bounded-wait failure path
 * without faulting or hanging a GPU, and to see which path a size takes.
 */
#ifndef NVFP4_TESTING_H
#define NVFP4_TESTING_H

#include <stdint.h>

#include "nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Sets, for the following nvfp4_gemm calls in this process, the timeout of
 * every bounded wait inside the GEMM kernel (timeout_ns, counted from the
 * start of each wait, so it bounds a lack of progress, not the kernel's run
 * time; 0 restores the default of 4 s) and debug flags (bit 0: the producer never issues the
 * copies of the first pipeline stage, so the consumer's wait for it runs out
 * and the kernel reports NVFP4_ERR_TIMEOUT through the workspace status word
 * after draining its in-flight work).  Not thread-safe; tests only. */
NVFP4_API void nvfp4_testing_set_gemm_wait(uint64_t timeout_ns, int debug_flags);

/* How nvfp4_gemv (weights = 1) or nvfp4_gemv_gated (2) splits a call on a device
 * of `sms` SMs: plan = {CTAs, CTAs that share a row tile, 256-wide steps of K whose
 * x is staged at a time, such pieces for a CTA, units of weights in flight per
 * warp}.  Returns 0 when the sizes are out of range.  Host only. */
NVFP4_API int nvfp4_testing_gemv_plan(int64_t M, int64_t N, int64_t K, int weights, int sms, int plan[5]);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_TESTING_H */
