/*
 * llchecks.h -- C ABI of the checks in libllprobes.so: steps inside the kernels of
 * liblinlayers.so whose exact results no entry point shows, run by themselves so
 * that a test can compare them bit for bit.
 *
 * Conventions as in llprobes.h: DEVICE pointers on the current device, calls only
 * enqueue work, 0 on success, -1 for an invalid argument (nothing is launched),
 * otherwise the hipError_t of the launch.
 */
#ifndef LLCHECKS_H
#define LLCHECKS_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The scale of a quantised block and the reciprocal its values are multiplied by
 * (quant8_run, rmsnorm_run), for the n largest magnitudes whose fp32 bit patterns are
 * first, first + 1, ...: scale[i] and inv[i] for pattern first + i.  q_type: 3 (LL_E4M3)
 * or 4 (LL_E5M2).  first + n at most 2^31, n >= 0; scale and inv: n floats each. */
int ll_check_scale8(int q_type, uint32_t first, int64_t n, float* scale, float* inv, void* stream);

#ifdef __cplusplus
}
#endif

#endif
