/*
 * nstrain_probe.h -- test helpers of the training operators.
 *
 * The layer norm's wide rows come through shared memory: a warp copies them, the
 * others wait for them.  Every wait has a limit, after which the kernel goes on and
 * ends, and what it did not get comes out as NaN.  These calls are ns_norm_forward and
 * ns_norm_backward with rows that never come, so that a test sees a wait run out.
 */
#ifndef NSTRAIN_PROBE_H
#define NSTRAIN_PROBE_H

#include <stdint.h>

#include "nstrain.h"

#ifdef __cplusplus
extern "C" {
#endif

/* As the calls they are named after, where only the first `fed` rows are copied (a multiple
 * of 4, the largest batch, or at least N): of the others nothing comes, and the call's
 * kernel takes some tenths of a second to give up.  Rows that are read straight from
 * memory do not wait.  Errors: as the calls, and INVALID_ARG for another fed. */
int ns_norm_probe_forward(const ns_norm_inputs *in, uint32_t fed, void *y, float *mean,
                          float *rstd, void *cuda_stream);
int ns_norm_probe_backward(const ns_norm_inputs *in, uint32_t fed, const float *mean,
                           const float *rstd, const void *dy, int64_t dy_row, void *dx,
                           void *dweight, void *dbias, void *workspace, void *cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* NSTRAIN_PROBE_H */
