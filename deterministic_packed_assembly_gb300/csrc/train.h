// Host-side launchers of the training operators' kernels (internal interface
// between the C ABI in train_api.cu and scan.cu, distill.cu, route.cu, embed.cu, norm.cu,
// experts.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "nstrain.h"

namespace nsk {

// Lets a kernel take as much dynamic shared memory as a block can have; asked once
// for a kernel and device by each thread that launches it.  `all`: an SM that runs it gives
// all that it has for shared memory, so that another kernel's blocks find room beside its own
// (what is set for one kernel's blocks alone stays until they have left).
cudaError_t allow_shared_memory(const void *kernel, bool all = false);

cudaError_t launch_scan_forward(const ns_scan_inputs &in, const float *h0, void *y, float *h_last,
                                float *states, cudaStream_t st);
// Rows of partial bias gradients that the backward pass writes ([rows][D]).
uint64_t scan_partial_rows(uint32_t B, uint32_t T, uint32_t D);
cudaError_t launch_scan_backward(const ns_scan_inputs &in, const float *states, const void *dy,
                                 int64_t dy_row, int64_t dy_time, const float *dh_last, void *dz,
                                 void *df, float *dbias, float *dh0, float *partial,
                                 cudaStream_t st);

cudaError_t launch_distill(const ns_distill_inputs &in, float *loss, void *dlogits,
                           int64_t dlogits_row, cudaStream_t st);

// Rows of partial sums that the forward kernel's blocks write.
uint32_t route_blocks(uint32_t N, uint32_t E);
cudaError_t launch_route_forward(const ns_route_inputs &in, int32_t *ids, float *weights,
                                 int32_t *counts, int32_t *tokens, float *loss, void *workspace,
                                 cudaStream_t st);
cudaError_t launch_route_backward(const ns_route_inputs &in, const int32_t *ids,
                                  const float *weights, const int32_t *counts,
                                  const int32_t *tokens, const float *d_weights,
                                  const float *d_loss, void *dlogits, cudaStream_t st);

uint64_t embed_workspace(uint32_t N, uint32_t V, uint32_t D);
cudaError_t launch_embed_forward(const ns_embed_inputs &in, const void *table, int64_t table_row,
                                 void *y, cudaStream_t st);
cudaError_t launch_embed_backward(const ns_embed_inputs &in, const void *dy, int64_t dy_row,
                                  void *dtable, void *workspace, cudaStream_t st);

uint64_t norm_workspace(uint32_t N, uint32_t D);
// fed: rows that come to the ring, but for a test (include/nstrain_probe.h) all of them.
cudaError_t launch_norm_forward(const ns_norm_inputs &in, void *y, float *mean, float *rstd,
                                cudaStream_t st, uint32_t fed = 0xffffffffu);
cudaError_t launch_norm_backward(const ns_norm_inputs &in, const float *mean, const float *rstd,
                                 const void *dy, int64_t dy_row, void *dx, void *dweight,
                                 void *dbias, float *partial, cudaStream_t st,
                                 uint32_t fed = 0xffffffffu);

uint64_t dispatch_workspace(uint32_t N, uint32_t k, uint32_t E);
cudaError_t launch_dispatch(const ns_expert_sizes &s, const int32_t *ids, const void *x,
                            int64_t x_row, int32_t *place, int32_t *slots, int32_t *offsets,
                            void *rows, void *workspace, cudaStream_t st);
cudaError_t launch_combine(const ns_expert_sizes &s, const int32_t *place, const int32_t *offsets,
                           const float *weights, const void *rows, int64_t rows_row, void *out,
                           cudaStream_t st);
cudaError_t launch_combine_backward(const ns_expert_sizes &s, const int32_t *place,
                                    const int32_t *offsets, const float *weights,
                                    const void *rows, int64_t rows_row, const void *d_out,
                                    int64_t d_out_row, void *d_rows, float *d_weights,
                                    cudaStream_t st);

}  // namespace nsk
