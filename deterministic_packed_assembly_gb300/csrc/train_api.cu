// C entry points of the training operators (include/nstrain.h): every check of
// the arguments, then the launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "nstrain.h"
#include "train.h"

namespace {

// Bytes of an element, 0 for an unknown type.
uint64_t size_of(int32_t dtype) {
  return dtype == NS_F32 ? 4 : dtype == NS_BF16 || dtype == NS_F16 ? 2 : 0;
}

// A pointer that a kernel may use as elements of `align` bytes; NULL is let
// through where the argument is optional or nothing is there.
bool usable(const void *p, uint64_t align, bool optional = false) {
  return p ? reinterpret_cast<uintptr_t>(p) % align == 0 : optional;
}

// [a, a + na) and [b, b + nb) share a byte.
bool overlap(const void *a, uint64_t na, const void *b, uint64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

int done(cudaError_t e) { return e == cudaSuccess ? NS_OK : NS_ERR_CUDA; }

bool check_scan(const ns_scan_inputs *in) {
  if (!in || !size_of(in->dtype)) return false;
  if (in->B >= (1u << 31) || in->T > NS_SCAN_MAX_T || in->D >= (1u << 31)) return false;
  // blocks of a launch: at most eight along time for each 32 channels of a row
  if ((uint64_t)in->B * ((in->D + 31) / 32) >= (1ull << 31) / 8) return false;
  // a stride that reaches past the address space cannot be one
  const int64_t most = (int64_t)1 << 44;
  for (int64_t s : {in->z_row, in->z_time, in->f_row, in->f_time})
    if (s < 0 || s > most) return false;
  const bool none = in->B == 0 || in->T == 0 || in->D == 0;
  const uint64_t es = size_of(in->dtype);
  return usable(in->z, es, none) && usable(in->f, es, none) && usable(in->bias, 4, true) &&
         usable(in->pos, 4, true) && usable(in->doc, 4, true);
}

}  // namespace

namespace nsk {

cudaError_t allow_shared_memory(const void *kernel, bool all) {
  struct Known {
    const void *kernel;
    int device;
  };
  thread_local Known known[64];
  thread_local unsigned count = 0;
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  for (unsigned i = 0; e == cudaSuccess && i < count && i < 64; ++i)
    if (known[i].kernel == kernel && known[i].device == device) return cudaSuccess;
  cudaFuncAttributes a;
  int most = 0;
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, kernel);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, device);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             most - (int)a.sharedSizeBytes);
  if (e == cudaSuccess && all)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return e;
  }
  known[count++ % 64] = {kernel, device};
  return cudaSuccess;
}

}  // namespace nsk

extern "C" {

int ns_scan_forward(const ns_scan_inputs *in, const float *h0, void *y, float *h_last,
                    float *states, void *cuda_stream) {
  if (!check_scan(in)) return NS_ERR_INVALID_ARG;
  if (in->B == 0 || in->D == 0) return NS_OK;
  if (!usable(h0, 4, true) || !usable(h_last, 4) || !usable(y, size_of(in->dtype), in->T == 0) ||
      !usable(states, 4, true))
    return NS_ERR_INVALID_ARG;
  return done(nsk::launch_scan_forward(*in, h0, y, h_last, states,
                                       static_cast<cudaStream_t>(cuda_stream)));
}

uint64_t ns_scan_workspace(uint32_t B, uint32_t T, uint32_t D) {
  return nsk::scan_partial_rows(B, T, D) * D * sizeof(float);
}

int ns_scan_backward(const ns_scan_inputs *in, const float *states, const void *dy,
                     int64_t dy_row, int64_t dy_time, const float *dh_last, void *dz, void *df,
                     float *dbias, float *dh0, void *workspace, void *cuda_stream) {
  if (!check_scan(in)) return NS_ERR_INVALID_ARG;
  const int64_t most = (int64_t)1 << 44;
  if (dy_row < 0 || dy_time < 0 || dy_row > most || dy_time > most) return NS_ERR_INVALID_ARG;
  if (in->D == 0) return NS_OK;
  const uint64_t es = size_of(in->dtype);
  const bool none = in->B == 0 || in->T == 0;
  if (!usable(states, 4, none) || !usable(dy, es, none) || !usable(dz, es, none) ||
      !usable(df, es, none) || !usable(dh_last, 4, true) || !usable(dbias, 4, true) ||
      !usable(dh0, 4, true) || !usable(workspace, 4, !dbias || in->B == 0))
    return NS_ERR_INVALID_ARG;
  return done(nsk::launch_scan_backward(*in, states, dy, dy_row, dy_time, dh_last, dz, df, dbias,
                                        dh0, static_cast<float *>(workspace),
                                        static_cast<cudaStream_t>(cuda_stream)));
}

int ns_distill(const ns_distill_inputs *in, float *loss, void *dlogits, int64_t dlogits_row,
               void *cuda_stream) {
  if (!in) return NS_ERR_INVALID_ARG;
  const uint64_t es = size_of(in->dtype), ts = size_of(in->top_dtype);
  if (!es || !ts || in->V == 0 || in->V * es > NS_DISTILL_MAX_ROW || in->K == 0 ||
      in->K > NS_DISTILL_MAX_TOP || in->N >= (1u << 28) ||
      (in->V * es > NS_DISTILL_WIDE_ROW && in->K > NS_DISTILL_WIDE_TOP))
    return NS_ERR_INVALID_ARG;
  if (!(in->temperature > 0.0f) || !std::isfinite(in->temperature) ||
      !std::isfinite(2.0f / in->temperature))
    return NS_ERR_INVALID_ARG;
  const int64_t most = (int64_t)1 << 44;
  if (in->N == 0) return NS_OK;
  if (in->logits_row < (int64_t)in->V || in->logits_row > most) return NS_ERR_INVALID_ARG;
  if (!usable(in->logits, es) || !usable(in->top_logits, ts) ||
      !usable(in->top_ids, in->ids_64 ? 8 : 4) || !usable(in->teacher_lse, 4, true) ||
      !usable(in->weight, 4, true) || !usable(loss, 4) || !usable(dlogits, es, true))
    return NS_ERR_INVALID_ARG;
  if (dlogits) {
    if (dlogits_row < (int64_t)in->V || dlogits_row > most) return NS_ERR_INVALID_ARG;
    // the gradient takes the logits' place element by element, or lies elsewhere
    const bool same = dlogits == in->logits && dlogits_row == in->logits_row;
    if (!same && overlap(in->logits, ((in->N - 1) * (uint64_t)in->logits_row + in->V) * es,
                         dlogits, ((in->N - 1) * (uint64_t)dlogits_row + in->V) * es))
      return NS_ERR_INVALID_ARG;
  }
  return done(nsk::launch_distill(*in, loss, dlogits, dlogits_row,
                                  static_cast<cudaStream_t>(cuda_stream)));
}

static bool check_route(const ns_route_inputs *in) {
  if (!in || !size_of(in->dtype) || in->E == 0 || in->E > NS_ROUTE_MAX_EXPERTS || in->k == 0 ||
      in->k > in->E || in->k > NS_ROUTE_MAX_K || (uint64_t)in->N * in->k >= (1ull << 31))
    return false;
  if (in->N == 0) return true;
  if (in->logits_row < (int64_t)in->E || in->logits_row > ((int64_t)1 << 44)) return false;
  return usable(in->logits, size_of(in->dtype)) && usable(in->doc, 4, true);
}

uint64_t ns_route_workspace(uint32_t N, uint32_t E) {
  if (E > NS_ROUTE_MAX_EXPERTS) return 0;  // the layout is not made for them
  return nsk::route_blocks(N, E) * (8ull * E + 4);
}

int ns_route_forward(const ns_route_inputs *in, int32_t *ids, float *weights, int32_t *counts,
                     int32_t *tokens, float *loss, void *workspace, void *cuda_stream) {
  if (!check_route(in)) return NS_ERR_INVALID_ARG;
  if (!usable(ids, 4, in->N == 0) || !usable(weights, 4, in->N == 0) || !usable(counts, 4) ||
      !usable(tokens, 4) || !usable(loss, 4) ||
      !usable(workspace, 4, ns_route_workspace(in->N, in->E) == 0))
    return NS_ERR_INVALID_ARG;
  return done(nsk::launch_route_forward(*in, ids, weights, counts, tokens, loss, workspace,
                                        static_cast<cudaStream_t>(cuda_stream)));
}

int ns_route_backward(const ns_route_inputs *in, const int32_t *ids, const float *weights,
                      const int32_t *counts, const int32_t *tokens, const float *d_weights,
                      const float *d_loss, void *dlogits, void *cuda_stream) {
  if (!check_route(in)) return NS_ERR_INVALID_ARG;
  if (in->N == 0) return NS_OK;
  if (!usable(ids, 4) || !usable(weights, 4) || !usable(counts, 4) || !usable(tokens, 4) ||
      !usable(d_weights, 4, true) || !usable(d_loss, 4, true) ||
      !usable(dlogits, size_of(in->dtype)))
    return NS_ERR_INVALID_ARG;
  return done(nsk::launch_route_backward(*in, ids, weights, counts, tokens, d_weights, d_loss,
                                         dlogits, static_cast<cudaStream_t>(cuda_stream)));
}

}  // extern "C"
