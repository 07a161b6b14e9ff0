// C entry points of the training operators (include/nstrain.h, nstrain_probe.h): every
// check of the arguments, then the launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "nstrain.h"
#include "nstrain_probe.h"
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

// ---- rows of a table -------------------------------------------------------------
// Strides of rows of D elements, where there is more than one row.
static bool fits_row(int64_t row, uint32_t D, uint32_t N) {
  return N <= 1 || (row >= (int64_t)D && row <= ((int64_t)1 << 44));
}

static bool check_embed(const ns_embed_inputs *in) {
  if (!in || !size_of(in->table_dtype) || !size_of(in->dtype)) return false;
  if (in->N >= (1u << 31) || in->V >= (1u << 31) || in->D >= (1u << 30)) return false;
  // blocks of a launch, and bytes of a workspace: past any memory long before
  if ((uint64_t)in->N * in->D >= (1ull << 42) || (uint64_t)in->V * in->D >= (1ull << 42))
    return false;
  if (!std::isfinite(in->scale)) return false;
  return usable(in->tokens, in->ids_64 ? 8 : 4, in->N == 0) && usable(in->doc, 4, true);
}

int ns_embed_forward(const ns_embed_inputs *in, const void *table, int64_t table_row, void *y,
                     void *cuda_stream) {
  if (!check_embed(in) || !fits_row(table_row, in->D, in->V)) return NS_ERR_INVALID_ARG;
  if (in->N == 0 || in->D == 0) return NS_OK;
  if (!usable(table, size_of(in->table_dtype), in->V == 0) || !usable(y, size_of(in->dtype)))
    return NS_ERR_INVALID_ARG;
  return done(nsk::launch_embed_forward(*in, table, table_row, y,
                                        static_cast<cudaStream_t>(cuda_stream)));
}

uint64_t ns_embed_workspace(uint32_t N, uint32_t V, uint32_t D) {
  if (N >= (1u << 31) || V >= (1u << 31) || D >= (1u << 30) || (uint64_t)N * D >= (1ull << 42))
    return 0;
  return nsk::embed_workspace(N, V, D);
}

int ns_embed_backward(const ns_embed_inputs *in, const void *dy, int64_t dy_row, void *dtable,
                      void *workspace, void *cuda_stream) {
  if (!check_embed(in) || !fits_row(dy_row, in->D, in->N)) return NS_ERR_INVALID_ARG;
  if (in->V == 0 || in->D == 0) return NS_OK;
  if (!usable(dy, size_of(in->dtype), in->N == 0) || !usable(dtable, size_of(in->table_dtype)) ||
      !usable(workspace, 16))
    return NS_ERR_INVALID_ARG;
  return done(nsk::launch_embed_backward(*in, dy, dy_row, dtable, workspace,
                                         static_cast<cudaStream_t>(cuda_stream)));
}

// ---- layer norm ------------------------------------------------------------------
static bool check_norm(const ns_norm_inputs *in) {
  if (!in || !size_of(in->dtype) ||
      (in->weight_dtype != NS_F32 && in->weight_dtype != in->dtype))
    return false;
  if (in->N >= (1u << 31) || in->D == 0 || in->D >= (1u << 30)) return false;
  if (!(in->eps >= 0.0f) || !std::isfinite(in->eps)) return false;
  if (!fits_row(in->x_row, in->D, in->N)) return false;
  const uint64_t es = size_of(in->dtype), ws = size_of(in->weight_dtype);
  return usable(in->x, es, in->N == 0) && usable(in->weight, ws, true) &&
         usable(in->bias, ws, true) && usable(in->doc, 4, true);
}

static int run_norm_forward(const ns_norm_inputs *in, uint32_t fed, void *y, float *mean,
                            float *rstd, void *cuda_stream) {
  if (!check_norm(in)) return NS_ERR_INVALID_ARG;
  if (in->N == 0) return NS_OK;
  if (!usable(y, size_of(in->dtype)) || !usable(mean, 4, true) || !usable(rstd, 4, true))
    return NS_ERR_INVALID_ARG;
  return done(nsk::launch_norm_forward(*in, y, mean, rstd, static_cast<cudaStream_t>(cuda_stream),
                                       fed));
}

uint64_t ns_norm_workspace(uint32_t N, uint32_t D) {
  return N < (1u << 31) && D < (1u << 30) ? nsk::norm_workspace(N, D) : 0;
}

static int run_norm_backward(const ns_norm_inputs *in, uint32_t fed, const float *mean,
                             const float *rstd, const void *dy, int64_t dy_row, void *dx,
                             void *dweight, void *dbias, void *workspace, void *cuda_stream) {
  if (!check_norm(in) || !fits_row(dy_row, in->D, in->N)) return NS_ERR_INVALID_ARG;
  const uint64_t es = size_of(in->dtype), ws = size_of(in->weight_dtype);
  const bool none = in->N == 0;
  if (!usable(mean, 4, none) || !usable(rstd, 4, none) || !usable(dy, es, none) ||
      !usable(dx, es, none) || !usable(dweight, ws, true) || !usable(dbias, ws, true) ||
      !usable(workspace, 4, none || (!dweight && !dbias)))
    return NS_ERR_INVALID_ARG;
  return done(nsk::launch_norm_backward(*in, mean, rstd, dy, dy_row, dx, dweight, dbias,
                                        static_cast<float *>(workspace),
                                        static_cast<cudaStream_t>(cuda_stream), fed));
}

int ns_norm_forward(const ns_norm_inputs *in, void *y, float *mean, float *rstd,
                    void *cuda_stream) {
  return run_norm_forward(in, 0xffffffffu, y, mean, rstd, cuda_stream);
}

int ns_norm_backward(const ns_norm_inputs *in, const float *mean, const float *rstd,
                     const void *dy, int64_t dy_row, void *dx, void *dweight, void *dbias,
                     void *workspace, void *cuda_stream) {
  return run_norm_backward(in, 0xffffffffu, mean, rstd, dy, dy_row, dx, dweight, dbias, workspace,
                           cuda_stream);
}

int ns_norm_probe_forward(const ns_norm_inputs *in, uint32_t fed, void *y, float *mean,
                          float *rstd, void *cuda_stream) {
  if (!in || (fed < in->N && fed % 4)) return NS_ERR_INVALID_ARG;
  return run_norm_forward(in, fed, y, mean, rstd, cuda_stream);
}

int ns_norm_probe_backward(const ns_norm_inputs *in, uint32_t fed, const float *mean,
                           const float *rstd, const void *dy, int64_t dy_row, void *dx,
                           void *dweight, void *dbias, void *workspace, void *cuda_stream) {
  if (!in || (fed < in->N && fed % 4)) return NS_ERR_INVALID_ARG;
  return run_norm_backward(in, fed, mean, rstd, dy, dy_row, dx, dweight, dbias, workspace,
                           cuda_stream);
}

// ---- tokens by expert, and back ----------------------------------------------------
static bool check_experts(const ns_expert_sizes *s) {
  return s && size_of(s->dtype) && s->k >= 1 && s->E >= 1 && s->E <= NS_DISPATCH_MAX_EXPERTS &&
         (uint64_t)s->N * s->k < (1ull << 31) && s->D < (1u << 30) &&
         (uint64_t)s->N * s->k * s->D < (1ull << 42);
}

uint64_t ns_dispatch_workspace(uint32_t N, uint32_t k, uint32_t E) {
  if (k == 0 || E == 0 || E > NS_DISPATCH_MAX_EXPERTS || (uint64_t)N * k >= (1ull << 31)) return 0;
  return nsk::dispatch_workspace(N, k, E);
}

int ns_dispatch(const ns_expert_sizes *sizes, const int32_t *ids, const void *x, int64_t x_row,
                int32_t *place, int32_t *slots, int32_t *offsets, void *rows, void *workspace,
                void *cuda_stream) {
  if (!check_experts(sizes) || !fits_row(x_row, sizes->D, sizes->N)) return NS_ERR_INVALID_ARG;
  const uint64_t es = size_of(sizes->dtype);
  const bool none = sizes->N == 0, nothing = none || sizes->D == 0;
  if (!usable(ids, 4, none) || !usable(x, es, nothing) || !usable(place, 4, none) ||
      !usable(slots, 4, none) || !usable(offsets, 4) || !usable(rows, es, nothing) ||
      !usable(workspace, 16, ns_dispatch_workspace(sizes->N, sizes->k, sizes->E) == 0))
    return NS_ERR_INVALID_ARG;
  return done(nsk::launch_dispatch(*sizes, ids, x, x_row, place, slots, offsets, rows, workspace,
                                   static_cast<cudaStream_t>(cuda_stream)));
}

int ns_combine(const ns_expert_sizes *sizes, const int32_t *place, const int32_t *offsets,
               const float *weights, const void *rows, int64_t rows_row, void *out,
               void *cuda_stream) {
  if (!check_experts(sizes) || !fits_row(rows_row, sizes->D, sizes->N * sizes->k))
    return NS_ERR_INVALID_ARG;
  if (sizes->N == 0 || sizes->D == 0) return NS_OK;
  const uint64_t es = size_of(sizes->dtype);
  if (!usable(place, 4) || !usable(offsets, 4) || !usable(weights, 4, true) ||
      !usable(rows, es) || !usable(out, es))
    return NS_ERR_INVALID_ARG;
  return done(nsk::launch_combine(*sizes, place, offsets, weights, rows, rows_row, out,
                                  static_cast<cudaStream_t>(cuda_stream)));
}

int ns_combine_backward(const ns_expert_sizes *sizes, const int32_t *place,
                        const int32_t *offsets, const float *weights, const void *rows,
                        int64_t rows_row, const void *d_out, int64_t d_out_row, void *d_rows,
                        float *d_weights, void *cuda_stream) {
  if (!check_experts(sizes) || !fits_row(d_out_row, sizes->D, sizes->N) ||
      (d_weights && !fits_row(rows_row, sizes->D, sizes->N * sizes->k)))
    return NS_ERR_INVALID_ARG;
  if (sizes->N == 0) return NS_OK;
  const uint64_t es = size_of(sizes->dtype);
  const bool nothing = sizes->D == 0;
  if (!usable(place, 4) || !usable(offsets, 4) || !usable(weights, 4, true) ||
      !usable(rows, es, nothing || !d_weights) || !usable(d_out, es, nothing) ||
      !usable(d_rows, es, nothing) || !usable(d_weights, 4, true))
    return NS_ERR_INVALID_ARG;
  return done(nsk::launch_combine_backward(*sizes, place, offsets, weights, rows, rows_row, d_out,
                                           d_out_row, d_rows, d_weights,
                                           static_cast<cudaStream_t>(cuda_stream)));
}

}  // extern "C"
