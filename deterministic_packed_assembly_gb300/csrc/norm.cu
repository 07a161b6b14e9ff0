// Layer norm of packed positions, and its gradients: the choice of kernels and the last sums.
//
//   m = mean of x, r = 1 / sqrt(mean of (x - m)^2 + eps), xh = (x - m) r, y = xh w + b
//   g = dy w,  dx = r (g - mean of g - xh mean of (g xh))
//   dw = sum of dy xh and db = sum of dy over the positions
//
// Memory bounds both passes, and next to it instructions: they go by pairs of values
// (elem.cuh).  A row's columns lie on threads in one way, whatever kernel takes it: eight a
// lane (rows.cuh), up to 15 warps and five spans a warp (norm.cuh).  The variance is taken
// from the values less their mean, so that a mean far from 0 costs no digits.
//
// Rows come through a ring in shared memory (ring.cuh), filled by the bulk copy engine, so
// that memory is kept busy while sums are exchanged, and rows that begin anywhere cost no
// more than others; a batch of up to four rows shares the barriers.  Rows of up to 512
// columns, which a warp or a part of one has, and forward calls of few rows are read
// straight from memory.  Backward each thread keeps the sums of its columns' dw and db over
// all its block's rows; blocks write them out once, and the last kernel adds the blocks'
// rows in order.  Rows of more than 19200 columns, and backward those that do not fit the ring
// twice beside their weights (more than 17920 columns of 16 bits, or 11520 floats), are read
// again instead of kept.
//
// 32768 x 2560 bf16: forward 59 us (83 % of the copy's bandwidth), backward 88 (84 %); 9973 x
// 5003 floats 71 and 96 (82, 92 %).  What keeps them from it is a batch's steps, which
// wait for one another: 48 and 45 % of the issue slots, DRAM 42 and 56 % by the counters.
// Narrow rows are far from it: 131072 x 64 bf16 11 and 19 us of 5 and 7, 131072 x 512 79 and 89 of 40
// and 59.  Their kernels wait too, for their own arithmetic and shuffles (40 and 36 % of the issue
// slots, registers for 31 and 25 % of the warps), and dw and db take a launch of 4 us more.

#include "norm.cuh"

namespace nsk {
namespace {

// The blocks' rows, added in order: 32 columns a block, its warps a run of rows each.
constexpr int kTotalWarps = 32;
template <class W>
__global__ void __launch_bounds__(32 * kTotalWarps) norm_total_kernel(const NormParams p) {
  pdl_wait();
  __shared__ float sums[kTotalWarps][33];
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32, which = blockIdx.y;
  W *to = static_cast<W *>(which ? p.dbias : p.dweight);
  if (!to) return;
  const uint64_t c = (uint64_t)blockIdx.x * 32 + lane;
  const uint32_t run = (p.blocks + kTotalWarps - 1) / kTotalWarps;
  const uint32_t a = min(p.blocks, warp * run), b = min(p.blocks, a + run);
  float sum = 0.0f;
  if (c < p.D) {
#pragma unroll 8
    for (uint32_t i = a; i < b; ++i) sum += p.partial[((uint64_t)i * 2 + which) * p.D + c];
  }
  sums[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && c < p.D) {
    for (int k = 1; k < kTotalWarps; ++k) sum += sums[k][lane];
    to[c] = from_f32<W>(sum);
  }
}

NormParams params_of(const ns_norm_inputs &in, uint32_t fed) {
  NormParams p = {};
  p.x = in.x, p.x_row = in.x_row, p.weight = in.weight, p.bias = in.bias, p.doc = in.doc;
  p.N = in.N, p.D = in.D, p.eps = in.eps, p.floats = in.weight_dtype == NS_F32;
  p.fed = std::min(in.N, fed);
  return p;
}
// By the rows' type.
template <class F>
cudaError_t by_type(const ns_norm_inputs &in, F &&call) {
  if (in.dtype == NS_F32) return call(float{});
  return in.dtype == NS_BF16 ? call(__nv_bfloat16{}) : call(__half{});
}
int piece_of_inputs(const ns_norm_inputs &in, const void *y) {
  const uint64_t es = in.dtype == NS_F32 ? 4 : 2, ws = in.weight_dtype == NS_F32 ? 4 : 2;
  return std::min(std::min(piece_of(in.x, in.x_row, in.D, es), piece_of(y, in.D, in.D, es)),
                  std::min(piece_of(in.weight, 0, in.D, ws), piece_of(in.bias, 0, in.D, ws)));
}

}  // namespace

uint64_t norm_workspace(uint32_t N, uint32_t D) {
  // rows of partial sums: as many as any kernel has blocks, of which each has a row at least
  uint32_t rows = 4 * kNormSMs;
  if (D > kNormNarrow) rows = std::max<uint32_t>(rows, 8 * kNormSMs * 256 / D + 1);
  return (uint64_t)std::min(N, rows) * 2 * D * sizeof(float);
}

cudaError_t launch_norm_forward(const ns_norm_inputs &in, void *y, float *mean, float *rstd,
                                cudaStream_t st, uint32_t fed) {
  NormParams p = params_of(in, fed);
  p.y = y, p.mean = mean, p.rstd = rstd;
  const int piece = piece_of_inputs(in, y);
  return by_type(in, [&](auto e) { return norm_forward<decltype(e)>(p, piece, st); });
}

cudaError_t launch_norm_backward(const ns_norm_inputs &in, const float *mean, const float *rstd,
                                 const void *dy, int64_t dy_row, void *dx, void *dweight,
                                 void *dbias, float *partial, cudaStream_t st, uint32_t fed) {
  NormParams p = params_of(in, fed);
  p.mean = const_cast<float *>(mean), p.rstd = const_cast<float *>(rstd);
  p.dy = dy, p.dy_row = dy_row, p.y = dx, p.dweight = dweight, p.dbias = dbias;
  p.partial = dweight || dbias ? partial : nullptr;
  const int piece =
      std::min(piece_of_inputs(in, dx), piece_of(dy, dy_row, in.D, in.dtype == NS_F32 ? 4 : 2));
  const cudaError_t e =
      in.N ? by_type(in, [&](auto e) { return norm_backward<decltype(e)>(p, piece, st); })
           : cudaSuccess;
  if (e != cudaSuccess || (!dweight && !dbias)) return e;
  const dim3 grid((in.D + 31) / 32, 2);
  ++launch_counter();
  if (in.weight_dtype == NS_F32)
    pdl_launch(norm_total_kernel<float>, grid, dim3(32 * kTotalWarps), 0, st, p);
  else if (in.weight_dtype == NS_BF16)
    pdl_launch(norm_total_kernel<__nv_bfloat16>, grid, dim3(32 * kTotalWarps), 0, st, p);
  else
    pdl_launch(norm_total_kernel<__half>, grid, dim3(32 * kTotalWarps), 0, st, p);
  return cudaGetLastError();
}

}  // namespace nsk
