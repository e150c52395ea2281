// ssm_ssd_step.cu -- one token of the state-space dual: per head h = a h + beta B x^T (an N x P state
// in fp32, updated in place), y = h^T C + D x.
//
// Reading and rewriting the state (8 bytes per element) is all the work, so the kernel is a stream:
// the columns of a head's state are independent, a CTA takes `cols` of them, its threads stand on
// consecutive 16-byte column groups, and each walks every `groups`-th state row in batches of four, the next batch
// loaded before the one at hand is used (and the first before the head's factors are formed). The row sums of C h
// meet in shared memory once at the end. Heads are split over CTAs by columns where there are too few heads to
// fill the GPU. 64 x 64 heads of 128 x 64 states: 47 us, 5.7 TB/s; with 256 threads a CTA 56 us, eight rows a batch
// 49 us, without the batch ahead 50 us.
#include "ssm_internal.h"
#include "ssm_vec.cuh"

namespace ssm {

namespace {
constexpr int kStepThreads = 128;
constexpr int kRows = 4;  // state rows per batch; a thread has one batch at work and one on its way
}  // namespace

template <typename T, typename Tout, int V>
__global__ void __launch_bounds__(kStepThreads) ssd_step_kernel(const SsdStepParams p, int cols, int slabs) {
  __shared__ float red[kStepThreads * V];
  const int slab = (int)(blockIdx.x % slabs);
  const int64_t bh = blockIdx.x / slabs, b = bh / p.H, hd = bh - b * p.H;
  const int P = (int)p.P, N = (int)p.N;
  const int c_lo = slab * cols;                       // first column of the slab
  const int n_col = min(cols, P - c_lo) / V;          // column groups of this CTA
  const int groups = kStepThreads / n_col;
  const int col = threadIdx.x % n_col, grp = threadIdx.x / n_col;
  const bool live = grp < groups;
  const int c0 = c_lo + col * V;
  float *hb = p.h + bh * p.N * p.P + c0;
  const T *Bp = static_cast<const T *>(p.B) + b * p.N, *Cp = static_cast<const T *>(p.C) + b * p.N;
  const T *xp = static_cast<const T *>(p.x) + bh * p.P + c0;
  struct Batch {
    alignas(16) float h[kRows][V];
    T B[kRows], C[kRows];
  };
  auto load = [&](int n0, Batch &q) {
#pragma unroll
    for (int k = 0; k < kRows; k++) {
      const int n = n0 + k * groups;
      if (live && n < N) {
        if constexpr (V == 4) {
          *reinterpret_cast<float4 *>(q.h[k]) = *reinterpret_cast<const float4 *>(hb + (int64_t)n * P);
        } else {
          q.h[k][0] = hb[(int64_t)n * P];
        }
        q.B[k] = Bp[n];
        q.C[k] = Cp[n];
      }
    }
  };
  Batch cur, nxt;
  load(grp, cur);  // on its way while the head's factors are formed
  float x[V], y[V];
#pragma unroll
  for (int j = 0; j < V; j++) {
    x[j] = live ? to_f32(xp[j]) : 0.f;
    y[j] = 0.f;
  }
  const float dv = to_f32(static_cast<const T *>(p.dt)[bh]) + (p.dt_bias ? p.dt_bias[hd] : 0.f);
  const float rate = expf(p.A_log[hd]);
  const float delta = p.delta_softplus ? softplus<true>(dv) : dv;
  // two functions: 1 + expm1 would lose a small a's digits, exp - 1 those of a small step
  const float a = expf(-delta * rate), beta = p.euler ? delta : -expm1f(-delta * rate) / rate;
  for (int n0 = grp; n0 < N; n0 += groups * kRows) {
    load(n0 + groups * kRows, nxt);
#pragma unroll
    for (int k = 0; k < kRows; k++) {
      const int n = n0 + k * groups;
      if (live && n < N) {
        const float in = beta * to_f32(cur.B[k]), out = to_f32(cur.C[k]);
#pragma unroll
        for (int j = 0; j < V; j++) {
          cur.h[k][j] = fmaf(a, cur.h[k][j], in * x[j]);
          y[j] = fmaf(out, cur.h[k][j], y[j]);
        }
        if constexpr (V == 4) {
          *reinterpret_cast<float4 *>(hb + (int64_t)n * P) = *reinterpret_cast<const float4 *>(cur.h[k]);
        } else {
          hb[(int64_t)n * P] = cur.h[k][0];
        }
      }
    }
    cur = nxt;
  }
  // sums over the row groups, in their order
  const int width = n_col * V;
  if (live) {
#pragma unroll
    for (int j = 0; j < V; j++) red[grp * width + col * V + j] = y[j];
  }
  __syncthreads();
  for (int j = threadIdx.x; j < width; j += kStepThreads) {
    float s = 0.f;
    for (int g = 0; g < groups; g++) s += red[g * width + j];
    const int64_t at = bh * p.P + c_lo + j;
    s = fmaf(p.D ? p.D[hd] : 0.f, to_f32(static_cast<const T *>(p.x)[at]), s);
    static_cast<Tout *>(p.out)[at] = from_f32<Tout>(s);
  }
}

namespace {
template <typename T, typename Tout> cudaError_t step_t(const SsdStepParams &p, cudaStream_t s) {
  const int64_t heads = p.Bt * p.H;
  const int V = p.vec ? 4 : 1;
  // whole heads where those give two CTAs per SM, else slabs of at least 16 columns (64-byte runs)
  int cols = (int)p.P, slabs = 1;
  if (cols / V > kStepThreads) cols = (cols + 1) / 2;  // a thread per column group (P <= 256)
  slabs = (int)((p.P + cols - 1) / cols);
  while (heads * slabs < 2 * 148 && cols >= 32 && cols % (2 * V) == 0) cols /= 2, slabs *= 2;
  slabs = (int)((p.P + cols - 1) / cols);
  if (heads * slabs > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const unsigned grid = (unsigned)(heads * slabs);
  if (p.vec)
    ssd_step_kernel<T, Tout, 4><<<grid, kStepThreads, 0, s>>>(p, cols, slabs);
  else
    ssd_step_kernel<T, Tout, 1><<<grid, kStepThreads, 0, s>>>(p, cols, slabs);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_ssd_step(const SsdStepParams &p, int in_bf16, int out_bf16, cudaStream_t s) {
  if (in_bf16) return out_bf16 ? step_t<__nv_bfloat16, __nv_bfloat16>(p, s) : step_t<__nv_bfloat16, float>(p, s);
  return out_bf16 ? step_t<float, __nv_bfloat16>(p, s) : step_t<float, float>(p, s);
}

}  // namespace ssm
