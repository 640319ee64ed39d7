// kda_scan.cu -- gated linear recurrence of one number per channel, its
// gradients, and its single-token step.
//
//   z:  a = exp(-5 sigmoid(e^A z)),  h_t = a h_{t-1} + (1 - a) x_t
//   g:  a = exp(g),                  h_t = a h_{t-1} + x_t
//
// Backwards with l_t = dy_t + a_{t+1} l_{t+1}:  dx = (1 - a) l  (z) or l (g),
// dg = a (h_{t-1} - x) l  (z) or a h_{t-1} l (g).
//
// One thread owns one channel of one sequence and walks its tokens; the
// gradient walks them backwards in spans of 64 and recomputes the states of a
// span from the state that the forward saved at its start.
#include "kda_common.cuh"
#include "kda_launch.h"

namespace kda {

namespace {

constexpr int kSpan = 64;  // tokens between saved states (KDA_SCAN_INTERVAL)
constexpr int kThreads = 64;
constexpr int kGroups = 64;  // sequences walked at the same time

// Token range of sequence n, kept inside [0, T] whatever cu holds.
__device__ __forceinline__ void tokens_of(const ScanArgs& a, int n, int& t0, int& t1) {
  seq_bounds(a.cu, n, a.L, t0, t1);
  t0 = min(max(t0, 0), a.T);
  t1 = min(max(t1, t0), a.T);
}

struct Gate {
  float a, m, p;  // decay, input scale, s (1 - s) (z only)
};

template <typename T, bool kZ>
__device__ __forceinline__ Gate gate_of(const ScanArgs& a, size_t i, float expA) {
  if (kZ) {
    // 1 - s = e s with e = exp(-u): the difference would lose the digits of s near 1
    const float e = expf(-expA * to_f(((const T*)a.z)[i])), s = 1.f / (1.f + e);
    const float g = kGateMin * s;
    return {expf(g), -expm1f(g), s == 0.f ? 0.f : s * (s * e)};
  }
  return {expf(a.g[i]), 1.f, 0.f};
}

template <typename T, bool kZ>
__global__ void __launch_bounds__(kThreads) scan_kernel(const ScanArgs a) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= a.C) return;
  const float expA = kZ && a.T > 0 ? expf(a.A[c]) : 0.f;
  for (int n = blockIdx.y; n < a.N; n += gridDim.y) {
    int t0, t1;
  tokens_of(a, n, t0, t1);
  float h = a.h0 ? a.h0[(size_t)n * a.C + c] : 0.f;
  for (int t = t0; t < t1; ++t) {
    const size_t i = (size_t)t * a.C + c;
    if (a.states && t % kSpan == 0) a.states[(size_t)(t / kSpan) * a.C + c] = h;
    const Gate u = gate_of<T, kZ>(a, i, expA);
    h = fmaf(u.a, h, u.m * to_f(((const T*)a.x)[i]));
    ((T*)a.y)[i] = from_f<T>(h);
  }
  if (a.h_final) a.h_final[(size_t)n * a.C + c] = h;
  }
}

template <typename T, bool kZ>
__global__ void __launch_bounds__(kThreads) scan_backward_kernel(const ScanArgs a) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= a.C) return;
  const float expA = kZ && a.T > 0 ? expf(a.A[c]) : 0.f;
  float dA = 0.f;
  for (int n = blockIdx.y; n < a.N; n += gridDim.y) {
    int t0, t1;
  tokens_of(a, n, t0, t1);
  float back = a.dh_final ? a.dh_final[(size_t)n * a.C + c] : 0.f;
  float prev[kSpan];
  for (int e = t1; e > t0;) {
    const int b = max((e - 1) / kSpan * kSpan, t0);
    float h = b == t0 ? (a.h0 ? a.h0[(size_t)n * a.C + c] : 0.f)
                      : a.states[(size_t)(b / kSpan) * a.C + c];
    for (int t = b; t < e; ++t) {
      const size_t i = (size_t)t * a.C + c;
      const Gate u = gate_of<T, kZ>(a, i, expA);
      prev[t - b] = h;
      h = fmaf(u.a, h, u.m * to_f(((const T*)a.x)[i]));
    }
    for (int t = e - 1; t >= b; --t) {
      const size_t i = (size_t)t * a.C + c;
      const Gate u = gate_of<T, kZ>(a, i, expA);
      const float l = to_f(((const T*)a.dy)[i]) + back;
      back = u.a * l;
      ((T*)a.dx)[i] = from_f<T>(u.m * l);
      if (kZ) {
        const float d = back * (prev[t - b] - to_f(((const T*)a.x)[i])) * kGateMin * u.p *
                        expA;
        ((T*)a.dz)[i] = from_f<T>(d);
        dA = fmaf(d, to_f(((const T*)a.z)[i]), dA);
      } else {
        a.dg[i] = back * prev[t - b];
      }
    }
    e = b;
  }
  if (a.dh0) a.dh0[(size_t)n * a.C + c] = back;
  }
  if (kZ) ((float*)a.ws)[(size_t)blockIdx.y * a.C + c] = dA;
}

__global__ void __launch_bounds__(kThreads)
    sum_rows_kernel(const float* part, int rows, int C, float* out) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= C) return;
  float s = 0.f;
  for (int n = 0; n < rows; ++n) s += part[(size_t)n * C + c];
  out[c] = s;
}

template <typename T>
__global__ void __launch_bounds__(256)
    step_kernel(const T* x, const T* z, const float* A, float* h, size_t count, int C, T* y) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (size_t)gridDim.x * 256) {
    const float g = gate_logdecay(to_f(z[i]), expf(A[i % C]));
    const float v = fmaf(expf(g), h[i], -expm1f(g) * to_f(x[i]));
    h[i] = v;
    y[i] = from_f<T>(v);
  }
}

}  // namespace

size_t scan_workspace_bytes(int T, int C) { return (size_t)kGroups * C * sizeof(float); }

cudaError_t launch_scan(const ScanArgs& a) {
  const dim3 grid((a.C + kThreads - 1) / kThreads, min(a.N, kGroups));
  if (a.g) {
    if (a.bf16) scan_kernel<__nv_bfloat16, false><<<grid, kThreads, 0, a.stream>>>(a);
    else scan_kernel<float, false><<<grid, kThreads, 0, a.stream>>>(a);
  } else {
    if (a.bf16) scan_kernel<__nv_bfloat16, true><<<grid, kThreads, 0, a.stream>>>(a);
    else scan_kernel<float, true><<<grid, kThreads, 0, a.stream>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_scan_backward(const ScanArgs& a) {
  const dim3 grid((a.C + kThreads - 1) / kThreads, min(a.N, kGroups));
  if (!a.dA) {
    if (a.bf16) scan_backward_kernel<__nv_bfloat16, false><<<grid, kThreads, 0, a.stream>>>(a);
    else scan_backward_kernel<float, false><<<grid, kThreads, 0, a.stream>>>(a);
    return cudaGetLastError();
  }
  if (a.bf16) scan_backward_kernel<__nv_bfloat16, true><<<grid, kThreads, 0, a.stream>>>(a);
  else scan_backward_kernel<float, true><<<grid, kThreads, 0, a.stream>>>(a);
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  sum_rows_kernel<<<grid.x, kThreads, 0, a.stream>>>((const float*)a.ws, grid.y, a.C, a.dA);
  return cudaGetLastError();
}

cudaError_t launch_scan_step(const void* x, const void* z, const float* A, float* h, int B, int C,
                             bool bf16, void* y, cudaStream_t stream) {
  const size_t count = (size_t)B * C;
  const int grid = (int)(count / 256 < 148 * 8 ? (count + 255) / 256 : 148 * 8);
  if (bf16)
    step_kernel<<<grid, 256, 0, stream>>>((const __nv_bfloat16*)x, (const __nv_bfloat16*)z, A, h,
                                          count, C, (__nv_bfloat16*)y);
  else
    step_kernel<<<grid, 256, 0, stream>>>((const float*)x, (const float*)z, A, h, count, C,
                                          (float*)y);
  return cudaGetLastError();
}

}  // namespace kda
