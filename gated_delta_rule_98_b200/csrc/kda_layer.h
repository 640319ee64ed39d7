// kda_layer.h -- host-side launch descriptors of the operators around the
// recurrence: gated scan, gradient of the input prologue, norm and rotation of
// the query and key heads (internal; not part of the C ABI).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

// Gradient of the input prologue.
struct ConvBackwardArgs {
  const void *x, *dy;  // [T, channels]
  const float* w;      // [channels, width]
  const int32_t* cu;   // nullptr = N equal sequences of L tokens
  int N, T, L, channels, width;
  bool bf16;
  void* dx;
  float* dw;
  void* ws;
  cudaStream_t stream;
};
size_t conv_backward_workspace_bytes(int T, int channels, int width);
cudaError_t launch_conv_swish_backward(const ConvBackwardArgs& a);

// Gated linear recurrence (z, A or g; dy set: its gradient).
struct ScanArgs {
  const void* x;      // [T, C] input
  const void* z;      // [T, C] gate input, with A; or null
  const float* A;     // [C]
  const float* g;     // [T, C] log-decay, or null
  const float* h0;    // [N, C] or null (zeros)
  const int32_t* cu;  // nullptr = N equal sequences of L tokens
  int N, T, L, C;
  bool bf16;
  void* y;         // [T, C]
  float* h_final;  // [N, C] or null
  float* states;   // [ceil(T / KDA_SCAN_INTERVAL), C]: written by the forward (or null), read by the backward
  void* ws;
  cudaStream_t stream;
  const void* dy = nullptr;  // [T, C]
  const float* dh_final = nullptr;
  void *dx = nullptr, *dz = nullptr;  // [T, C]
  float *dg = nullptr, *dA = nullptr, *dh0 = nullptr;
};
size_t scan_workspace_bytes(int T, int C);
cudaError_t launch_scan(const ScanArgs& a);
cudaError_t launch_scan_backward(const ScanArgs& a);
cudaError_t launch_scan_step(const void* x, const void* z, const float* A, float* h, int B, int C,
                             bool bf16, void* y, cudaStream_t stream);

// Norm and rotation of the query and key heads (dout set: the gradient).
struct QkSide {
  const void* x;     // [T, heads, d]
  const void* dout;  // gradient of the output, or null
  void* out;         // output, or the gradient of x
  const float* weight;  // [d] or null (ones)
  float* dweight;       // [d] or null
  long long x_stride, dout_stride, out_stride;  // elements between tokens
  int heads;
};
struct QkArgs {
  QkSide side[2];  // q, k
  const int32_t* positions;
  const double* freqs;
  float eps;
  int T, d, rot;
  bool interleaved, bf16;
  void* ws;
  cudaStream_t stream;
};
size_t qk_backward_workspace_bytes(int T, int d);
cudaError_t launch_qk_norm_rope(const QkArgs& a);
cudaError_t launch_qk_norm_rope_backward(const QkArgs& a);

}  // namespace kda
