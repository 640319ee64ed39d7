// kda_prologue_backward.cu -- gradient of the input prologue (causal depthwise
// short convolution along each sequence's tokens, then Swish):
//
//   u = conv(x), p = sigmoid(u), du = dy p (1 + u (1 - p))
//   dx[s] = sum_j w[W-1-j] du[s+j],   dw[W-1-j] = sum_t du[t] x[t-j]
//
// A thread owns kVec channels of a run of tokens and slides along it: u needs
// the W - 1 inputs before a token (a register window), dx of a token is
// complete W - 1 tokens later (a register window of unfinished sums), so each
// run reads W - 1 halo rows on either side and every row is read once more at
// most from cache.  A block's 8 warps take 8 runs that follow one another for
// the same channels and add their dw through shared memory; the blocks' sums
// are added by a second launch, in a fixed order.
#include "kda_common.cuh"
#include "kda_launch.h"

namespace kda {

namespace {

constexpr int kVec = 4;    // channels of one thread: 8-byte bf16 vectors
constexpr int kWarps = 8;  // runs of one block
constexpr int kMaxSplits = 512;

template <typename T>
__device__ __forceinline__ void ld4(const T* p, float* f);
template <>
__device__ __forceinline__ void ld4<__nv_bfloat16>(const __nv_bfloat16* p, float* f) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  f[0] = __uint_as_float(u.x << 16); f[1] = __uint_as_float(u.x & 0xffff0000u);
  f[2] = __uint_as_float(u.y << 16); f[3] = __uint_as_float(u.y & 0xffff0000u);
}
template <>
__device__ __forceinline__ void ld4<float>(const float* p, float* f) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
}
template <typename T>
__device__ __forceinline__ void st4(T* p, const float* f);
template <>
__device__ __forceinline__ void st4<__nv_bfloat16>(__nv_bfloat16* p, const float* f) {
  __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
  uint2 u;
  u.x = *reinterpret_cast<uint32_t*>(&a);
  u.y = *reinterpret_cast<uint32_t*>(&b);
  *reinterpret_cast<uint2*>(p) = u;
}
template <>
__device__ __forceinline__ void st4<float>(float* p, const float* f) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}

// First token of the sequence that holds token t, and the first boundary after
// t; both kept in range whatever cu holds ([0, t] and [t + 1, end]).
__device__ __forceinline__ void sequence_at(const ConvBackwardArgs& a, int end, int t, int& start,
                                            int& next) {
  if (!a.cu) {
    start = a.L > 0 ? t / a.L * a.L : 0;
    next = a.L > 0 ? min(start + a.L, end) : end;
    return;
  }
  int lo = 0, hi = a.N;  // first m in [0, N) with cu[m] > t, else N
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a.cu[mid] > t) hi = mid; else lo = mid + 1;
  }
  start = lo > 0 ? min(max(a.cu[lo - 1], 0), t) : 0;
  next = min(max(a.cu[lo], t + 1), end);
}

template <typename T, int W>
__global__ void __launch_bounds__(kWarps * 32)
    conv_swish_backward_kernel(const ConvBackwardArgs a, int run, float* part) {
  constexpr int H = W - 1;
  __shared__ float s_dw[kWarps][W][32 * kVec];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = (blockIdx.x * 32 + lane) * kVec;
  const bool in = c0 < a.channels;
  const int end = a.cu ? min(max(a.cu[a.N], 0), a.T) : a.T;
  float dw[W][kVec] = {};
  for (int64_t tile = blockIdx.y; tile * kWarps * run < end; tile += gridDim.y) {
    const int64_t r0 = (tile * kWarps + warp) * run;
    if (!in || r0 >= end) continue;
    const int t0 = (int)r0, t1 = min(t0 + run, end), t2 = min(t1 + H, end);
    const size_t C = a.channels;
    const T* x = (const T*)a.x + c0;
    const T* dy = (const T*)a.dy + c0;
    T* dx = (T*)a.dx + c0;
    float w[W][kVec];
#pragma unroll
    for (int i = 0; i < W; ++i)
#pragma unroll
      for (int e = 0; e < kVec; ++e) w[i][e] = a.w[(size_t)(c0 + e) * W + i];
    int start, next;
    sequence_at(a, end, t0, start, next);
    // win[j] = x of token t - H + j; sum[j] = dx of token t - H + j so far
    float win[H + 1][kVec], sum[H + 1][kVec];
#pragma unroll
    for (int j = 0; j < H; ++j) {
#pragma unroll
      for (int e = 0; e < kVec; ++e) win[j][e] = sum[j][e] = 0.f;
      if (t0 - H + j >= start) ld4<T>(x + (t0 - H + j) * C, win[j]);
    }
    int emit = t0;  // dx of tokens below this one is written or belongs to another run
    for (int t = t0; t < t2; ++t) {
      if (t == next) {
        // a sequence starts: the last one's unfinished sums are complete, nothing is carried
#pragma unroll
        for (int j = 0; j < H; ++j) {
          const int s = t - H + j;
          if (s >= emit && s < t1) st4<T>(dx + s * C, sum[j]);
#pragma unroll
          for (int e = 0; e < kVec; ++e) win[j][e] = sum[j][e] = 0.f;
        }
        emit = t;
        sequence_at(a, end, t, start, next);
      }
      float dyv[kVec], du[kVec];
      ld4<T>(x + t * C, win[H]);
      ld4<T>(dy + t * C, dyv);
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        float u = w[H][e] * win[H][e];
#pragma unroll
        for (int i = 0; i < H; ++i) u = fmaf(w[i][e], win[i][e], u);
        const float p = out_sigmoid(u);
        du[e] = dyv[e] * p * fmaf(u, 1.f - p, 1.f);
        sum[H][e] = 0.f;
#pragma unroll
        for (int j = 0; j <= H; ++j) sum[j][e] = fmaf(w[H - (H - j)][e], du[e], sum[j][e]);
        if (t < t1)
#pragma unroll
          for (int i = 0; i < W; ++i) dw[i][e] = fmaf(du[e], win[i][e], dw[i][e]);
      }
      if (t - H >= emit && t - H < t1) st4<T>(dx + (t - H) * C, sum[0]);
#pragma unroll
      for (int j = 0; j < H; ++j)
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          win[j][e] = win[j + 1][e];
          sum[j][e] = sum[j + 1][e];
        }
    }
    // the tokens whose later rows lie past the end
#pragma unroll
    for (int j = 0; j < H; ++j) {
      const int s = t2 - H + j;
      if (s >= emit && s < t1) st4<T>(dx + s * C, sum[j]);
    }
  }
#pragma unroll
  for (int i = 0; i < W; ++i)
#pragma unroll
    for (int e = 0; e < kVec; ++e) s_dw[warp][i][lane * kVec + e] = dw[i][e];
  __syncthreads();
  for (int k = threadIdx.x; k < W * 32 * kVec; k += kWarps * 32) {
    const int i = k / (32 * kVec), e = k % (32 * kVec), c = blockIdx.x * 32 * kVec + e;
    float v = 0.f;
#pragma unroll
    for (int r = 0; r < kWarps; ++r) v += s_dw[r][i][e];
    if (c < a.channels) part[((size_t)blockIdx.y * a.channels + c) * W + i] = v;
  }
}

__global__ void __launch_bounds__(128)
    sum_splits_kernel(const float* part, int splits, size_t count, float* out) {
  const size_t i = (size_t)blockIdx.x * 128 + threadIdx.x;
  if (i >= count) return;
  float s = 0.f;
  for (int r = 0; r < splits; ++r) s += part[r * count + i];
  out[i] = s;
}

// Tokens of one run and blocks along the tokens.
void split(int T, int& run, int& splits) {
  run = 32;
  const int64_t tiles = ((int64_t)T + kWarps * run - 1) / (kWarps * run);
  splits = (int)(tiles < 1 ? 1 : tiles > kMaxSplits ? kMaxSplits : tiles);
}

template <typename T>
cudaError_t launch_t(const ConvBackwardArgs& a) {
  int run, splits;
  split(a.T, run, splits);
  float* part = (float*)a.ws;
  const dim3 grid((a.channels + 32 * kVec - 1) / (32 * kVec), splits);
  const int nt = kWarps * 32;
  switch (a.width) {
    case 1: conv_swish_backward_kernel<T, 1><<<grid, nt, 0, a.stream>>>(a, run, part); break;
    case 2: conv_swish_backward_kernel<T, 2><<<grid, nt, 0, a.stream>>>(a, run, part); break;
    case 3: conv_swish_backward_kernel<T, 3><<<grid, nt, 0, a.stream>>>(a, run, part); break;
    case 4: conv_swish_backward_kernel<T, 4><<<grid, nt, 0, a.stream>>>(a, run, part); break;
    default: return cudaErrorInvalidValue;
  }
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  const size_t count = (size_t)a.channels * a.width;
  sum_splits_kernel<<<(unsigned)((count + 127) / 128), 128, 0, a.stream>>>(part, splits, count,
                                                                           a.dw);
  return cudaGetLastError();
}

}  // namespace

size_t conv_backward_workspace_bytes(int T, int channels, int width) {
  int run, splits;
  split(T, run, splits);
  return (size_t)splits * channels * width * sizeof(float);
}

cudaError_t launch_conv_swish_backward(const ConvBackwardArgs& a) {
  return a.bf16 ? launch_t<__nv_bfloat16>(a) : launch_t<float>(a);
}

}  // namespace kda
