// kda_qk_rope.cu -- RMS norm of every query and key head and the position
// rotation of its channel pairs in one pass, and the gradient of that pass.
//
//   n = v r w, r = 1/sqrt(mean v^2 + eps);  out = R(angle) n
//   b = R^T dout, c = b w;  dv = r (c - v r^2 mean(c v));  dw = sum b v r
//
// HBM-bound: one read of each input row, one write.  D / 8 lanes own one head
// row of D numbers; a lane holds two groups of four channels, placed so that
// every rotated pair lies in one lane: (4l.., rot/2 + 4l..) when channel i is
// paired with i + rot/2, 8 consecutive channels otherwise.  So a row needs
// shuffles only for its sums, and a lane needs the sines of four angles
// whatever the layout.  The sines of a token's rot/2 angles are formed once by
// the block that owns the token and shared by all its heads.
#include "kda_common.cuh"
#include "kda_launch.h"

namespace kda {

namespace {

constexpr int kThreads = 128;
constexpr int kTokens = 4;  // tokens of one block's step
constexpr int kMaxBlocks = 148 * 8;

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

// Sum over the G lanes of a head row.
template <int G>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Turns the lane's four pairs by (cos, sin); neg: by the opposite angle.
// Pairs are (v[2i], v[2i+1]) when interleaved, else (v[i], v[4+i]).
__device__ __forceinline__ void turn(float* v, const float2* cs, bool interleaved, bool neg) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int ia = interleaved ? 2 * i : i, ib = interleaved ? 2 * i + 1 : 4 + i;
    const float c = cs[i].x, s = neg ? -cs[i].y : cs[i].y;
    const float x = v[ia], y = v[ib];
    v[ia] = x * c - y * s;
    v[ib] = y * c + x * s;
  }
}

template <typename T, int D, bool kPairs, bool kBack>
__global__ void __launch_bounds__(kThreads) qk_kernel(const QkArgs a, float* part) {
  constexpr int G = D / 8;             // lanes of a row
  constexpr int ROWS = kThreads / G;   // rows of a pass
  __shared__ float2 s_cs[kTokens][D / 2];
  __shared__ float s_dw[kBack ? 2 : 1][kBack ? ROWS : 1][D];
  const int l = threadIdx.x % G, row = threadIdx.x / G;
  const int half = a.rot / 2;
  const bool turned = 8 * l < a.rot;
  const int o1 = !kPairs && turned ? 4 * l : 8 * l;
  const int o2 = !kPairs && turned ? half + 4 * l : 8 * l + 4;
  float w[2][8], dw[2][8] = {};
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w[s][e] = a.side[s].weight ? a.side[s].weight[o1 + e] : 1.f;
      w[s][4 + e] = a.side[s].weight ? a.side[s].weight[o2 + e] : 1.f;
    }
  for (int64_t t0 = (int64_t)blockIdx.x * kTokens; t0 < a.T; t0 += (int64_t)gridDim.x * kTokens) {
    const int count = (int)(a.T - t0 < kTokens ? a.T - t0 : kTokens);
    __syncthreads();
    for (int i = threadIdx.x; i < count * half; i += kThreads) {
      // in turns, reduced to [-1/2, 1/2] in 64 bits; the rest fits 32
      const double turns = (double)a.positions[t0 + i / half] *
                           (a.freqs[i % half] * 0.15915494309189533577);
      float s, c;
      sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
      s_cs[i / half][i % half] = make_float2(c, s);
    }
    __syncthreads();
    for (int k = 0; k < count; ++k) {
      float2 cs[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) cs[i] = turned ? s_cs[k][4 * l + i] : make_float2(1.f, 0.f);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const QkSide& q = a.side[s];
        const T* x = (const T*)q.x + (t0 + k) * q.x_stride;
        T* out = (T*)q.out + (t0 + k) * q.out_stride;
        for (int h0 = 0; h0 < q.heads; h0 += ROWS) {
          const int h = h0 + row;
          const bool in = h < q.heads;
          float v[8] = {}, b[8] = {};
          if (in) {
            ld4<T>(x + h * D + o1, v);
            ld4<T>(x + h * D + o2, v + 4);
            if (kBack) {
              const T* d = (const T*)q.dout + (t0 + k) * q.dout_stride + h * D;
              ld4<T>(d + o1, b);
              ld4<T>(d + o2, b + 4);
            }
          }
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(v[e], v[e], ss);
          const float r = rsqrtf(row_sum<G>(ss) * (1.f / D) + a.eps);
          if (!kBack) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= r * w[s][e];
            if (turned) turn(v, cs, kPairs, false);
          } else {
            if (turned) turn(b, cs, kPairs, true);
            float cv = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              if (in) dw[s][e] = fmaf(b[e], v[e] * r, dw[s][e]);  // r is inf off the rows at eps 0
              b[e] *= w[s][e];
              cv = fmaf(b[e], v[e], cv);
            }
            const float m = row_sum<G>(cv) * (1.f / D) * r * r;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = r * (b[e] - v[e] * m);
          }
          if (in) {
            st4<T>(out + h * D + o1, v);
            st4<T>(out + h * D + o2, v + 4);
          }
        }
      }
    }
  }
  if (kBack && part) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s_dw[s][row][o1 + e] = dw[s][e];
        s_dw[s][row][o2 + e] = dw[s][4 + e];
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
      float v = 0.f;
      for (int r = 0; r < ROWS; ++r) v += s_dw[i / D][r][i % D];
      part[(size_t)blockIdx.x * 2 * D + i] = v;
    }
  }
}

// dq_weight, dk_weight: the blocks' sums, added in order.
__global__ void __launch_bounds__(128)
    qk_weight_kernel(const float* part, int blocks, int d, float* dq, float* dk) {
  __shared__ float s_sum[128];
  const int i = blockIdx.x;
  float v = 0.f;
  for (int b = threadIdx.x; b < blocks; b += 128) v += part[(size_t)b * 2 * d + i];
  s_sum[threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    v = s_sum[threadIdx.x] + s_sum[threadIdx.x + 32] + s_sum[threadIdx.x + 64] +
        s_sum[threadIdx.x + 96];
    v = warp_sum(v);
    float* out = i < d ? dq : dk;
    if (threadIdx.x == 0 && out) out[i % d] = v;
  }
}

int blocks_for(int T) {
  const int b = (int)(((int64_t)T + kTokens - 1) / kTokens);
  return b < 1 ? 1 : b > kMaxBlocks ? kMaxBlocks : b;
}

template <typename T, int D, bool kPairs>
cudaError_t launch_k(const QkArgs& a, bool back) {
  const int grid = blocks_for(a.T);
  if (!back) {
    qk_kernel<T, D, kPairs, false><<<grid, kThreads, 0, a.stream>>>(a, nullptr);
    return cudaGetLastError();
  }
  const bool weights = a.side[0].dweight || a.side[1].dweight;
  qk_kernel<T, D, kPairs, true>
      <<<grid, kThreads, 0, a.stream>>>(a, weights ? (float*)a.ws : nullptr);
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess || !weights) return err;
  qk_weight_kernel<<<2 * D, 128, 0, a.stream>>>((const float*)a.ws, grid, D, a.side[0].dweight,
                                                a.side[1].dweight);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const QkArgs& a, bool back) {
  switch (a.d * 2 + (a.interleaved ? 1 : 0)) {
    case 64: return launch_k<T, 32, false>(a, back);
    case 65: return launch_k<T, 32, true>(a, back);
    case 128: return launch_k<T, 64, false>(a, back);
    case 129: return launch_k<T, 64, true>(a, back);
    case 256: return launch_k<T, 128, false>(a, back);
    case 257: return launch_k<T, 128, true>(a, back);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch(const QkArgs& a, bool back) {
  return a.bf16 ? launch_t<__nv_bfloat16>(a, back) : launch_t<float>(a, back);
}

}  // namespace

size_t qk_backward_workspace_bytes(int T, int d) {
  return (size_t)blocks_for(T) * 2 * d * sizeof(float);
}

cudaError_t launch_qk_norm_rope(const QkArgs& a) { return launch(a, false); }
cudaError_t launch_qk_norm_rope_backward(const QkArgs& a) { return launch(a, true); }

}  // namespace kda
