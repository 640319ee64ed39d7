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
// the block that owns the token and shared by all its heads.  A lane group goes
// along the heads of one token, two of q and two of k at a time with the next
// ones on the way (16384 x (16 + 16) x 128 bf16: one row at a time 72 us, two 53,
// with the next on the way 48, 86% of the copy rate).  With few heads the lane
// groups take several tokens side by side.  Dealing rows out freely, each with
// its own token and head, takes half as many instructions again (62 us).
#include "kda_common.cuh"
#include "kda_layer.h"

namespace kda {

namespace {

constexpr int kThreads = 128;
constexpr int kMaxTokens = 16;  // tokens of a block's step
constexpr int kRows = 2;        // rows of a lane's batch
constexpr int kMaxBlocks = 148 * 8;  // of the gradient: each leaves a row of weight sums

__device__ __forceinline__ float2 splat(float x) { return make_float2(x, x); }

// A lane's eight channels as its four pairs (lo, hi), two pairs a register pair:
// the halves of every rotated pair lie in lo and in hi.
struct Row {
  float2 lo[2], hi[2];
};
// The two groups of four channels as they lie in memory, and their pairs:
// (a[i], b[i]), or neighbours when interleaved.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint2 a, b;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, const __nv_bfloat16* q) {
    a = *reinterpret_cast<const uint2*>(p);
    b = *reinterpret_cast<const uint2*>(q);
  }
  __device__ __forceinline__ void clear() { a = b = make_uint2(0u, 0u); }
  template <bool kPairs>
  __device__ __forceinline__ Row get() const {
    auto l = [](uint32_t u) { return __uint_as_float(u << 16); };
    auto h = [](uint32_t u) { return __uint_as_float(u & 0xffff0000u); };
    if (kPairs)
      return Row{{make_float2(l(a.x), l(a.y)), make_float2(l(b.x), l(b.y))},
                 {make_float2(h(a.x), h(a.y)), make_float2(h(b.x), h(b.y))}};
    return Row{{make_float2(l(a.x), h(a.x)), make_float2(l(a.y), h(a.y))},
               {make_float2(l(b.x), h(b.x)), make_float2(l(b.y), h(b.y))}};
  }
};
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p, const float* q) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(q);
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  template <bool kPairs>
  __device__ __forceinline__ Row get() const {
    if (kPairs)
      return Row{{make_float2(a.x, a.z), make_float2(b.x, b.z)},
                 {make_float2(a.y, a.w), make_float2(b.y, b.w)}};
    return Row{{make_float2(a.x, a.y), make_float2(a.z, a.w)},
               {make_float2(b.x, b.y), make_float2(b.z, b.w)}};
  }
};
// The inverse of Raw::get: the two groups of four channels.
template <bool kPairs>
__device__ __forceinline__ void groups_of(const Row& r, float4& a, float4& b) {
  if (kPairs) {
    a = make_float4(r.lo[0].x, r.hi[0].x, r.lo[0].y, r.hi[0].y);
    b = make_float4(r.lo[1].x, r.hi[1].x, r.lo[1].y, r.hi[1].y);
  } else {
    a = make_float4(r.lo[0].x, r.lo[0].y, r.lo[1].x, r.lo[1].y);
    b = make_float4(r.hi[0].x, r.hi[0].y, r.hi[1].x, r.hi[1].y);
  }
}
__device__ __forceinline__ void st4(__nv_bfloat16* p, float4 f) {
  __nv_bfloat162 a = __floats2bfloat162_rn(f.x, f.y), b = __floats2bfloat162_rn(f.z, f.w);
  uint2 u;
  u.x = *reinterpret_cast<uint32_t*>(&a);
  u.y = *reinterpret_cast<uint32_t*>(&b);
  *reinterpret_cast<uint2*>(p) = u;
}
__device__ __forceinline__ void st4(float* p, float4 f) { *reinterpret_cast<float4*>(p) = f; }

__device__ __forceinline__ Row mul(const Row& a, const Row& b) {
  Row r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    r.lo[i] = __fmul2_rn(a.lo[i], b.lo[i]);
    r.hi[i] = __fmul2_rn(a.hi[i], b.hi[i]);
  }
  return r;
}
__device__ __forceinline__ Row scale(const Row& a, float f) {
  Row r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    r.lo[i] = __fmul2_rn(a.lo[i], splat(f));
    r.hi[i] = __fmul2_rn(a.hi[i], splat(f));
  }
  return r;
}
__device__ __forceinline__ Row fma(const Row& a, const Row& b, const Row& c) {
  Row r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    r.lo[i] = __ffma2_rn(a.lo[i], b.lo[i], c.lo[i]);
    r.hi[i] = __ffma2_rn(a.hi[i], b.hi[i], c.hi[i]);
  }
  return r;
}
__device__ __forceinline__ float dot(const Row& a, const Row& b) {
  float2 s = __fmul2_rn(a.lo[0], b.lo[0]);
  s = __ffma2_rn(a.lo[1], b.lo[1], s);
  s = __ffma2_rn(a.hi[0], b.hi[0], s);
  s = __ffma2_rn(a.hi[1], b.hi[1], s);
  return s.x + s.y;
}

// Sum over the G lanes of a head row.
template <int G>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The lane's four pairs turned by the angles with these cosines and sines.
__device__ __forceinline__ Row turn(const Row& v, const float2 (&c)[2], const float2 (&s)[2]) {
  Row r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 n = __fmul2_rn(s[i], splat(-1.f));
    r.lo[i] = __ffma2_rn(v.lo[i], c[i], __fmul2_rn(v.hi[i], n));
    r.hi[i] = __ffma2_rn(v.hi[i], c[i], __fmul2_rn(v.lo[i], s[i]));
  }
  return r;
}

// across: lane groups along the heads (a power of two); the others take other tokens.
template <typename T, int D, bool kPairs>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 7 : 4)
    qk_kernel(const QkArgs a, int tokens, int across) {
  constexpr int G = D / 8;            // lanes of a row
  constexpr int SLOTS = kThreads / G; // rows of a pass
  constexpr int U = kRows;
  __shared__ __align__(16) float s_cos[kMaxTokens][D / 2], s_sin[kMaxTokens][D / 2];
  __shared__ double s_freq[D / 2];  // turns per position
  const int l = threadIdx.x % G, slot = threadIdx.x / G;
  const int half = a.rot / 2;
  const bool turned = 8 * l < a.rot;
  const int o1 = !kPairs && turned ? 4 * l : 8 * l;
  const int o2 = (!kPairs && turned ? half + 4 * l : 8 * l + 4) - o1;
  const int lane_token = slot / across, lane_head = slot % across, side_by_side = SLOTS / across;
  const int most = max(a.side[0].heads, a.side[1].heads);
  Row weight[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    Raw<float> w;
    w.a = w.b = make_float4(1.f, 1.f, 1.f, 1.f);
    if (a.side[s].weight) w.load(a.side[s].weight + o1, a.side[s].weight + o1 + o2);
    weight[s] = w.template get<kPairs>();
  }
  for (int i = threadIdx.x; i < half; i += kThreads) s_freq[i] = a.freqs[i] * 0.15915494309189533577;

  for (int64_t t0 = (int64_t)blockIdx.x * tokens; t0 < a.T; t0 += (int64_t)gridDim.x * tokens) {
    const int count = (int)(a.T - t0 < tokens ? a.T - t0 : tokens);
    // heads h0.. of token k0 + lane_token of the step: two rows of either side
    Raw<T> next[2][U];
    auto load = [&](int k0, int h0) {
      const bool here = k0 + lane_token < count;
      const int64_t t = t0 + (here ? k0 + lane_token : 0);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const QkSide& q = a.side[s];
        const T* p = (const T*)q.x + t * q.x_stride + (h0 + lane_head) * D + o1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (here && h0 + u * across + lane_head < q.heads)
            next[s][u].load(p + u * across * D, p + u * across * D + o2);
          else
            next[s][u].clear();
        }
      }
    };
    load(0, 0);
    __syncthreads();  // the last step's sines are read
    for (int i = threadIdx.x; i < count * half; i += kThreads) {
      // in turns, reduced to [-1/2, 1/2] in 64 bits; the rest fits 32
      const int k = i / half, f = i - k * half;
      const double turns = (double)a.positions[t0 + k] * s_freq[f];
      float sn, cn;
      sincospif(2.f * (float)(turns - rint(turns)), &sn, &cn);
      s_cos[k][f] = cn;
      s_sin[k][f] = sn;
    }
    __syncthreads();
    for (int k0 = 0, h0 = 0; k0 < count;) {
      Raw<T> x[2][U];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int u = 0; u < U; ++u) x[s][u] = next[s][u];
      const int at = h0, k = k0 + lane_token;
      const bool here = k < count;
      h0 += across * U;
      if (h0 >= most) {
        h0 = 0;
        k0 += side_by_side;
      }
      if (k0 < count) load(k0, h0);
      float2 c[2], sn[2];
      if (turned) {
        const float4 c4 = *reinterpret_cast<const float4*>(&s_cos[here ? k : 0][4 * l]);
        const float4 s4 = *reinterpret_cast<const float4*>(&s_sin[here ? k : 0][4 * l]);
        c[0] = make_float2(c4.x, c4.y);
        c[1] = make_float2(c4.z, c4.w);
        sn[0] = make_float2(s4.x, s4.y);
        sn[1] = make_float2(s4.z, s4.w);
      }
      const int64_t t = t0 + (here ? k : 0);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const QkSide& q = a.side[s];
        T* p = (T*)q.out + t * q.out_stride + (at + lane_head) * D + o1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int h = at + u * across;
          if (h >= q.heads) break;
          const Row v = x[s][u].template get<kPairs>();
          const float rn = rsqrtf(row_sum<G>(dot(v, v)) * (1.f / D) + a.eps);
          Row out = mul(v, scale(weight[s], rn));
          if (turned) out = turn(out, c, sn);
          if (here && h + lane_head < q.heads) {
            float4 f1, f2;
            groups_of<kPairs>(out, f1, f2);
            st4(p + u * across * D, f1);
            st4(p + u * across * D + o2, f2);
          }
        }
      }
    }
  }
}

// The gradient walks likewise, one side at a time (its two inputs a row take the
// registers of the other side): 16384 x (16 + 16) x 128 bf16 88 us, 70% of the
// copy rate; 94 with rows dealt out freely.
template <typename T, int D, bool kPairs>
__global__ void __launch_bounds__(kThreads, 4)
    qk_backward_kernel(const QkArgs a, int tokens, int across, float* part) {
  constexpr int G = D / 8;            // lanes of a row
  constexpr int SLOTS = kThreads / G; // rows of a pass
  constexpr int U = kRows;
  __shared__ __align__(16) float s_cos[kMaxTokens][D / 2], s_sin[kMaxTokens][D / 2];
  __shared__ __align__(16) float s_dw[2][SLOTS][D];
  __shared__ double s_freq[D / 2];  // turns per position
  const int l = threadIdx.x % G, slot = threadIdx.x / G;
  const int half = a.rot / 2;
  const bool turned = 8 * l < a.rot;
  const int o1 = !kPairs && turned ? 4 * l : 8 * l;
  const int o2 = (!kPairs && turned ? half + 4 * l : 8 * l + 4) - o1;
  const int lane_token = slot / across, lane_head = slot % across, side_by_side = SLOTS / across;
  Row weight[2], dw[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    Raw<float> w;
    w.a = w.b = make_float4(1.f, 1.f, 1.f, 1.f);
    if (a.side[s].weight) w.load(a.side[s].weight + o1, a.side[s].weight + o1 + o2);
    weight[s] = w.template get<kPairs>();
    dw[s] = Row{{splat(0.f), splat(0.f)}, {splat(0.f), splat(0.f)}};
  }
  for (int i = threadIdx.x; i < half; i += kThreads) s_freq[i] = a.freqs[i] * 0.15915494309189533577;
  const int first_side = a.side[0].heads > 0 ? 0 : 1;
  const bool both = a.side[0].heads > 0 && a.side[1].heads > 0;

  for (int64_t t0 = (int64_t)blockIdx.x * tokens; t0 < a.T; t0 += (int64_t)gridDim.x * tokens) {
    const int count = (int)(a.T - t0 < tokens ? a.T - t0 : tokens);
    // heads h0.. of side s of token k0 + lane_token of the step
    Raw<T> next_x[U], next_d[U];
    auto load = [&](int k0, int s, int h0) {
      const bool here = k0 + lane_token < count;
      const int64_t t = t0 + (here ? k0 + lane_token : 0);
      const QkSide& q = a.side[s];
      const int at = (h0 + lane_head) * D + o1;
      const T* p = (const T*)q.x + t * q.x_stride + at;
      const T* g = (const T*)q.dout + t * q.dout_stride + at;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (here && h0 + u * across + lane_head < q.heads) {
          next_x[u].load(p + u * across * D, p + u * across * D + o2);
          next_d[u].load(g + u * across * D, g + u * across * D + o2);
        } else {
          next_x[u].clear();
          next_d[u].clear();
        }
      }
    };
    load(0, first_side, 0);
    __syncthreads();  // the last step's sines are read
    for (int i = threadIdx.x; i < count * half; i += kThreads) {
      // in turns, reduced to [-1/2, 1/2] in 64 bits; the rest fits 32
      const int k = i / half, f = i - k * half;
      const double turns = (double)a.positions[t0 + k] * s_freq[f];
      float sn, cn;
      sincospif(2.f * (float)(turns - rint(turns)), &sn, &cn);
      s_cos[k][f] = cn;
      s_sin[k][f] = -sn;  // the gradient turns back
    }
    __syncthreads();
    for (int k0 = 0, s = first_side, h0 = 0; k0 < count;) {
      Raw<T> x[U], d[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        x[u] = next_x[u];
        d[u] = next_d[u];
      }
      const int at = h0, k = k0 + lane_token, side = s;
      const bool here = k < count;
      h0 += across * U;
      if (h0 >= a.side[s].heads) {
        h0 = 0;
        if (both && s == 0) {
          s = 1;
        } else {
          s = first_side;
          k0 += side_by_side;
        }
      }
      if (k0 < count) load(k0, s, h0);
      const QkSide& q = a.side[side];
      float2 c[2], sn[2];
      if (turned) {
        const float4 c4 = *reinterpret_cast<const float4*>(&s_cos[here ? k : 0][4 * l]);
        const float4 s4 = *reinterpret_cast<const float4*>(&s_sin[here ? k : 0][4 * l]);
        c[0] = make_float2(c4.x, c4.y);
        c[1] = make_float2(c4.z, c4.w);
        sn[0] = make_float2(s4.x, s4.y);
        sn[1] = make_float2(s4.z, s4.w);
      }
      Row w;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w.lo[i] = side ? weight[1].lo[i] : weight[0].lo[i];
        w.hi[i] = side ? weight[1].hi[i] : weight[0].hi[i];
      }
      T* p = (T*)q.out + (t0 + (here ? k : 0)) * q.out_stride + (at + lane_head) * D + o1;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = at + u * across;
        if (h >= q.heads) break;
        const bool in = here && h + lane_head < q.heads;
        const Row v = x[u].template get<kPairs>();
        Row b = d[u].template get<kPairs>();
        const float rn = rsqrtf(row_sum<G>(dot(v, v)) * (1.f / D) + a.eps);
        if (turned) b = turn(b, c, sn);
        const Row vr = scale(v, rn);
        if (in) {  // rn is inf off the rows at eps 0
          if (side) dw[1] = fma(b, vr, dw[1]);
          else dw[0] = fma(b, vr, dw[0]);
        }
        b = mul(b, w);
        // r (c - v r^2 mean(c v)) = r c - (v r) r mean(c (v r))
        const float m = row_sum<G>(dot(b, vr)) * (-1.f / D) * rn;
        Row ms;
        ms.lo[0] = ms.lo[1] = ms.hi[0] = ms.hi[1] = splat(m);
        const Row out = fma(vr, ms, scale(b, rn));
        if (in) {
          float4 f1, f2;
          groups_of<kPairs>(out, f1, f2);
          st4(p + u * across * D, f1);
          st4(p + u * across * D + o2, f2);
        }
      }
    }
  }
  if (part) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float4 f1, f2;
      groups_of<kPairs>(dw[s], f1, f2);
      st4(&s_dw[s][slot][o1], f1);
      st4(&s_dw[s][slot][o1 + o2], f2);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
      float v = 0.f;
      for (int r = 0; r < SLOTS; ++r) v += s_dw[i / D][r][i % D];
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

// Tokens of a block's step and blocks.  One token a step while that fills the GPU
// no more than twice (the smallest calls are bound by latency); above, four (the
// sines of four tokens are formed in one go) or `enough`.  Blocks go on in strides.
void steps_for(int T, int enough, int most_blocks, int& tokens, int& blocks) {
  tokens = 1;
  if (T > 148 * 16) {
    tokens = 4;
    while (tokens < kMaxTokens && tokens < enough) tokens *= 2;
  }
  const int64_t b = ((int64_t)T + tokens - 1) / tokens;
  blocks = (int)(b < 1 ? 1 : b > most_blocks ? most_blocks : b);
}

template <typename T, int D, bool kPairs>
cudaError_t launch_k(const QkArgs& a, bool back) {
  constexpr int SLOTS = kThreads / (D / 8);
  const int hq = a.side[0].heads, hk = a.side[1].heads;
  int tokens, blocks;
  // lane groups along the heads: two heads of the larger side each, up to the
  // block's; the others take tokens side by side
  int across = 1;
  while (across * kRows < (hq > hk ? hq : hk) && across < SLOTS) across *= 2;
  steps_for(a.T, SLOTS / across, back ? kMaxBlocks : 148 * 64, tokens, blocks);
  if (!back) {
    qk_kernel<T, D, kPairs><<<blocks, kThreads, 0, a.stream>>>(a, tokens, across);
    return cudaGetLastError();
  }
  const bool weights = a.side[0].dweight || a.side[1].dweight;
  qk_backward_kernel<T, D, kPairs>
      <<<blocks, kThreads, 0, a.stream>>>(a, tokens, across, weights ? (float*)a.ws : nullptr);
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess || !weights) return err;
  qk_weight_kernel<<<2 * D, 128, 0, a.stream>>>((const float*)a.ws, blocks, D,
                                                a.side[0].dweight, a.side[1].dweight);
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
  const int blocks = T < 1 ? 1 : T < kMaxBlocks ? T : kMaxBlocks;
  return (size_t)blocks * 2 * d * sizeof(float);
}

cudaError_t launch_qk_norm_rope(const QkArgs& a) { return launch(a, false); }
cudaError_t launch_qk_norm_rope_backward(const QkArgs& a) { return launch(a, true); }

}  // namespace kda
