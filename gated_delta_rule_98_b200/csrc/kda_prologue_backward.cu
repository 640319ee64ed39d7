// kda_prologue_backward.cu -- gradient of the input prologue (causal depthwise
// short convolution along each sequence's tokens, then Swish):
//
//   u = conv(x), p = sigmoid(u), du = dy p (1 + u (1 - p))
//   dx[s] = sum_j w[W-1-j] du[s+j],   dw[W-1-j] = sum_t du[t] x[t-j]
//
// HBM-bound: x and dy read once, dx written once.  A lane owns 4 channels (a
// warp: 128, 256 bytes of a bf16 row) of a run of tokens and slides along it:
// u needs the W - 1 inputs before a token (a register window), dx of a token
// is complete W - 1 tokens later (a register window of unfinished sums), so a
// run computes W - 1 tokens twice and reads W - 1 more rows at either end,
// from cache.  Rows come by cp.async, 8 tokens at a time, into slots private to
// the warp, two groups ahead, so that no barrier joins the block and the loads
// in flight do not depend on the number of resident warps.  A block's 8 warps
// take 8 runs that follow one another and add their dw through shared memory;
// the blocks' sums are added by a second launch, in a fixed order.
//
// Measured, W = 4: 32768 x 6144 bf16 233 us (5.2 TB/s, 79% of the copy rate: 56% of
// the issue slots, 39% of the special function unit), 16384 x 4096 fp32 134 us (6.0
// TB/s, 92%).
#include "kda_common.cuh"
#include "kda_layer.h"

namespace kda {

namespace {

constexpr int kVec = 4;         // channels of a lane
constexpr int kWarps = 8;       // runs of a block
constexpr int kGroup = 8;       // tokens fetched together
constexpr int kSlots = 3;       // groups in flight or in use
constexpr int kCols = 32 * kVec;
constexpr int kMaxSplits = 512;

__device__ __forceinline__ float2 splat(float x) { return make_float2(x, x); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct Vec {
  float2 lo, hi;
};
__device__ __forceinline__ Vec ld4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return Vec{make_float2(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u)),
             make_float2(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u))};
}
__device__ __forceinline__ Vec ld4(const float* p) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  return Vec{make_float2(a.x, a.y), make_float2(a.z, a.w)};
}
__device__ __forceinline__ void st4(__nv_bfloat16* p, const Vec& v) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v.lo.x, v.lo.y),
                 b = __floats2bfloat162_rn(v.hi.x, v.hi.y);
  uint2 u;
  u.x = *reinterpret_cast<uint32_t*>(&a);
  u.y = *reinterpret_cast<uint32_t*>(&b);
  *reinterpret_cast<uint2*>(p) = u;
}
__device__ __forceinline__ void st4(float* p, const Vec& v) {
  *reinterpret_cast<float4*>(p) = make_float4(v.lo.x, v.lo.y, v.hi.x, v.hi.y);
}
__device__ __forceinline__ Vec zero() { return Vec{splat(0.f), splat(0.f)}; }
__device__ __forceinline__ Vec mul(const Vec& a, const Vec& b) {
  return Vec{__fmul2_rn(a.lo, b.lo), __fmul2_rn(a.hi, b.hi)};
}
__device__ __forceinline__ Vec fma(const Vec& a, const Vec& b, const Vec& c) {
  return Vec{__ffma2_rn(a.lo, b.lo, c.lo), __ffma2_rn(a.hi, b.hi, c.hi)};
}

// d Swish(u) / du = p (1 + u (1 - p)), p = sigmoid(u).
__device__ __forceinline__ float2 slope(float2 u) {
  const float2 e = __fmul2_rn(u, splat(-1.4426950408889634f));
  const float2 d = __fadd2_rn(make_float2(ex2(e.x), ex2(e.y)), splat(1.f));
  const float2 p = make_float2(rcp(d.x), rcp(d.y));
  const float2 q = __ffma2_rn(p, splat(-1.f), splat(1.f));
  return __fmul2_rn(p, __ffma2_rn(u, q, splat(1.f)));
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
__global__ void __launch_bounds__(kWarps * 32, sizeof(T) == 2 ? 2 : 1)
    conv_swish_backward_kernel(const ConvBackwardArgs a, int run, float* part) {
  constexpr int H = W - 1;
  constexpr int ROW = kCols * (int)sizeof(T), CH = ROW / 16, ROWS = 32 * 16 / ROW;
  constexpr int TILE = kGroup * ROW;  // one tensor's group
  static_assert(ROWS >= 1 && kGroup % ROWS == 0, "rows of a copy");
  extern __shared__ __align__(16) unsigned char s_raw[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cb = blockIdx.x * kCols, c0 = cb + lane * kVec;
  const bool in = c0 < a.channels;
  const int end = a.cu ? min(max(a.cu[a.N], 0), a.T) : a.T;
  const size_t C = a.channels;
  unsigned char* slots = s_raw + warp * (kSlots * 2 * TILE);
  const uint32_t slots_s = (uint32_t)__cvta_generic_to_shared(slots);

  Vec w[W], dw[W];
#pragma unroll
  for (int i = 0; i < W; ++i) {
    float f[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) f[e] = in ? a.w[(size_t)(c0 + e) * W + i] : 0.f;
    w[i] = Vec{make_float2(f[0], f[1]), make_float2(f[2], f[3])};
    dw[i] = zero();
  }
  for (int64_t tile = blockIdx.y; tile * kWarps * run < end; tile += gridDim.y) {
    const int64_t r0 = (tile * kWarps + warp) * run;
    if (r0 >= end) continue;
    const int t0 = (int)r0, t1 = min(t0 + run, end), t2 = min(t1 + H, end);
    const int groups = (t2 - t0 + kGroup - 1) / kGroup;
    // lane `lane` brings chunk lane % CH of row lane / CH of each ROWS rows
    const int ch = lane % CH, row = lane / CH;
    const bool chunk_in = cb + ch * (16 / (int)sizeof(T)) < a.channels;
    auto request = [&](int g) {
      if (g < groups) {
        const uint32_t to = slots_s + (g % kSlots) * (2 * TILE) + row * ROW + ch * 16;
#pragma unroll
        for (int r = 0; r < kGroup; r += ROWS) {
          const int t = t0 + g * kGroup + r + row;
          const bool live = chunk_in && t < t2;
          const size_t at = live ? ((size_t)t * C + cb) * sizeof(T) + ch * 16 : 0;
          copy16(to + r * ROW, (const char*)a.x + at, live);
          copy16(to + r * ROW + TILE, (const char*)a.dy + at, live);
        }
      }
      copy_commit();
    };
    __syncwarp();  // the last tile's slots are read
#pragma unroll
    for (int g = 0; g < kSlots - 1; ++g) request(g);

    int start, next;
    sequence_at(a, end, t0, start, next);
    // win[j] = x of token t - H + j; sum[j] = dx of token t - H + j so far
    Vec win[W], sum[W];
#pragma unroll
    for (int j = 0; j < H; ++j) {
      win[j] = sum[j] = zero();
      const int s = t0 - H + j;
      if (in && s >= start) win[j] = ld4((const T*)a.x + s * C + c0);
    }
    int emit = t0;  // dx of tokens below this one is written or belongs to another run
    for (int g = 0; g < groups; ++g) {
      __syncwarp();
      request(g + kSlots - 1);
      copy_wait<kSlots - 1>();
      __syncwarp();
      const int tg = t0 + g * kGroup;
      const T* sx = (const T*)(slots + (g % kSlots) * (2 * TILE)) + lane * kVec;
      const T* sd = sx + TILE / (int)sizeof(T);
      T* dx = (T*)a.dx + (size_t)tg * C + c0;
      // one token of the group; kWhole: no boundary in the group, all of it in the run
      auto token = [&](int j, bool whole) {
        const int t = tg + j;
        win[H] = ld4(sx + j * kCols);
        const Vec dyv = ld4(sd + j * kCols);
        Vec u = mul(w[H], win[H]);
#pragma unroll
        for (int i = 0; i < H; ++i) u = fma(w[i], win[i], u);
        const Vec du = mul(dyv, Vec{slope(u.lo), slope(u.hi)});
#pragma unroll
        for (int i = 0; i < H; ++i) sum[i] = fma(w[i], du, sum[i]);
        sum[H] = mul(w[H], du);
        if (whole || t < t1)
#pragma unroll
          for (int i = 0; i < W; ++i) dw[i] = fma(du, win[i], dw[i]);
        if (in && t - H >= emit && (whole || t - H < t1))
          st4(dx + ((int64_t)j - H) * (int64_t)C, sum[0]);
#pragma unroll
        for (int i = 0; i < H; ++i) {
          win[i] = win[i + 1];
          sum[i] = sum[i + 1];
        }
      };
      if (tg + kGroup <= t1 && next >= tg + kGroup) {
#pragma unroll
        for (int j = 0; j < kGroup; ++j) token(j, true);
      } else {
#pragma unroll 1
        for (int j = 0; j < kGroup && tg + j < t2; ++j) {
          const int t = tg + j;
          if (t == next) {
            // a sequence starts: the last one's unfinished sums are complete, nothing is carried
#pragma unroll
            for (int i = 0; i < H; ++i) {
              const int s = t - H + i;
              if (in && s >= emit && s < t1) st4((T*)a.dx + s * C + c0, sum[i]);
              win[i] = sum[i] = zero();
            }
            emit = t;
            sequence_at(a, end, t, start, next);
          }
          token(j, false);
        }
      }
    }
    // the tokens whose later rows lie past the end
#pragma unroll
    for (int j = 0; j < H; ++j) {
      const int s = t2 - H + j;
      if (in && s >= emit && s < t1) st4((T*)a.dx + s * C + c0, sum[j]);
    }
    copy_wait<0>();
  }
  // dw over the warps, in order; the slots are free
  __syncthreads();
  float* s_dw = (float*)s_raw;  // [kWarps][W][kCols]
#pragma unroll
  for (int i = 0; i < W; ++i)
    st4(s_dw + (warp * W + i) * kCols + lane * kVec, dw[i]);
  __syncthreads();
  for (int k = threadIdx.x; k < W * kCols; k += kWarps * 32) {
    const int i = k / kCols, c = cb + k % kCols;
    float v = 0.f;
#pragma unroll
    for (int r = 0; r < kWarps; ++r) v += s_dw[r * W * kCols + k];
    if (c < a.channels) part[((size_t)blockIdx.y * C + c) * W + i] = v;
  }
}

// out[i] = sum over r of part[r][i]: 32 numbers a block, 8 threads a number.
__global__ void __launch_bounds__(256)
    sum_splits_kernel(const float* part, int splits, size_t count, float* out) {
  __shared__ float s_sum[8][32];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const size_t i = (size_t)blockIdx.x * 32 + x;
  float s = 0.f;
  if (i < count) {
#pragma unroll 4
    for (int r = y; r < splits; r += 8) s += part[r * count + i];
  }
  s_sum[y][x] = s;
  __syncthreads();
  if (y == 0 && i < count) {
#pragma unroll
    for (int r = 1; r < 8; ++r) s += s_sum[r][x];
    out[i] = s;
  }
}

// Tokens of a run and blocks along the tokens: the longest run (fewest tokens
// computed twice, fewest weight sums) that gives `want` blocks, else the shortest.
void split(int T, int channels, int want, int& run, int& splits) {
  const int64_t cols = (channels + kCols - 1) / kCols;
  run = 128;
  int64_t tiles;
  for (;; run /= 2) {
    tiles = ((int64_t)T + kWarps * run - 1) / (kWarps * run);
    if (run == kGroup || tiles * cols >= want) break;
  }
  splits = (int)(tiles < 1 ? 1 : tiles > kMaxSplits ? kMaxSplits : tiles);
}
int blocks_wanted(bool bf16) { return bf16 ? 240 : 120; }

template <typename T, int W>
cudaError_t launch_w(const ConvBackwardArgs& a) {
  int run, splits;
  split(a.T, a.channels, blocks_wanted(a.bf16), run, splits);
  constexpr int smem = kWarps * kSlots * 2 * kGroup * kCols * (int)sizeof(T);
  static_assert(smem >= kWarps * W * kCols * (int)sizeof(float), "dw fits the slots");
  auto* kernel = conv_swish_backward_kernel<T, W>;
  cudaError_t err =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  const dim3 grid((a.channels + kCols - 1) / kCols, splits);
  float* part = splits > 1 ? (float*)a.ws : a.dw;
  kernel<<<grid, kWarps * 32, smem, a.stream>>>(a, run, part);
  if ((err = cudaGetLastError()) != cudaSuccess || splits == 1) return err;
  const size_t count = (size_t)a.channels * W;
  sum_splits_kernel<<<(unsigned)((count + 31) / 32), 256, 0, a.stream>>>(part, splits, count,
                                                                         a.dw);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const ConvBackwardArgs& a) {
  switch (a.width) {
    case 1: return launch_w<T, 1>(a);
    case 2: return launch_w<T, 2>(a);
    case 3: return launch_w<T, 3>(a);
    case 4: return launch_w<T, 4>(a);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

size_t conv_backward_workspace_bytes(int T, int channels, int width) {
  int run, splits;
  split(T, channels, blocks_wanted(true), run, splits);  // of the two types' the more
  return (size_t)splits * channels * width * sizeof(float);
}

cudaError_t launch_conv_swish_backward(const ConvBackwardArgs& a) {
  return a.bf16 ? launch_t<__nv_bfloat16>(a) : launch_t<float>(a);
}

}  // namespace kda
