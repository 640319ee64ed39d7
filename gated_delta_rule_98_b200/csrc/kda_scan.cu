// kda_scan.cu -- gated linear recurrence of one number per channel, its
// gradients, and its single-token step.
//
//   z:  a = exp(-5 sigmoid(e^A z)),  h_t = a h_{t-1} + (1 - a) x_t
//   g:  a = exp(g),                  h_t = a h_{t-1} + x_t
//
// Backwards with l_t = dy_t + a_{t+1} l_{t+1}:  dx = (1 - a) l  (z) or l (g),
// dg = a (h_{t-1} - x) l  (z) or a h_{t-1} l (g).
//
// HBM-bound: every input read once, every output written once.  A run of
// tokens maps the state entering it to P h + H (P = prod a, H the run from 0),
// and such maps compose, so tokens are worked on in parallel and only the
// composition is sequential.  Three levels:
//  * a thread owns 2 channels of 8 tokens and runs them twice, once for (P, H)
//    and once, from the state that enters, for h (longer runs compose less often
//    but spill: 16 tokens took 128 registers' worth of decays alone);
//  * a warp owns a span of 32 tokens x 16 channels of bf16 (64 x 8 of fp32: 32
//    bytes of a row) and composes its 4 (8) runs by shuffles;
//  * a block owns those channels of the whole token axis (or one of `segments`
//    parts of it) and its warps take the spans in turn, handing the state from
//    warp to warp through shared memory and a named barrier per warp.  A warp
//    needs the state only after it has (P, H), so the hand-over is short and
//    the loads and the arithmetic of the other warps overlap it.
// Spans are fetched by cp.async into slots private to a warp, so no barrier
// joins the block.  With few channels the token axis is cut into segments: a
// first launch forms each segment's (P, H), reading only what follows the
// segment's last sequence start, and each block composes those before its own.
//
// Sequences are packed along the tokens: a start cuts the composition (P is
// then negative, and what lies before the cut is not multiplied by 0 but left
// out, so that an infinity or NaN stays in its sequence).
//
// The gradient walks the spans backwards; h_{t-1} is recomputed from the state
// that the forward saved at every span, in 32 bits, instead of being read back
// as rounded y (2 bytes an element less to read, and no second rounding).
//
// Measured: 65536 x 2048 bf16 forward 200 us (4.0 TB/s), gradient 343 us (3.9);
// 32768 x 4096 forward 201 us, gradient 340 us (3.9); 16384 x 2048 fp32 88 us (4.6)
// and 156 us (4.3).  Bound by the latency and issue of the gates' arithmetic (65%
// of the issue slots), not by the hand-over: without it the times are the same.
#include <type_traits>

#include "../../include/kda.h"
#include "kda_common.cuh"
#include "kda_layer.h"

namespace kda {

namespace {

constexpr int kSaved = KDA_SCAN_INTERVAL;  // tokens between saved states
// Warps of a block that has an SM to itself, and of one of two that share an SM: at
// most 15 (a named barrier each, 0 is __syncthreads), and what the registers allow:
// 128 a thread in the forward (96 are slower, 203 -> 293 us at 65536 x 2048); in the
// gradient 168 alone (65536 x 2048: 340 us, with 128: 361) and 128 in pairs (32768 x
// 4096: 336 us, with 168 and 6 warps 356).
constexpr int kAlone = 15, kPaired = 8;
constexpr int kAloneBack = 12, kPairedBack = 8;
constexpr int kSlots = 3;     // spans of a warp in flight or in use
constexpr int kMaxSegments = 64;
constexpr int kBrought = 256;  // states brought to the first cache: 16 KB
constexpr int kRoom = 222 * 1024;  // dynamic shared memory of a block that has an SM to itself
constexpr float kLog2e = 1.4426950408889634f;

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
__device__ __forceinline__ float2 splat(float x) { return make_float2(x, x); }

__device__ __forceinline__ float2 lds2(const __nv_bfloat16* p) {
  const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ float2 lds2(const float* p) {
  return *reinterpret_cast<const float2*>(p);
}
__device__ __forceinline__ void stg2(__nv_bfloat16* p, float2 v) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
}
__device__ __forceinline__ void stg2(float* p, float2 v) { *reinterpret_cast<float2*>(p) = v; }

// a = 2^t and 1 - a, t = g log2(e) <= 0.  Near 1 the difference loses digits, so
// above 2^-0.2 = 0.87 it is t times a polynomial: (1 - 2^t) / t interpolated at
// the Chebyshev nodes of [-0.2005, 0] (5e-8 of it at most); below, the rounding of
// a is at most 15 units of 2^-24 of 1 - a.
constexpr float kNear = -0.2f;
__device__ __forceinline__ float2 near_one(float2 t) {
  float2 q = splat(-0.00910008978f);
  q = __ffma2_rn(q, t, splat(-0.0554398298f));
  q = __ffma2_rn(q, t, splat(-0.240223944f));
  q = __ffma2_rn(q, t, splat(-0.693147182f));
  return __fmul2_rn(q, t);
}
__device__ __forceinline__ void decay(float2 t, float2& a, float2& m) {
  a = make_float2(ex2(t.x), ex2(t.y));
  const float2 q = near_one(t);
  // single additions here and in the sigmoid take their constant from the
  // instruction, a packed one from two registers, which are scarce
  m.x = t.x > kNear ? q.x : 1.f - a.x;
  m.y = t.y > kNear ? q.y : 1.f - a.y;
}

// -e^A log2(e) of two channels, rounded once.  sigmoid(u) far below 0 is e^u and takes
// |u| times the relative error of u = e^A z, which is that of this rounding and of the
// product's: 2 |u| units of 2^-24 together, as much as a step of z to its neighbours
// makes in float32 (4.5 |u| with e^A in 32 bits).
__device__ __forceinline__ float2 gate_scale(float2 A) {
  return make_float2((float)(-1.4426950408889634 * exp((double)A.x)),
                     (float)(-1.4426950408889634 * exp((double)A.y)));
}

// The library's gate on two channels: k = -e^A log2(e).
struct GateZ {
  float2 t, a, m, p;  // log2 of the decay, decay, 1 - decay, s (1 - s)
};
template <bool kSlope>
__device__ __forceinline__ GateZ gate_z(float2 z, float2 k) {
  const float2 u = __fmul2_rn(z, k);
  const float2 e = make_float2(ex2(u.x), ex2(u.y));  // e^{-e^A z}
  const float2 d = make_float2(e.x + 1.f, e.y + 1.f);
  const float2 s = make_float2(rcp(d.x), rcp(d.y));
  GateZ g;
  g.t = __fmul2_rn(s, splat(kGateMin * kLog2e));
  decay(g.t, g.a, g.m);
  if (kSlope) {
    // 1 - s = e s: the difference would lose the digits of s near 1.  e = inf gives s = 0.
    g.p.x = s.x == 0.f ? 0.f : s.x * (s.x * e.x);
    g.p.y = s.y == 0.f ? 0.f : s.y * (s.y * e.y);
  }
  return g;
}

// Composition of affine maps h -> P h + H; P < 0: a sequence starts inside, H is the state.
struct Map {
  float2 P, H;
};
__device__ __forceinline__ float then_p(float first, float second) {
  return second < 0.f ? second : first < 0.f ? first : first * second;
}
__device__ __forceinline__ float apply1(float P, float H, float h) {
  return P < 0.f ? H : fmaf(P, h, H);
}
__device__ __forceinline__ float2 apply(const Map& m, float2 h) {
  return make_float2(apply1(m.P.x, m.H.x, h.x), apply1(m.P.y, m.H.y, h.y));
}
__device__ __forceinline__ Map then(const Map& first, const Map& second) {
  Map r;
  r.H = apply(second, first.H);
  r.P = make_float2(then_p(first.P.x, second.P.x), then_p(first.P.y, second.P.y));
  return r;
}
// Without a sequence start in either.
__device__ __forceinline__ Map then_plain(const Map& first, const Map& second) {
  return Map{__fmul2_rn(first.P, second.P), __ffma2_rn(second.P, first.H, second.H)};
}
template <bool kUp>
__device__ __forceinline__ Map shuffle(const Map& m, int lanes) {
  auto s = [&](float v) {
    return kUp ? __shfl_up_sync(0xffffffffu, v, lanes) : __shfl_down_sync(0xffffffffu, v, lanes);
  };
  Map r;
  r.P = make_float2(s(m.P.x), s(m.P.y));
  r.H = make_float2(s(m.H.x), s(m.H.y));
  return r;
}

// Composes the maps of a span's GR runs (LC lanes each), in rising order of the
// runs or falling: `run` becomes the map up to and with the lane's run, the
// result is the map up to it.  kPlain: no sequence starts inside.
template <int LC, bool kUp, bool kPlain>
__device__ __forceinline__ Map compose(Map& run, int lane) {
  const int at = kUp ? lane : 31 - lane;
#pragma unroll
  for (int o = LC; o < 32; o <<= 1) {
    const Map m = shuffle<kUp>(run, o);
    if (at >= o) run = kPlain ? then_plain(m, run) : then(m, run);
  }
  const Map before = shuffle<kUp>(run, LC);
  return at < LC ? Map{splat(1.f), splat(0.f)} : before;
}

// Slow channels.  A decay near 1 is rounded to 2^-24 of itself however small 1 - a
// is, and a state that lasts collects those errors: with products of the rounded
// decays alone, h = x = 1 drifts by 0.45% over 65536 tokens.  Below 2^kNear = 0.87 a
// product holds enough digits, and its errors are forgotten with the state; above it
//  * bf16 takes a run's product as 1 - q, with q from the state's own recursion for
//    x = 1, q' = a q + (1 - a), or, with g given, from the sum of the logarithms: one
//    rounding a run instead of one a token, a drift of 0.025% (65536 x 2048 forward
//    194 -> 200 us, gradient 340 -> 343);
//  * fp32 takes the state over the whole span as h + (H - q h), q from the sum of the
//    logarithms, rounded once to h's digits: a drift of 0.002%.  It costs 1% there
//    (16384 x 2048: 87 -> 88 us, 155 -> 156), where the loads leave time; in bf16 it
//    took 250 us at 65536 x 2048, and the outputs hold 8 bits.
// A segment's map has its product from the sum of the logarithms too.

// Sum over a span of its runs' sums of log2 a (LC lanes each).
template <int LC>
__device__ __forceinline__ float2 span_sum(float2 S) {
#pragma unroll
  for (int o = LC; o < 32; o <<= 1) {
    S.x += __shfl_xor_sync(0xffffffffu, S.x, o);
    S.y += __shfl_xor_sync(0xffffffffu, S.y, o);
  }
  return S;
}
// 1 - 2^S, or 2 where the product is to be used.
__device__ __forceinline__ float2 complement(float2 S) {
  const float2 q = near_one(S);
  return make_float2(S.x > kNear && S.x <= 0.f ? q.x : 2.f,
                     S.y > kNear && S.y <= 0.f ? q.y : 2.f);
}
// A run's product: 1 - q where that is near 1.
__device__ __forceinline__ float2 product(float2 P, float2 q) {
  return make_float2(q.x < 0.13f ? 1.f - q.x : P.x, q.y < 0.13f ? 1.f - q.y : P.y);
}
// `by_p` is P h + H; an infinite h takes it (here it would be inf - inf).
__device__ __forceinline__ float apply_slow1(float q, float H, float h, float by_p) {
  const float by_q = h + fmaf(-q, h, H);
  return q < 1.f && by_q == by_q ? by_q : by_p;
}
__device__ __forceinline__ float2 apply_slow(float2 q, float2 H, float2 h, float2 by_p) {
  return make_float2(apply_slow1(q.x, H.x, h.x, by_p.x), apply_slow1(q.y, H.y, h.y, by_p.y));
}

// A segment's map: rows 2 s and 2 s + 1 of `maps` hold H and log2 P, or kStarted in
// the place of log2 P where a sequence starts (backwards: ends) inside.
constexpr float kStarted = 3.0e38f;
__device__ __forceinline__ float2 apply_map(const float* maps, int s, int C, int c, bool in,
                                            float2 h) {
  if (!in) return h;
  const float2* p = reinterpret_cast<const float2*>(maps + (size_t)2 * s * C + c);
  const float2 H = p[0], S = p[C / 2];
  if (S.x == kStarted) return H;  // a start is one of all channels
  return apply_slow(complement(S), H, h, apply(Map{make_float2(ex2(S.x), ex2(S.y)), H}, h));
}
__device__ __forceinline__ void put_start(float* maps, int C, int c, bool in) {
  if (!in) return;
  float2* p = reinterpret_cast<float2*>(maps + (size_t)2 * blockIdx.y * C + c);
  p[0] = splat(0.f);
  p[C / 2] = splat(kStarted);
}
// log2 P of a block's segment, added over its runs and warps in a fixed order.
template <int LC>
__device__ __forceinline__ void put_sum(float2 sum, bool started, float2* s_sum, float* maps, int C,
                                        int c, bool in, int lane, int warp, int W) {
  sum = span_sum<LC>(sum);
  if (lane < LC) s_sum[warp * LC + lane] = sum;
  __syncthreads();
  if (warp != 0 || lane >= LC || !in) return;
  for (int w = 1; w < W; ++w) sum = __fadd2_rn(sum, s_sum[w * LC + lane]);
  *reinterpret_cast<float2*>(maps + ((size_t)2 * blockIdx.y + 1) * C + c) =
      started ? splat(kStarted) : sum;
}

// Tile geometry: a span of SPAN tokens, rows of 32 bytes of x, 2 channels a lane.
template <typename T, int SPAN>
struct Geo {
  static constexpr int CB = 32 / (int)sizeof(T);  // channels of a block
  static constexpr int LC = CB / 2;               // lanes along the channels
  static constexpr int GR = 32 / LC;              // runs of a span
  static constexpr int K = SPAN / GR;             // tokens of a run
};
// Bytes of one tensor's span in shared memory: a spare row after each run moves
// the runs to different banks, so that a warp's reads do not collide.
template <typename G, typename E>
__host__ __device__ constexpr int tile_bytes() {
  return G::GR * (G::K + 1) * G::CB * (int)sizeof(E);
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
// One tensor's way into a warp's slots: lane `lane` brings 16 bytes of a row, a
// span takes COPIES copies of ROWS rows each.
template <typename G, typename E>
struct Source {
  static constexpr int RB = G::CB * (int)sizeof(E), CH = RB / 16, PER = 16 / (int)sizeof(E);
  static constexpr int SPAN = G::GR * G::K, ROWS = 32 / CH, COPIES = SPAN / ROWS;
  const char* base;
  const char* p;   // this lane's piece of the first copy's row of span 0
  int row, pitch;  // the row in that copy; bytes of a row of the tensor
  uint32_t dst;    // the piece's place in a slot
  bool in;         // the piece is in the tensor
  __device__ Source(const void* src, int C, int c0, int lane) {
    const int ch = lane % CH;
    base = (const char*)src;
    row = lane / CH;
    pitch = C * (int)sizeof(E);
    in = c0 + ch * PER < C;
    p = (const char*)src + (int64_t)row * pitch + (int64_t)(in ? c0 + ch * PER : 0) * sizeof(E);
    dst = (row + row / G::K) * RB + ch * 16;
  }
  // Span j into the tile; zeros outside the tensor and from token `end` on.
  __device__ __forceinline__ void fetch(uint32_t tile, int j, int end) const {
    const char* q = p + (int64_t)j * SPAN * pitch;
    const int left = end - j * SPAN - row;  // rows from this lane's first one to the end
#pragma unroll
    for (int it = 0; it < COPIES; ++it) {
      static_assert(ROWS % G::K == 0 || G::K % ROWS == 0, "spare rows");
      const bool live = in && it * ROWS < left;
      copy16(tile + dst + (it * ROWS + it * ROWS / G::K) * RB,
             live ? q + (int64_t)(it * ROWS) * pitch : base, live);
    }
  }
};

// The state's way from warp to warp: warp w waits for its turn on barrier 1 + w.
__device__ __forceinline__ void turn_wait(int w) {
  asm volatile("bar.sync %0, 64;" ::"r"(1 + w) : "memory");
}
__device__ __forceinline__ void turn_pass(int w) {
  asm volatile("bar.arrive %0, 64;" ::"r"(1 + w) : "memory");
}

// ------------------------------------------------------------- sequences ----

// Sequence bounds: entry k of cu_seqlens, or k * L; `end` is the end of the last sequence.
struct Bounds {
  const int32_t* cu;
  int N, L, end;
  __device__ Bounds(const ScanArgs& a) : cu(a.cu), N(a.N), L(a.L) {
    end = cu ? min(max(cu[N], 0), a.T) : a.T;
  }
  __device__ __forceinline__ int64_t at(int k) const { return cu ? cu[k] : (int64_t)k * L; }
  // First entry in [lo, N] that is >= t (N + 1 if there is none).
  __device__ __forceinline__ int lower(int lo, int64_t t) const {
    if (!cu) return L > 0 ? (int)((t + L - 1) / L) : 0;
    int hi = N + 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (cu[mid] >= t) hi = mid; else lo = mid + 1;
    }
    return lo;
  }
  // The sequence that holds token t, in [0, N - 1] whatever cu holds.
  __device__ __forceinline__ int of(int64_t t) const {
    return min(max(lower(0, t + 1) - 1, 0), N - 1);
  }
  __device__ __forceinline__ int up(int n, int64_t t) const {  // of(t) from a lower n
    while (n < N - 1 && at(n + 1) <= t) ++n;
    return n;
  }
  __device__ __forceinline__ int down(int n, int64_t t) const {  // of(t) from a higher n
    while (n > 0 && at(n) > t) --n;
    return n;
  }
};

// Boundaries (sequence starts, and the end) at tokens [t0, t0 + SPAN]: bit i of
// `bits` is token t0 + i, `last` is token t0 + SPAN.
struct Marks {
  uint64_t bits;
  bool last;
  __device__ __forceinline__ bool any() const { return bits != 0 || last; }
};
// A warp's view of the boundaries of the spans it takes, in rising or falling
// order: no boundary lies between the last span and `clear`.
template <bool kRising, int SPAN>
struct Marker {
  int k = 0;
  int clear = kRising ? -1 : 0x7fffffff;
  __device__ __forceinline__ Marks look(const Bounds& b, int t0, int lane) {
    Marks m{0, false};
    const int t1 = t0 + SPAN;
    const bool quiet = kRising ? clear > t1 : clear < t0;
    if (quiet && b.end > t1) return m;
    if (b.end == t1) m.last = true;
    else if (b.end < t1) m.bits |= 1ull << (b.end - t0);
    if (quiet) return m;
    k = b.lower(kRising ? min(k, b.N) : 0, t0);
    if (kRising) clear = k <= b.N ? (int)b.at(k) : 0x7fffffff;  // first boundary from t0 on
    else clear = k <= b.N && b.at(k) == t0 ? t0 : k > 0 ? (int)b.at(k - 1) : -1;  // last up to t0
    uint32_t lo = 0, hi = 0, at_end = 0;
    for (int i = k; i <= b.N; i += 32) {
      const int64_t v = i + lane <= b.N ? b.at(i + lane) - t0 : INT64_MAX;
      if (v == SPAN) at_end = 1;
      else if (v >= 0 && v < 32) lo |= 1u << v;
      else if (v >= 32 && v < SPAN) hi |= 1u << (v - 32);
      // entries do not fall, so a lane beyond the span ends the search
      if (__any_sync(0xffffffffu, v > SPAN)) break;
    }
    lo = __reduce_or_sync(0xffffffffu, lo);
    hi = __reduce_or_sync(0xffffffffu, hi);
    m.bits |= (uint64_t)hi << 32 | lo;
    m.last |= __reduce_or_sync(0xffffffffu, at_end) != 0;
    return m;
  }
};

__device__ __forceinline__ float2 row2(const float* p, int n, int C, int c, bool in) {
  if (!p || !in) return splat(0.f);
  return *reinterpret_cast<const float2*>(p + (size_t)n * C + c);
}
__device__ __forceinline__ void put2(float* p, int n, int C, int c, bool in, float2 v) {
  if (p && in) *reinterpret_cast<float2*>(p + (size_t)n * C + c) = v;
}

// Brings the block's channels of the sequences' states near: a span with a sequence
// start waits for them, and all spans behind it wait for that one.
__device__ __forceinline__ void bring(const Bounds& b, const float* p, int C, int c0) {
  if (!p) return;
  for (int n = threadIdx.x; n < min(b.N, kBrought); n += blockDim.x)
    asm volatile("prefetch.global.L1 [%0];" ::"l"(p + (size_t)n * C + c0));
}

// What empty sequences hand through (`from`, or zeros) to `to`, for the block's channels.
__device__ __forceinline__ void pass_empty(const Bounds& b, const float* from, float* to, int C,
                                           int c0, int CB) {
  if (!to || (!b.cu && b.L > 0)) return;
  for (int n = threadIdx.x; n < b.N; n += blockDim.x)
    if (!b.cu || b.cu[n + 1] <= b.cu[n])
      for (int c = c0; c < min(c0 + CB, C); c += 2)
        put2(to, n, C, c, true, row2(from, n, C, c, true));
}

// ---------------------------------------------------------------- forward ----

// kMaps: form the segment's map (P, H) in `maps` instead of y; else compose
// the maps of the segments before this one.
template <typename T, bool kZ, bool kMaps, int SPAN>
__global__ void __launch_bounds__(kAlone * 32, 1)
    scan_kernel(const ScanArgs a, int seg_spans, float* maps) {
  using G = Geo<T, SPAN>;
  using E = typename std::conditional<kZ, T, float>::type;
  constexpr int XB = tile_bytes<G, T>(), STAGE = XB + tile_bytes<G, E>(), D = kSlots;
  constexpr int K = G::K, LC = G::LC, GR = G::GR, CB = G::CB;
  // the correction of slow channels, over the span or over each run; a map sums the
  // logarithms in any case
  constexpr bool kExact = sizeof(T) == 4, kRun = !kExact, kByState = kRun && kZ && !kMaps;
  extern __shared__ __align__(16) unsigned char s_raw[];
  __shared__ float2 s_h[2][LC], s_sum[kMaps ? kAlone : 1][LC];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5;
  const int l = lane % LC, grp = lane / LC;
  const int C = a.C, c0 = blockIdx.x * CB, c = c0 + 2 * l;
  const bool in = c < C;
  const Bounds b(a);
  const int spans = (int)(((int64_t)b.end + SPAN - 1) / SPAN);
  int j0 = blockIdx.y * seg_spans;
  bool started = false;  // a sequence starts in the segment
  const int j1 = min(j0 + seg_spans, spans);
  if (kMaps) {
    // the map that later segments need: nothing before the last sequence start matters
    if (j0 >= j1 || j1 == spans) return;
    const int64_t te = (int64_t)j1 * SPAN;
    const int k = b.lower(0, te);
    if (k <= b.N && b.at(k) == te) {
      if (warp == 0 && grp == 0) put_start(maps, C, c, in);
      return;
    }
    if (k > 0) {
      const int64_t start = max(b.at(k - 1), (int64_t)0);
      started = start >= (int64_t)j0 * SPAN;
      j0 = max(j0, (int)(start / SPAN));
    }
  } else if (blockIdx.y == 0) {
    pass_empty(b, a.h0, a.h_final, C, c0, CB);
  }
  const uint32_t tiles =
      (uint32_t)__cvta_generic_to_shared(s_raw) + warp * (D * STAGE);
  const unsigned char* tiles_p = s_raw + warp * (D * STAGE);
  bring(b, a.h0, C, c0);
  const Source<G, T> X(a.x, C, c0, lane);
  const Source<G, E> Z(kZ ? a.z : (const void*)a.g, C, c0, lane);
  auto request = [&](int j, int slot) {
    if (j < j1) {
      X.fetch(tiles + slot * STAGE, j, b.end);
      Z.fetch(tiles + slot * STAGE + XB, j, b.end);
    }
    copy_commit();
  };
#pragma unroll
  for (int i = 0; i < D - 1; ++i) request(j0 + warp + i * W, i);
  float2 k = splat(0.f);
  if (kZ && in && b.end > 0) k = gate_scale(*reinterpret_cast<const float2*>(a.A + c));
  Marker<true, SPAN> marker;
  float2 sum = splat(0.f);  // of log2 a over the lane's tokens
  int slot = 0;
  for (int j = j0 + warp; j < j1; j += W) {
    __syncwarp();
    request(j + (D - 1) * W, slot == 0 ? D - 1 : slot - 1);
    copy_wait<D - 1>();
    __syncwarp();
    const int t0 = j * SPAN, tk = t0 + grp * K;
    const T* sx = (const T*)(tiles_p + slot * STAGE) + grp * (K + 1) * CB + 2 * l;
    const E* sz = (const E*)(tiles_p + slot * STAGE + XB) + grp * (K + 1) * CB + 2 * l;
    slot = slot == D - 1 ? 0 : slot + 1;
    const Marks marks = marker.look(b, t0, lane);
    const bool cut = marks.any();
    const uint32_t starts = (uint32_t)(marks.bits >> (grp * K)) & ((1u << K) - 1);

    float2 A[K], B[K], S = splat(0.f), q = splat(0.f);
    Map run{splat(1.f), splat(0.f)};
    if (!kZ) {
#pragma unroll
      for (int i = 0; i < K; ++i) S = __fadd2_rn(S, lds2(sz + i * CB));
      S = __fmul2_rn(S, splat(kLog2e));
    }
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const float2 x = lds2(sx + i * CB), z = lds2(sz + i * CB);
      if (kZ) {
        const GateZ g = gate_z<false>(z, k);
        A[i] = g.a;
        B[i] = __fmul2_rn(g.m, x);
        if (kByState) q = __ffma2_rn(g.a, q, g.m);
        else S = __fadd2_rn(S, g.t);
      } else {
        A[i] = make_float2(ex2(z.x * kLog2e), ex2(z.y * kLog2e));
        B[i] = x;
      }
      // with no start inside; here, and not behind a branch, so that this chain
      // runs between the gates' independent instructions
      run.H = __ffma2_rn(A[i], run.H, B[i]);
      run.P = __fmul2_rn(run.P, A[i]);
    }
    const bool slow =
        kExact && !cut && __any_sync(0xffffffffu, in && (S.x > kNear || S.y > kNear));
    if (kRun) run.P = product(run.P, kByState ? q : complement(S));
    if (kMaps) sum = __fadd2_rn(sum, S);
    if (slow) q = complement(span_sum<LC>(S));
    if (cut) {
      run = Map{splat(1.f), splat(0.f)};
      int n = starts ? b.of(tk) : 0;
#pragma unroll
      for (int i = 0; i < K; ++i) {
        if (starts >> i & 1) {
          // B takes the state after the token: the second run must not read h0 again,
          // which may be h_final and by then hold a sequence's end
          n = b.up(n, tk + i);
          B[i] = __ffma2_rn(A[i], row2(a.h0, n, C, c, in && tk + i < b.end), B[i]);
          run.H = B[i];
          run.P = splat(-1.f);
        } else {
          run.H = __ffma2_rn(A[i], run.H, B[i]);
        }
        run.P = make_float2(run.P.x < 0.f ? -1.f : run.P.x * A[i].x,
                            run.P.y < 0.f ? -1.f : run.P.y * A[i].y);
      }
    }
    const Map before = cut ? compose<LC, true, false>(run, lane) : compose<LC, true, true>(run, lane);

    // the state before this span
    float2 h_in = splat(0.f);
    if (j > j0) {
      if (W > 1) turn_wait(warp);
      h_in = s_h[j & 1][l];
    } else if (!kMaps) {
      for (int s = 0; s < (int)blockIdx.y; ++s) h_in = apply_map(maps, s, C, c, in, h_in);
    }
    // slot j + 1 was last read by the warp of span j - 1, before it passed the turn
    float2 h_out = apply(run, h_in);
    if (slow) h_out = apply_slow(q, run.H, h_in, h_out);
    if (grp == GR - 1) {
      s_h[(j + 1) & 1][l] = h_out;
      if (kMaps && j == j1 - 1) put2(maps, 2 * blockIdx.y, C, c, in, h_out);
    }
    __syncwarp();
    if (j + 1 < j1 && W > 1) turn_pass(warp + 1 == W ? 0 : warp + 1);
    if (kMaps) continue;

    float2 h = apply(before, h_in);
    if (grp * K % kSaved == 0 && tk < b.end) put2(a.states, tk / kSaved, C, c, in, h);
    char* y = (char*)a.y + ((int64_t)tk * C + c) * (int64_t)sizeof(T);
    const int pitch = C * (int)sizeof(T);
    if (!cut) {
#pragma unroll
      for (int i = 0; i < K; ++i) {
        h = __ffma2_rn(A[i], h, B[i]);
        if (in) stg2((T*)(y + (int64_t)i * pitch), h);
      }
    } else {
      const uint32_t ends = (uint32_t)((marks.bits >> 1 | (uint64_t)marks.last << (SPAN - 1)) >> (grp * K)) &
                            ((1u << K) - 1);
      int n = (starts | ends) ? b.of(tk) : 0;
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const bool live = in && tk + i < b.end;
        if (starts >> i & 1) {
          n = b.up(n, tk + i);
          h = B[i];
        } else {
          h = __ffma2_rn(A[i], h, B[i]);
        }
        if (live) {
          stg2((T*)(y + (int64_t)i * pitch), h);
          if (ends >> i & 1) put2(a.h_final, n, C, c, true, h);
        }
      }
    }
  }
  copy_wait<0>();
  if (kMaps) put_sum<LC>(sum, started, &s_sum[0][0], maps, C, c, in, lane, warp, W);
}

// --------------------------------------------------------------- backward ----

// kMaps: form the map of the gradient through the segment, from its last token
// to its first, in `maps`; else compose the maps of the segments after this
// one.  dA of the segment's tokens goes to row blockIdx.y of dA_part.
template <typename T, bool kZ, bool kMaps, int SPAN, bool kPair>
__global__ void __launch_bounds__((kPair ? kPairedBack : kAloneBack) * 32, kPair ? 2 : 1)
    scan_backward_kernel(const ScanArgs a, int seg_spans, float* maps, float* dA_part) {
  using G = Geo<T, SPAN>;
  using E = typename std::conditional<kZ, T, float>::type;
  constexpr int XB = tile_bytes<G, T>(), ZB = tile_bytes<G, E>(), STAGE = 2 * XB + ZB, D = kSlots;
  constexpr int K = G::K, LC = G::LC, CB = G::CB;
  // the correction of slow channels, over the span or over each run; a map sums the
  // logarithms in any case
  constexpr bool kExact = sizeof(T) == 4, kRun = !kExact, kByState = kRun && kZ && !kMaps;
  extern __shared__ __align__(16) unsigned char s_raw[];
  __shared__ float2 s_h[2][LC], s_dA[kPair ? kPairedBack : kAloneBack][LC];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5;
  const int l = lane % LC, grp = lane / LC;
  const int C = a.C, c0 = blockIdx.x * CB, c = c0 + 2 * l;
  const bool in = c < C;
  const Bounds b(a);
  const int spans = (int)(((int64_t)b.end + SPAN - 1) / SPAN);
  const int j0 = blockIdx.y * seg_spans;
  int j1 = min(j0 + seg_spans, spans);
  bool ended = false;  // a sequence ends in the segment
  if (kMaps) {
    // the map that earlier segments need: nothing after the first sequence end matters
    if (j0 >= j1 || j0 == 0) return;
    const int64_t ts = (int64_t)j0 * SPAN;
    const int k = b.lower(0, ts);
    if (k <= b.N && b.at(k) == ts) {
      if (warp == 0 && grp == 0) put_start(maps, C, c, in);
      return;
    }
    if (k <= b.N) {
      const int64_t e = min(b.at(k), (int64_t)b.end);
      ended = e <= (int64_t)j1 * SPAN;
      j1 = min(j1, (int)((e + SPAN - 1) / SPAN));
    }
  } else if (blockIdx.y == 0) {
    pass_empty(b, a.dh_final, a.dh0, C, c0, CB);
  }
  const uint32_t tiles = (uint32_t)__cvta_generic_to_shared(s_raw) + warp * (D * STAGE);
  const unsigned char* tiles_p = s_raw + warp * (D * STAGE);
  bring(b, a.h0, C, c0);
  bring(b, a.dh_final, C, c0);
  const Source<G, T> X(a.x, C, c0, lane), DY(a.dy, C, c0, lane);
  const Source<G, E> Z(kZ ? a.z : (const void*)a.g, C, c0, lane);
  auto request = [&](int j, int slot) {
    if (j >= j0) {
      if (!kMaps) X.fetch(tiles + slot * STAGE, j, b.end);
      DY.fetch(tiles + slot * STAGE + XB, j, b.end);
      Z.fetch(tiles + slot * STAGE + 2 * XB, j, b.end);
    }
    copy_commit();
  };
#pragma unroll
  for (int i = 0; i < D - 1; ++i) request(j1 - 1 - warp - i * W, i);
  float2 k = splat(0.f);
  if (kZ && in && b.end > 0) k = gate_scale(*reinterpret_cast<const float2*>(a.A + c));
  // -5 e^A, the constant factors of dz
  const float2 kz = __fmul2_rn(k, splat(-kGateMin / kLog2e));
  float2 dA = splat(0.f);
  Marker<false, SPAN> marker;
  float2 sum = splat(0.f);  // of log2 a over the lane's tokens
  int slot = 0;
  for (int j = j1 - 1 - warp; j >= j0; j -= W) {
    __syncwarp();
    request(j - (D - 1) * W, slot == 0 ? D - 1 : slot - 1);
    const float2 state = kMaps ? splat(0.f) : row2(a.states, j * (SPAN / kSaved), C, c, in);
    copy_wait<D - 1>();
    __syncwarp();
    const int t0 = j * SPAN, tk = t0 + grp * K;
    const unsigned char* tile = tiles_p + slot * STAGE;
    const int off = grp * (K + 1) * CB + 2 * l;
    const T* sx = (const T*)tile + off;
    const T* sd = (const T*)(tile + XB) + off;
    const E* sz = (const E*)(tile + 2 * XB) + off;
    slot = slot == D - 1 ? 0 : slot + 1;
    const Marks marks = marker.look(b, t0, lane);
    const bool cut = marks.any();
    const uint32_t starts = (uint32_t)(marks.bits >> (grp * K)) & ((1u << K) - 1);
    const uint32_t ends =
        (uint32_t)((marks.bits >> 1 | (uint64_t)marks.last << (SPAN - 1)) >> (grp * K)) & ((1u << K) - 1);

    // fwd: the state through the run; bwd: the gradient that leaves its first token,
    // for the gradient entering behind its last one.  The gate's decay, input scale
    // and slope stay in registers for the second walk (8 tokens a run leave room)
    float2 A[K], H[K], M[kZ ? K : 1], S[kZ ? K : 1];
    Map fwd{splat(1.f), splat(0.f)}, bwd{splat(1.f), splat(0.f)};
    float2 logs = splat(0.f), q = splat(0.f);
    if (!kZ) {
#pragma unroll
      for (int i = 0; i < K; ++i) logs = __fadd2_rn(logs, lds2(sz + i * CB));
      logs = __fmul2_rn(logs, splat(kLog2e));
    }
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const float2 z = lds2(sz + i * CB);
      if (kZ) {
        const GateZ g = gate_z<!kMaps>(z, k);
        A[i] = g.a;
        if (kByState) q = __ffma2_rn(g.a, q, g.m);
        else logs = __fadd2_rn(logs, g.t);
        if (!kMaps) {
          M[i] = g.m;
          S[i] = g.p;
          H[i] = __fmul2_rn(g.m, lds2(sx + i * CB));
        }
      } else {
        A[i] = make_float2(ex2(z.x * kLog2e), ex2(z.y * kLog2e));
        if (!kMaps) H[i] = lds2(sx + i * CB);
      }
      // with no start inside, as in the forward
      if (!kMaps) fwd.H = __ffma2_rn(A[i], fwd.H, H[i]);
      bwd.P = __fmul2_rn(bwd.P, A[i]);
      bwd.H = __ffma2_rn(bwd.P, lds2(sd + i * CB), bwd.H);
    }
    fwd.P = bwd.P;
    const bool slow =
        kExact && !cut && __any_sync(0xffffffffu, in && (logs.x > kNear || logs.y > kNear));
    if (kRun) bwd.P = product(bwd.P, kByState ? q : complement(logs));
    if (kMaps) sum = __fadd2_rn(sum, logs);
    if (slow) q = complement(span_sum<LC>(logs));
    int n_first = 0;
    if (cut) {
      fwd = bwd = Map{splat(1.f), splat(0.f)};
      n_first = (starts | ends) ? b.of(tk) : 0;
      int n = n_first;
      float2 P = splat(1.f);  // product up to the run's first sequence end
      bool open = true;
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const bool live = in && tk + i < b.end;
        if (starts >> i & 1) {
          n = b.up(n, tk + i);
          fwd.H = row2(a.h0, n, C, c, live);
          fwd.P = splat(-1.f);
        }
        if (!kMaps) {
          fwd.H = __ffma2_rn(A[i], fwd.H, H[i]);
          fwd.P = make_float2(fwd.P.x < 0.f ? -1.f : fwd.P.x * A[i].x,
                              fwd.P.y < 0.f ? -1.f : fwd.P.y * A[i].y);
        }
        if (open) {
          P = __fmul2_rn(P, A[i]);
          float2 d = lds2(sd + i * CB);
          if (ends >> i & 1) d = __fadd2_rn(d, row2(a.dh_final, n, C, c, live));
          bwd.H = __ffma2_rn(P, d, bwd.H);
          if (ends >> i & 1) open = false;
        }
      }
      bwd.P = open ? P : splat(-1.f);
    }
    Map before{splat(1.f), splat(0.f)}, after;
    if (cut) {
      if (!kMaps) before = compose<LC, true, false>(fwd, lane);
      after = compose<LC, false, false>(bwd, lane);
    } else {
      if (!kMaps) before = compose<LC, true, true>(fwd, lane);
      after = compose<LC, false, true>(bwd, lane);
    }

    float2 l_in = splat(0.f);
    if (j < j1 - 1) {
      if (W > 1) turn_wait(warp);
      l_in = s_h[j & 1][l];
    } else if (!kMaps) {
      const int last = (spans + seg_spans - 1) / seg_spans - 1;
      for (int s = last; s > (int)blockIdx.y; --s) l_in = apply_map(maps, s, C, c, in, l_in);
    }
    float2 l_out = apply(bwd, l_in);
    if (slow) l_out = apply_slow(q, bwd.H, l_in, l_out);
    if (grp == 0) {
      s_h[(j - 1) & 1][l] = l_out;
      if (kMaps && j == j0) put2(maps, 2 * blockIdx.y, C, c, in, l_out);
    }
    __syncwarp();
    if (j > j0 && W > 1) turn_pass(warp + 1 == W ? 0 : warp + 1);
    if (kMaps) continue;

    // the state before each token, in place of the token's input
    float2 h = apply(before, state), back = apply(after, l_in), dA_span = splat(0.f);
    const int pitch = C * (int)sizeof(T), pitch_g = C * (int)sizeof(E);
    char* dx = (char*)a.dx + ((int64_t)tk * C + c) * (int64_t)sizeof(T);
    char* dg = (char*)(kZ ? a.dz : (void*)a.dg) + ((int64_t)tk * C + c) * (int64_t)sizeof(E);
    auto token = [&](int i, bool live) {
      const float2 lam = __fadd2_rn(lds2(sd + i * CB), back);
      back = __fmul2_rn(A[i], lam);
      if (kZ) {
        const float2 d = __ffma2_rn(lds2(sx + i * CB), splat(-1.f), H[i]);
        const float2 dz = __fmul2_rn(__fmul2_rn(back, d), __fmul2_rn(S[i], kz));
        if (live) {
          stg2((T*)(dx + (int64_t)i * pitch), __fmul2_rn(M[i], lam));
          stg2((E*)(dg + (int64_t)i * pitch_g), dz);
          dA_span = __ffma2_rn(dz, lds2(sz + i * CB), dA_span);
        }
      } else if (live) {
        stg2((T*)(dx + (int64_t)i * pitch), lam);
        stg2((E*)(dg + (int64_t)i * pitch_g), __fmul2_rn(back, H[i]));
      }
    };
    if (!cut) {
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const float2 now = h;
        h = __ffma2_rn(A[i], h, H[i]);
        H[i] = now;
      }
#pragma unroll
      for (int i = K - 1; i >= 0; --i) token(i, in);
    } else {
      int n = n_first;
#pragma unroll
      for (int i = 0; i < K; ++i) {
        if (starts >> i & 1) {
          n = b.up(n, tk + i);
          h = row2(a.h0, n, C, c, in && tk + i < b.end);
        }
        const float2 now = h;
        h = __ffma2_rn(A[i], h, H[i]);
        H[i] = now;
      }
#pragma unroll
      for (int i = K - 1; i >= 0; --i) {
        const bool live = in && tk + i < b.end;
        if (ends >> i & 1) {
          n = b.down(n, tk + i);
          back = row2(a.dh_final, n, C, c, live);
        }
        token(i, live);
        if (starts >> i & 1) {
          n = b.down(n, tk + i);
          put2(a.dh0, n, C, c, live, back);
        }
      }
    }
    dA = __fadd2_rn(dA, dA_span);
  }
  copy_wait<0>();
  if (kMaps) put_sum<LC>(sum, ended, &s_dA[0][0], maps, C, c, in, lane, warp, W);
  if (kZ && !kMaps) {
    // over the runs, then over the warps, in a fixed order
#pragma unroll
    for (int o = LC; o < 32; o <<= 1) {
      dA.x += __shfl_xor_sync(0xffffffffu, dA.x, o);
      dA.y += __shfl_xor_sync(0xffffffffu, dA.y, o);
    }
    if (grp == 0) s_dA[warp][l] = dA;
    __syncthreads();
    if (warp == 0 && grp == 0) {
      float2 v = s_dA[0][l];
      for (int w = 1; w < W; ++w) v = __fadd2_rn(v, s_dA[w][l]);
      put2(dA_part, blockIdx.y, C, c, in, v);
    }
  }
}

__global__ void __launch_bounds__(64)
    sum_rows_kernel(const float* part, int rows, int C, float* out) {
  const int c = blockIdx.x * 64 + threadIdx.x;
  if (c >= C) return;
  float s = 0.f;
  for (int n = 0; n < rows; ++n) s += part[(size_t)n * C + c];
  out[c] = s;
}

// ------------------------------------------------------------------- step ----

template <typename T>
__global__ void __launch_bounds__(256)
    step_kernel(const T* x, const T* z, const float* A, float* h, size_t count, int C, T* y) {
  const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 2;
  if (i >= count) return;
  const int c = (int)(i % C);
  const float2 a = *reinterpret_cast<const float2*>(A + c);
  const float2 xv = lds2(x + i), zv = lds2(z + i), hv = lds2(h + i);
  const GateZ g = gate_z<false>(zv, gate_scale(a));
  // by the complement where a is near 1, as a span of the prefill
  const float2 b = __fmul2_rn(g.m, xv), by_a = __ffma2_rn(g.a, hv, b);
  const float2 by_m = apply_slow(g.m, b, hv, by_a);
  const float2 v = make_float2(g.t.x > kNear ? by_m.x : by_a.x, g.t.y > kNear ? by_m.y : by_a.y);
  stg2(h + i, v);
  stg2(y + i, v);
}

// ----------------------------------------------------------------- launch ----

// Segments of the token axis.  None where the channels alone give a block to half
// the SMs: the maps' launch costs more than the idle SMs, forward and gradient (bf16,
// 32768 x 1408 in one segment 105 and 172 us, in three 130 and 176; x 2048 in one 105
// and 179, in two 170 and 251; x 1024 in one 102 and 167, in four 98 and 132).  Below,
// two blocks per SM (32768 x 512: 51 and 68 us with 288 blocks, 64 and 84 with 128, 62
// and 89 with 416), segments of 512 tokens at least (4096 x 256: 15.3 and 21.1 us, with
// 1024 17.8 and 24.0; 256 gains 0.5 and 0.9 and costs shorter calls a launch).
int segments(int T, int cols) {
  if (cols >= 74) return 1;
  const int s = 296 / cols < T / 512 ? 296 / cols : T / 512;
  return s < 1 ? 1 : s > kMaxSegments ? kMaxSegments : s;
}

struct Plan {
  int cols, segs, seg_spans, warps, smem;
  bool pair;  // two blocks an SM: when there are more blocks than SMs
};
template <typename G>
Plan plan(const ScanArgs& a, int warp_bytes, int alone, int paired, bool one_segment) {
  constexpr int SPAN = G::GR * G::K;
  Plan p;
  p.cols = (a.C + G::CB - 1) / G::CB;
  const int spans = (int)(((int64_t)a.T + SPAN - 1) / SPAN);
  const int segs = one_segment ? 1 : segments(a.T, p.cols);
  p.seg_spans = spans > 0 ? (spans + segs - 1) / segs : 1;
  p.segs = spans > 0 ? (spans + p.seg_spans - 1) / p.seg_spans : 1;
  p.pair = (int64_t)p.cols * p.segs > 148;
  const int room = p.pair ? kRoom / 2 - 1024 : kRoom, most = p.pair ? paired : alone;
  p.warps = room / warp_bytes < most ? room / warp_bytes : most;
  if (p.warps > p.seg_spans) p.warps = p.seg_spans;
  p.smem = p.warps * warp_bytes;
  return p;
}

// The same bound at every call, so that calls from several threads agree.
template <typename F>
cudaError_t allow(F* kernel) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRoom);
}

template <typename T, bool kZ>
cudaError_t forward_t(const ScanArgs& a) {
  constexpr int SPAN = sizeof(T) == 2 ? 32 : 64;  // 8 tokens a run
  using G = Geo<T, SPAN>;
  using E = typename std::conditional<kZ, T, float>::type;
  // a later segment writes h_final while an earlier one reads h0: not in place
  const Plan p = plan<G>(a, kSlots * (tile_bytes<G, T>() + tile_bytes<G, E>()), kAlone, kPaired,
                         a.h0 && a.h0 == a.h_final);
  float* maps = (float*)a.ws;
  const dim3 grid(p.cols, p.segs);
  auto* run = scan_kernel<T, kZ, false, SPAN>;
  cudaError_t err = allow(run);
  if (err != cudaSuccess) return err;
  if (p.segs > 1) {
    auto* form = scan_kernel<T, kZ, true, SPAN>;
    if ((err = allow(form)) != cudaSuccess) return err;
    form<<<grid, p.warps * 32, p.smem, a.stream>>>(a, p.seg_spans, maps);
    if ((err = cudaGetLastError()) != cudaSuccess) return err;
  }
  run<<<grid, p.warps * 32, p.smem, a.stream>>>(a, p.seg_spans, maps);
  return cudaGetLastError();
}

template <typename T, bool kZ, int SPAN, bool kPair>
cudaError_t backward_p(const ScanArgs& a, const Plan& p) {
  float* maps = (float*)a.ws;
  float* part = p.segs > 1 ? maps + (size_t)2 * p.segs * a.C : a.dA;
  const dim3 grid(p.cols, p.segs);
  auto* run = scan_backward_kernel<T, kZ, false, SPAN, kPair>;
  cudaError_t err = allow(run);
  if (err != cudaSuccess) return err;
  if (p.segs > 1) {
    auto* form = scan_backward_kernel<T, kZ, true, SPAN, kPair>;
    if ((err = allow(form)) != cudaSuccess) return err;
    form<<<grid, p.warps * 32, p.smem, a.stream>>>(a, p.seg_spans, maps, nullptr);
    if ((err = cudaGetLastError()) != cudaSuccess) return err;
  }
  run<<<grid, p.warps * 32, p.smem, a.stream>>>(a, p.seg_spans, maps, part);
  if ((err = cudaGetLastError()) != cudaSuccess || !kZ || p.segs == 1) return err;
  sum_rows_kernel<<<(a.C + 63) / 64, 64, 0, a.stream>>>(part, p.segs, a.C, a.dA);
  return cudaGetLastError();
}

template <typename T, bool kZ>
cudaError_t backward_t(const ScanArgs& a) {
  constexpr int SPAN = sizeof(T) == 2 ? 32 : 64;  // 8 tokens a run
  using G = Geo<T, SPAN>;
  using E = typename std::conditional<kZ, T, float>::type;
  const Plan p = plan<G>(a, kSlots * (2 * tile_bytes<G, T>() + tile_bytes<G, E>()), kAloneBack,
                         kPairedBack, false);
  return p.pair ? backward_p<T, kZ, SPAN, true>(a, p) : backward_p<T, kZ, SPAN, false>(a, p);
}

}  // namespace

size_t scan_workspace_bytes(int T, int C) {
  // a block owns 16 channels of bf16, 8 of fp32
  const int wide = segments(T, (C + 15) / 16), narrow = segments(T, (C + 7) / 8);
  // a segment's map, and its row of dA
  return (size_t)3 * (wide > narrow ? wide : narrow) * C * sizeof(float);
}

cudaError_t launch_scan(const ScanArgs& a) {
  if (a.g || !a.z) return a.bf16 ? forward_t<__nv_bfloat16, false>(a) : forward_t<float, false>(a);
  return a.bf16 ? forward_t<__nv_bfloat16, true>(a) : forward_t<float, true>(a);
}

cudaError_t launch_scan_backward(const ScanArgs& a) {
  if (!a.dA)
    return a.bf16 ? backward_t<__nv_bfloat16, false>(a) : backward_t<float, false>(a);
  return a.bf16 ? backward_t<__nv_bfloat16, true>(a) : backward_t<float, true>(a);
}

cudaError_t launch_scan_step(const void* x, const void* z, const float* A, float* h, int B, int C,
                             bool bf16, void* y, cudaStream_t stream) {
  const size_t count = (size_t)B * C;
  const size_t grid = (count / 2 + 255) / 256;
  if (grid > 0x7fffffffu) return cudaErrorInvalidValue;
  if (bf16)
    step_kernel<<<(unsigned)grid, 256, 0, stream>>>((const __nv_bfloat16*)x,
                                                    (const __nv_bfloat16*)z, A, h, count, C,
                                                    (__nv_bfloat16*)y);
  else
    step_kernel<<<(unsigned)grid, 256, 0, stream>>>((const float*)x, (const float*)z, A, h, count,
                                                    C, (float*)y);
  return cudaGetLastError();
}

}  // namespace kda
