// kda_conv.cu -- short causal depthwise convolution with a pool of its last inputs.
//
//   y_t = act(bias + sum_{i < W} w_i x_{t-(W-1)+i})      per channel, W = 2..4
//
// 2 W operations a value against 2 elements moved: the kernels are bound by HBM, so the design
// is one pass over x and y, four channels a thread (one where rows are not aligned to four), with
// enough rows in flight.
//
// Prompts: the packed tokens are cut into strips of kStrip; a thread walks one strip for its
// channels with the last W-1 inputs in registers, so x is read once but for the W-1 rows before
// a strip (from L2).  Sequences are found per block from cu_seqlens (every block looks through all
// of it; no order is assumed), which leaves each token's sequence and position in shared memory.
// The first W-1 tokens of a sequence need its state, which the call also overwrites in pool mode:
// the thread whose strip holds a sequence's first token also takes those next W-2 tokens, reads
// the initial state, and then writes the final one, so no other thread reads what it overwrites.
#include "kda_internal.cuh"
#include "tc_ptx.cuh"

namespace kda {
namespace {

KDA_DEBUG_FLAG_DEFINE();

constexpr int kStrips = 8;      // strips a block; a strip is S tokens, walked by one thread
constexpr int kLanes = 32;      // channel vectors a block
constexpr int kConvThreads = kLanes * kStrips;

// Channels [c, c + VEC) of a row: 4 where every row is aligned to as many elements, else 1 (an odd
// channel count or pitch).  Eight bf16 channels a thread, in 16-byte accesses, need 124 registers
// for taps, window and rows in flight, which leaves three warps a scheduler: 309 us for 32768 x 12288
// (1.6 GB) against 277 us, 5.8 TB/s or 86 % of a copy's rate, with 4 channels, eight rows in flight and
// three blocks an SM (four blocks: 282 us with four rows in flight, 316 with eight, which then spill).
// One channel a thread has less in flight, so there five blocks share an SM: 155 us for 16384 x 8193 in
// bf16 (with three: 189; 8192 channels, four a thread: 99), 227 us in fp32 (with two: 304; 211), of dense
// states; with a pool and SiLU 168 and 232 (8192 channels: 106 and 228).
template <typename T, int VEC> struct Row;
template <> struct Row<float, 4> {
  using Raw = uint4;
  static __device__ __forceinline__ Raw load(const float* p) { return *reinterpret_cast<const uint4*>(p); }
  static __device__ __forceinline__ void store(float* p, const Raw& r) { *reinterpret_cast<uint4*>(p) = r; }
  static __device__ __forceinline__ void unpack(const Raw& r, float* f) {
    f[0] = __uint_as_float(r.x); f[1] = __uint_as_float(r.y);
    f[2] = __uint_as_float(r.z); f[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ Raw pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ Raw zero() { return make_uint4(0, 0, 0, 0); }
};
template <> struct Row<__nv_bfloat16, 4> {
  using Raw = uint2;
  static __device__ __forceinline__ Raw load(const __nv_bfloat16* p) { return *reinterpret_cast<const uint2*>(p); }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const Raw& r) { *reinterpret_cast<uint2*>(p) = r; }
  static __device__ __forceinline__ void unpack(const Raw& r, float* f) {
    f[0] = __uint_as_float(r.x << 16); f[1] = __uint_as_float(r.x & 0xffff0000u);
    f[2] = __uint_as_float(r.y << 16); f[3] = __uint_as_float(r.y & 0xffff0000u);
  }
  static __device__ __forceinline__ Raw pack(const float* f) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
  static __device__ __forceinline__ Raw zero() { return make_uint2(0, 0); }
};
template <typename T> struct Row<T, 1> {
  using Raw = T;
  static __device__ __forceinline__ Raw load(const T* p) { return *p; }
  static __device__ __forceinline__ void store(T* p, const Raw& r) { *p = r; }
  static __device__ __forceinline__ void unpack(const Raw& r, float* f) { f[0] = to_f32(r); }
  static __device__ __forceinline__ Raw pack(const float* f) { return from_f32<T>(f[0]); }
  static __device__ __forceinline__ Raw zero() { return from_f32<T>(0.f); }
};

// s * sigmoid(s) = s / (1 + e^-s).  The fast exponential and reciprocal are good to ~2^-21 plus what the
// exponent's rounding to 24 bits does, |s| 2^-24 (2^-18 at s = -80): far below a bf16 result's rounding.
// fp32 results take the accurate ones.
template <typename T, int VEC> __device__ __forceinline__ void silu(float* s) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) s[i] = s[i] / (1.f + expf(-s[i]));
}
template <> __device__ __forceinline__ void silu<__nv_bfloat16, 1>(float* s) {
  s[0] = __fdividef(s[0], 1.f + __expf(-s[0]));
}
template <> __device__ __forceinline__ void silu<__nv_bfloat16, 4>(float* s) {
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    float a = s[i], b = s[i + 1];
    mul2(a, b, -1.4426950408889634f, -1.4426950408889634f);
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
    a += 1.f;
    b += 1.f;
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
    mul2(s[i], s[i + 1], a, b);
  }
}

// One token: window win[0..W-1], oldest first (win[W-1] is the token itself). Channels in pairs: the
// kernel's instructions would otherwise take as long as its bytes.
template <typename T, int VEC, int W>
__device__ __forceinline__ void apply(const float (&win)[W][VEC], const float (&wt)[W][VEC],
                                      const float (&bias)[VEC], bool act, float* out) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) out[i] = bias[i];
#pragma unroll
  for (int j = 0; j < W; ++j) {
    if constexpr (VEC == 4) {
      acc2(out[0], out[1], wt[j][0], wt[j][1], win[j][0], win[j][1]);
      acc2(out[2], out[3], wt[j][2], wt[j][3], win[j][2], win[j][3]);
    } else {
      out[0] = fmaf(wt[j][0], win[j][0], out[0]);
    }
  }
  if (act) silu<T, VEC>(out);
}

// The taps [VEC][W] of VEC channels are W vectors in a row.
template <typename T, int VEC, int W>
__device__ __forceinline__ void load_taps(const T* w, const T* bias, int c, float (&wt)[W][VEC],
                                          float (&b)[VEC]) {
  using R = Row<T, VEC>;
  float flat[W * VEC];
#pragma unroll
  for (int j = 0; j < W; ++j) R::unpack(R::load(w + (size_t)c * W + j * VEC), flat + j * VEC);
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
#pragma unroll
    for (int j = 0; j < W; ++j) wt[j][i] = flat[i * W + j];
    b[i] = 0.f;
  }
  if (bias) R::unpack(R::load(bias + c), b);
}

template <typename T, int VEC, int W, int kStrip>
__global__ void __launch_bounds__(kConvThreads, VEC == 1 ? 5 : sizeof(T) == 4 ? 2 : 3)
conv_prompt_kernel(const T* __restrict__ x, int64_t x_pitch, const T* __restrict__ w,
                   const T* __restrict__ bias, const int32_t* __restrict__ cu, const T* state_in,
                   const int32_t* __restrict__ idx, T* state_out, int64_t slot_stride,
                   int64_t num_slots, T* __restrict__ y, uint32_t* __restrict__ status, int N,
                   int64_t total, int ch, bool act) {
  using R = Row<T, VEC>;
  constexpr int H = W - 1;                 // inputs a state holds
  constexpr int kTile = kStrip * kStrips;
  constexpr int kAhead = VEC > 1 && sizeof(T) == 4 ? 4 : 8;  // rows in flight while as many are computed
  static_assert(kStrip % kAhead == 0, "a strip is whole groups of rows");
  constexpr int kSpan = kTile + W - 2;     // tokens a block may own (see above)
  __shared__ int s_seq[kSpan];             // sequence of each token, -1: none
  __shared__ int64_t s_bos[kSpan];

  const int tid = threadIdx.x;
  // x's tiles on grid.x (up to 2^31-1 of them), channel blocks on grid.y
  const int64_t t0 = (int64_t)blockIdx.x * kTile;
  if (blockIdx.x == 0 && blockIdx.y == 0)
    check_all(status, cu, idx, N, total, total, idx ? num_slots : 0);

  for (int i = tid; i < kSpan; i += kConvThreads) s_seq[i] = -1;
  __syncthreads();
  for (int base = 0; base < N; base += kConvThreads) {
    const int n = base + tid;
    int64_t a = 0, b = 0;
    bool hit = n < N && seq_bounds(cu, n, total, &a, &b) && a < t0 + kSpan && b > t0;
    if (hit && idx) hit = resolve_slot(idx, n, num_slots) >= 0;
    // a warp writes each of its hits together: a long sequence fills the whole tile
    unsigned m = __ballot_sync(0xffffffffu, hit);
    while (m) {
      const int src = __ffs(m) - 1;
      m &= m - 1;
      const int64_t sa = __shfl_sync(0xffffffffu, a, src), sb = __shfl_sync(0xffffffffu, b, src);
      const int sn = __shfl_sync(0xffffffffu, n, src);
      const int lo = (int)(sa > t0 ? sa - t0 : 0);
      const int hi = (int)(sb < t0 + kSpan ? sb - t0 : kSpan);
      for (int i = lo + (tid & 31); i < hi; i += 32) {
        s_seq[i] = sn;
        s_bos[i] = sa;
      }
    }
  }
  __syncthreads();

  const int c = (blockIdx.y * kLanes + tid % kLanes) * VEC;
  if (c >= ch) return;
  // Sequences of length zero own no token: in dense mode their state is copied here, shared out
  // over the tiles.
  if (!idx && state_out && state_out != state_in) {
    for (int64_t n = blockIdx.x * (int64_t)kStrips + tid / kLanes; n < N;
         n += gridDim.x * (int64_t)kStrips) {
      int64_t a, b;
      if (!seq_bounds(cu, (int)n, total, &a, &b) || a != b) continue;
      for (int j = 0; j < H; ++j) {
        const int64_t at = n * slot_stride + (int64_t)j * ch + c;
        R::store(state_out + at, state_in ? R::load(state_in + at) : R::zero());
      }
    }
  }
  const int s0 = (tid / kLanes) * kStrip;  // this strip's first token in the tile
  float wt[W][VEC], bv[VEC];
  load_taps<T, VEC, W>(w, bias, c, wt, bv);

  // A strip inside one sequence and past its first W-1 tokens (nearly all of a long prompt): no
  // state, no owner to find, so the window rotates in registers over unrolled tokens.
  const int n0 = s_seq[s0];
  if (n0 >= 0 && s_seq[s0 + kStrip - 1] == n0 && t0 + s0 - s_bos[s0] >= H) {
    float win[W][VEC];
#pragma unroll
    for (int j = 0; j < H; ++j)
      R::unpack(R::load(x + (t0 + s0 - H + j) * x_pitch + c), win[j]);
    const T* xt = x + (t0 + s0) * x_pitch + c;
    T* yt = y + (t0 + s0) * ch + c;
    typename R::Raw nxt[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) nxt[u] = R::load(xt + u * x_pitch);
#pragma unroll 1
    for (int i0 = 0; i0 < kStrip; i0 += kAhead) {
      typename R::Raw cur[kAhead];
      xt += kAhead * x_pitch;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        cur[u] = nxt[u];
        if (i0 + kAhead < kStrip) nxt[u] = R::load(xt + u * x_pitch);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        float out[VEC];
        R::unpack(cur[u], win[H]);
        apply<T, VEC, W>(win, wt, bv, act, out);
        R::store(yt + (size_t)u * ch, R::pack(out));
#pragma unroll
        for (int j = 0; j < H; ++j) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) win[j][e] = win[j + 1][e];
        }
      }
      yt += (size_t)kAhead * ch;
    }
    return;
  }

  typename R::Raw h[H];   // the last W-1 inputs, oldest first
#pragma unroll
  for (int j = 0; j < H; ++j) h[j] = R::zero();
  int have = -1;          // sequence whose inputs h holds
#pragma unroll 1
  for (int i0 = 0; i0 < kStrip + W - 2; i0 += kAhead) {
    typename R::Raw nxt[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = s0 + i0 + u;
      nxt[u] = R::zero();
      if (i0 + u < kStrip + W - 2 && s_seq[i] >= 0)
        nxt[u] = R::load(x + (t0 + i) * x_pitch + c);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = s0 + i0 + u;
      if (i0 + u >= kStrip + W - 2) break;
      const int n = s_seq[i];
      if (n < 0) continue;
      const int64_t t = t0 + i, bos = s_bos[i], pos = t - bos;
      // the first W-1 tokens of a sequence belong to the strip of its first token
      const bool own = pos < H ? bos >= t0 + s0 && bos < t0 + s0 + kStrip : i < s0 + kStrip;
      if (!own) continue;
      // Lengths that run backwards make sequences overlap, and a token goes to one of them. Where that
      // took a sequence's first token away, its next W-1 have no state to start from (and perhaps no rows
      // before them): they are skipped.
      if (pos != 0 && pos < H && have != n) continue;
      if (pos == 0) {
        const int64_t slot = idx ? resolve_slot(idx, n, num_slots) : n;
        const T* si = state_in ? state_in + slot * slot_stride + c : nullptr;
#pragma unroll
        for (int j = 0; j < H; ++j) h[j] = si ? R::load(si + (size_t)j * ch) : R::zero();
        if (state_out) {
          const int64_t len = (int64_t)cu[n + 1] - bos;
          T* so = state_out + slot * slot_stride + c;
#pragma unroll
          for (int j = 0; j < H; ++j) {
            const int64_t p = len - H + j;  // position of the j-th kept input
            typename R::Raw r = h[0];
            if (p >= 0) {
              r = R::load(x + (bos + p) * x_pitch + c);
            } else {
#pragma unroll
              for (int e = 1; e < H; ++e)
                if (p + H == e) r = h[e];
            }
            R::store(so + (size_t)j * ch, r);
          }
        }
        have = n;
      } else if (have != n) {
#pragma unroll
        for (int j = 0; j < H; ++j)
          h[j] = KDA_CHECK(t - H + j >= bos) ? R::load(x + (t - H + j) * x_pitch + c) : R::zero();
        have = n;
      }
      float win[W][VEC], out[VEC];
#pragma unroll
      for (int j = 0; j < H; ++j) R::unpack(h[j], win[j]);
      R::unpack(nxt[u], win[H]);
      apply<T, VEC, W>(win, wt, bv, act, out);
      if (KDA_CHECK(t >= 0 && t < total && c + VEC <= ch)) R::store(y + t * ch + c, R::pack(out));
#pragma unroll
      for (int j = 0; j + 1 < H; ++j) h[j] = h[j + 1];
      h[H - 1] = nxt[u];
    }
  }
  KDA_DEBUG_FOLD(status);
}

// One token, or a few drafted ones, a row: a thread holds the W-1 inputs of four channels (or one).
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(128)
conv_token_kernel(const T* __restrict__ x, int64_t x_pitch, const T* __restrict__ w,
                  const T* __restrict__ bias, const int32_t* __restrict__ cu, T* pool,
                  const int32_t* __restrict__ idx, int64_t slot_stride, int64_t num_slots,
                  T* __restrict__ y, uint32_t* __restrict__ status, int N, int64_t total, int ch,
                  bool act, T* __restrict__ cache, int64_t cache_pitch, int max_steps,
                  bool update_pool) {
  using R = Row<T, VEC>;
  constexpr int H = W - 1;
  if (blockIdx.x == 0 && blockIdx.y == 0)
    check_all(status, cu, idx, N, total, max_steps, num_slots);
  const int n = blockIdx.x;
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * VEC;
  if (c >= ch) return;
  int64_t bos = n, eos = n + 1;
  if (cu && (!seq_bounds(cu, n, total, &bos, &eos) || eos - bos > max_steps)) return;
  const int64_t slot = idx ? resolve_slot(idx, n, num_slots) : (n < num_slots ? n : -1);
  if (slot < 0) return;
  T* so = pool + slot * slot_stride + c;
  typename R::Raw h[H];
#pragma unroll
  for (int j = 0; j < H; ++j) h[j] = R::load(so + (size_t)j * ch);
  typename R::Raw cur = bos < eos ? R::load(x + bos * x_pitch + c) : R::zero();
  float wt[W][VEC], bv[VEC];
  load_taps<T, VEC, W>(w, bias, c, wt, bv);
  for (int64_t t = bos; t < eos; ++t) {
    const typename R::Raw nxt = t + 1 < eos ? R::load(x + (t + 1) * x_pitch + c) : R::zero();
    float win[W][VEC], out[VEC];
#pragma unroll
    for (int j = 0; j < H; ++j) R::unpack(h[j], win[j]);
    R::unpack(cur, win[H]);
    apply<T, VEC, W>(win, wt, bv, act, out);
    if (KDA_CHECK(t >= 0 && t < total && c + VEC <= ch)) R::store(y + t * ch + c, R::pack(out));
#pragma unroll
    for (int j = 0; j + 1 < H; ++j) h[j] = h[j + 1];
    h[H - 1] = cur;
    cur = nxt;
    if (cache) {
      T* co = cache + n * cache_pitch + (t - bos) * ((int64_t)H * ch) + c;
#pragma unroll
      for (int j = 0; j < H; ++j) R::store(co + (size_t)j * ch, h[j]);
    }
  }
  if (update_pool) {
#pragma unroll
    for (int j = 0; j < H; ++j) R::store(so + (size_t)j * ch, h[j]);
  }
  KDA_DEBUG_FOLD(status);
}

// ---- backward -------------------------------------------------------------------------------
// With z the sum before the activation and dz = dy act'(z):
//   by an input   sum over its taps of w_i dz_{t+(W-1)-i}, and the final state's derivative where it is one
//                 of the last W-1 inputs
//   by w_i        sum over the tokens of dz_t x_{t-(W-1)+i}        by the bias: sum of dz
// Two rows are read and one is written a token, and z is formed again: bound by HBM. A warp walks a long run of
// the packed rows for its channels, four a lane, and the W-1 rows behind it (whose dz its last rows' derivatives
// need; they are the next run's to count in the sums), with the last W inputs and dz in registers and the rows
// ahead of it on their way into shared memory, each lane's own. The sums by the weights stay in
// registers over the run, are added over a CTA's warps at its end, and over the CTAs by a second kernel, each
// in a fixed order. Four rows at a time: where they, and W-1 on either side, are of one sequence, nothing is looked up;
// else row by row. Which sequence a row belongs to is written down beforehand by a small kernel.
// 32768 x 12288 bf16, 4 taps, SiLU: 457 us, 5.3 TB/s, 78 % of the copy rate; its two special functions and some 30
// other instructions an element take about as long as its bytes. 2741 x 1003 fp32 in 37 sequences: 25 us, three
// launches and runs of 32 rows whose sequences are looked up one by one.
constexpr int kBackWarps = 8;
constexpr int kBackThreads = kBackWarps * 32;
constexpr int kQuad = 4;

// g *= act'(z): of z sigmoid(z) it is s + s (z - z s), s = sigmoid(z).
template <typename T, int VEC> __device__ __forceinline__ void silu_slope(const float (&z)[VEC], float (&g)[VEC]) {
  float s[VEC], q[VEC];
  if constexpr (sizeof(T) == 2 && VEC == 4) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      s[i] = z[i];
      s[i + 1] = z[i + 1];
      mul2(s[i], s[i + 1], -1.4426950408889634f, -1.4426950408889634f);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(s[i]));
    add2(s[0], s[1], 1.f, 1.f);
    add2(s[2], s[3], 1.f, 1.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(s[i]));
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      float m = z[i], n = z[i + 1];
      mul2(m, n, s[i], s[i + 1]);
      q[i] = z[i];
      q[i + 1] = z[i + 1];
      sub2(q[i], q[i + 1], m, n);
      fma2(q[i], q[i + 1], s[i], s[i + 1], s[i], s[i + 1]);
      mul2(g[i], g[i + 1], q[i], q[i + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float e = sizeof(T) == 2 ? __expf(-z[i]) : expf(-z[i]);
      s[i] = sizeof(T) == 2 ? __fdividef(1.f, 1.f + e) : 1.f / (1.f + e);
      g[i] *= fmaf(z[i] - z[i] * s[i], s[i], s[i]);
    }
  }
}
// d = x * y + c
__device__ __forceinline__ void fma3(float& d, float& e, float x, float y, float u, float v, float c, float f) {
  unsigned long long de, xy, uv, cf;
  asm("mov.b64 %0, {%1, %2};" : "=l"(xy) : "f"(x), "f"(y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(uv) : "f"(u), "f"(v));
  asm("mov.b64 %0, {%1, %2};" : "=l"(cf) : "f"(c), "f"(f));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(de) : "l"(xy), "l"(uv), "l"(cf));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d), "=f"(e) : "l"(de));
}
template <int VEC>
__device__ __forceinline__ void fma(float (&d)[VEC], const float (&x)[VEC], const float (&y)[VEC], const float (&c)[VEC]) {
  if constexpr (VEC == 4) {
    fma3(d[0], d[1], x[0], x[1], y[0], y[1], c[0], c[1]);
    fma3(d[2], d[3], x[2], x[3], y[2], y[3], c[2], c[3]);
  } else {
    d[0] = fmaf(x[0], y[0], c[0]);
  }
}
// d = x * y
template <int VEC> __device__ __forceinline__ void mul(float (&d)[VEC], const float (&x)[VEC], const float (&y)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) d[i] = x[i];
  if constexpr (VEC == 4) {
    mul2(d[0], d[1], y[0], y[1]);
    mul2(d[2], d[3], y[2], y[3]);
  } else {
    d[0] *= y[0];
  }
}
// a += x * y
template <int VEC> __device__ __forceinline__ void acc(float (&a)[VEC], const float (&x)[VEC], const float (&y)[VEC]) {
  if constexpr (VEC == 4) {
    acc2(a[0], a[1], x[0], x[1], y[0], y[1]);
    acc2(a[2], a[3], x[2], x[3], y[2], y[3]);
  } else {
    a[0] = fmaf(x[0], y[0], a[0]);
  }
}

// Four rows of x and dy on their way to `to`, [row][x, dy][lane]. Elements of two bytes, which no asynchronous copy
// takes, go through registers: those that were asked for last time are put down, the next ones are asked for (8192
// rows of 12287 channels: 304 us, 559 with each put down at once and one round of CTAs).
template <typename Raw> struct Ahead {};
template <> struct Ahead<__nv_bfloat16> { __nv_bfloat16 x[kQuad], dy[kQuad]; };
template <typename T, int VEC>
__device__ __forceinline__ void fetch_quad(typename Row<T, VEC>::Raw* to, Ahead<typename Row<T, VEC>::Raw>& ahead,
                                           const T*& x, int64_t x_pitch, const T*& dy, int64_t dy_pitch, int rows) {
  using Raw = typename Row<T, VEC>::Raw;
  if constexpr (sizeof(Raw) == 2) {
#pragma unroll
    for (int u = 0; u < kQuad; ++u) {
      to[(u * 2) * 32] = ahead.x[u];
      to[(u * 2 + 1) * 32] = ahead.dy[u];
    }
  }
  auto one = [&](int u) {
    if constexpr (sizeof(Raw) >= 4) {
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(tc::smem_u32(to + (u * 2) * 32)), "l"(x),
                   "n"((int)sizeof(Raw))
                   : "memory");
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(tc::smem_u32(to + (u * 2 + 1) * 32)), "l"(dy),
                   "n"((int)sizeof(Raw))
                   : "memory");
    } else {
      ahead.x[u] = Row<T, VEC>::load(x);
      ahead.dy[u] = Row<T, VEC>::load(dy);
    }
    x += x_pitch;
    dy += dy_pitch;
  };
  if (rows >= kQuad) {
#pragma unroll
    for (int u = 0; u < kQuad; ++u) one(u);
  } else if constexpr (sizeof(Raw) == 2) {
#pragma unroll
    for (int u = 0; u < kQuad; ++u)
      if (u < rows) one(u);
  } else {
#pragma unroll 1
    for (int u = 0; u < rows; ++u) one(u);
  }
  if constexpr (sizeof(Raw) >= 4) asm volatile("cp.async.commit_group;" ::: "memory");
}

// Fours of rows in shared memory, one of them in work (bf16, 32768 x 12288: 3 of them 460 us, 4 and 5 461, 6, which
// leave room for fewer CTAs, 514).
template <typename T, int VEC> constexpr int back_depth() { return sizeof(typename Row<T, VEC>::Raw) == 16 ? 2 : 3; }

template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kBackThreads, 2)
conv_back_kernel(const T* __restrict__ dy, int64_t dy_pitch, const T* __restrict__ x, int64_t x_pitch,
                 const T* __restrict__ w, const T* __restrict__ bias, const int32_t* __restrict__ cu,
                 const int32_t* __restrict__ seq, const T* __restrict__ state, const T* __restrict__ dfinal,
                 T* __restrict__ dx, T* __restrict__ dstate, float* __restrict__ part, uint32_t* __restrict__ status,
                 int64_t total, int64_t run, int ch, bool act, bool want_db) {
  using R = Row<T, VEC>;
  using Raw = typename R::Raw;
  constexpr int H = W - 1;
  constexpr int kDepth = back_depth<T, VEC>();
  extern __shared__ __align__(16) uint8_t s_ring[];   // [warp][four of rows][row][x, dy][lane]
  __shared__ float s_sum[kBackWarps][32 * VEC];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c = (blockIdx.x * 32 + lane) * VEC;
  const bool in = c < ch;
  const int64_t t_lo = ((int64_t)blockIdx.y * kBackWarps + warp) * run;
  const int64_t t_hi = t_lo + run < total ? t_lo + run : total;        // the rows of this run
  const int64_t t_end = t_hi + H < total ? t_hi + H : total;           // and those behind it
  float wt[W][VEC], bv[VEC], dw[W][VEC], db[VEC];
  float win[W][VEC];      // the last W inputs, oldest first
  float dz[W][VEC];       // dz of the last W tokens, oldest first
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    bv[i] = db[i] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) wt[j][i] = dw[j][i] = win[j][i] = dz[j][i] = 0.f;
  }
  if (in) load_taps<T, VEC, W>(w, bias, c, wt, bv);
  tc::grid_dep_wait();

  auto shift = [&] {
#pragma unroll
    for (int j = 0; j < H; ++j) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        win[j][e] = win[j + 1][e];
        dz[j][e] = dz[j + 1][e];
      }
    }
  };
  auto slope = [&] {   // dz of the newest token, from dy in its place
    if (!act) return;
    float z[VEC];
    fma<VEC>(z, win[0], wt[0], bv);
#pragma unroll
    for (int j = 1; j < W; ++j) acc<VEC>(z, win[j], wt[j]);
    silu_slope<T, VEC>(z, dz[H]);
  };
  auto count = [&] {
#pragma unroll
    for (int j = 0; j < W; ++j) acc<VEC>(dw[j], dz[H], win[j]);
    if (!want_db) return;   // (without a bias it is the derivative by one of zeros)
    if constexpr (VEC == 4) {
      add2(db[0], db[1], dz[H][0], dz[H][1]);
      add2(db[2], db[3], dz[H][2], dz[H][3]);
    } else {
      db[0] += dz[H][0];
    }
  };
  // One row by itself, t < t_end, of sequence n; the derivative of row t - H is complete then.
  int last = -1;          // sequence of the row before, as far as this run has seen it
  // derivative by the state of the sequence that began in this run (in registers it would spill: 557 against 462 us)
  float (*ds)[VEC] = reinterpret_cast<float(*)[VEC]>(s_ring + kBackThreads * kDepth * kQuad * 2 * sizeof(Raw)) + tid * H;
  auto row = [&](int64_t t, int n, const Raw& xr, const Raw& gr) {
    shift();
#pragma unroll
    for (int e = 0; e < VEC; ++e) dz[H][e] = 0.f;
    if (n >= 0) {
      const int64_t bos = cu[n], pos = t - bos;
      if (last != n) {
        // the inputs before the token: of the sequence, or of its state
#pragma unroll
        for (int j = 0; j < H; ++j) {
          const int64_t p = pos - H + j;
          if (p >= 0) R::unpack(R::load(x + (bos + p) * x_pitch + c), win[j]);
          else if (state) R::unpack(R::load(state + ((int64_t)n * H + H + p) * ch + c), win[j]);
          else
#pragma unroll
            for (int e = 0; e < VEC; ++e) win[j][e] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < H; ++j) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) ds[j][e] = 0.f;
        }
      }
      R::unpack(xr, win[H]);
      R::unpack(gr, dz[H]);
      slope();
      if (t < t_hi) count();
      // a sequence's state is read by its first W-1 tokens, which the run of the first one sees all
      if (dstate && pos < H && t - pos >= t_lo && t - pos < t_hi) {
        const int64_t len = (int64_t)cu[n + 1] - bos;
#pragma unroll
        for (int m = 0; m < H; ++m) {
#pragma unroll
          for (int p = 0; p <= m; ++p) {
            if (p == pos) {
#pragma unroll
              for (int e = 0; e < VEC; ++e) ds[m][e] = fmaf(dz[H][e], wt[m - p][e], ds[m][e]);
            }
          }
        }
        if (pos == H - 1 || pos == len - 1) {
#pragma unroll
          for (int m = 0; m < H; ++m) {
            if (dfinal && m >= len) {
              float f[VEC];
              R::unpack(R::load(dfinal + ((int64_t)n * H + m - len) * ch + c), f);
#pragma unroll
              for (int e = 0; e < VEC; ++e) ds[m][e] += f[e];
            }
            R::store(dstate + ((int64_t)n * H + m) * ch + c, R::pack(ds[m]));
          }
        }
      }
    }
    last = n;
  };
  // dx of row o, whose W-1 tokens behind it are in dz
  auto derive = [&](int64_t o) {
    const int n = seq[o];
    float out[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) out[e] = 0.f;
    if (n >= 0) {
#pragma unroll
      for (int d = 0; d < W; ++d)
        if (d == 0 || (o + d < total && seq[o + d] == n)) acc<VEC>(out, dz[d], wt[H - d]);
      if (dfinal) {
        const int64_t back = (int64_t)cu[n + 1] - o;   // 1 for the last token
        if (back <= H) {
          float f[VEC];
          R::unpack(R::load(dfinal + ((int64_t)n * H + H - back) * ch + c), f);
#pragma unroll
          for (int e = 0; e < VEC; ++e) out[e] += f[e];
        }
      }
    }
    if (KDA_CHECK(o >= 0 && o < total && c + VEC <= ch)) R::store(dx + o * ch + c, R::pack(out));
  };

  if (t_lo < t_hi) {
    Raw* const ring = reinterpret_cast<Raw*>(s_ring) + warp * (kDepth * kQuad * 2 * 32) + lane;
    const T *xp = x + t_lo * x_pitch + c, *gp = dy + t_lo * dy_pitch + c;
    int to_ask = in ? (int)(t_end - t_lo) : 0;   // rows that are not on their way yet
    int to = sizeof(Raw) == 2 ? kDepth - 1 : 0, from = 0;   // (what is put down first was not asked for)
    Ahead<Raw> asked = {};
    auto ahead = [&] {
      fetch_quad<T, VEC>(ring + to * (kQuad * 2 * 32), asked, xp, x_pitch, gp, dy_pitch, to_ask);
      to_ask -= kQuad;
      to = to + 1 == kDepth ? 0 : to + 1;
    };
#pragma unroll 1
    for (int q = 0; q + 1 < kDepth; ++q) ahead();
    // bit i: row t - H + 1 + i is of the same sequence as the row before it, of 16 rows t at a time; the next
    // 16 rows' are looked up ahead
    uint32_t follows = 0;
    int mine, prior;
    auto look = [&](int64_t t) {
      const int64_t u = t - H + 1 + lane;
      const bool ok = u > 0 && u < total;
      mine = ok ? seq[u] : -1;
      prior = ok ? seq[u - 1] : -1;
    };
    look(t_lo);
    T* op = dx + (t_lo - H) * ch + c;
#pragma unroll 1
    for (int64_t t = t_lo; t < t_end; t += kQuad) {
      const int at = (int)(t - t_lo) % 16;
      if (at == 0) {
        follows = __ballot_sync(0xffffffffu, mine >= 0 && mine == prior);
        look(t + 16);
      }
      ahead();
      asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
      const uint32_t bits = follows >> at;
      constexpr uint32_t kPlain = (1u << (kQuad - 1 + 2 * H)) - 1;
      const Raw* raw = ring + from * (kQuad * 2 * 32);
      from = from + 1 == kDepth ? 0 : from + 1;
      if ((bits & kPlain) == kPlain && t >= t_lo + H && t + kQuad <= t_hi) {
        if (in) {
#pragma unroll
          for (int u = 0; u < kQuad; ++u) {
            shift();
            R::unpack(raw[(u * 2) * 32], win[H]);
            R::unpack(raw[(u * 2 + 1) * 32], dz[H]);
            slope();
            count();
            float o[VEC];
            mul<VEC>(o, dz[0], wt[H]);
#pragma unroll
            for (int d = 1; d < W; ++d) acc<VEC>(o, dz[d], wt[H - d]);
            R::store(op + (int64_t)u * ch, R::pack(o));
          }
        }
        last = -2;   // of the rows' sequence; whoever goes on row by row reads the inputs again
      } else if (in) {
#pragma unroll 1
        for (int u = 0; u < kQuad; ++u) {
          if (t + u < t_end) row(t + u, seq[t + u], raw[(u * 2) * 32], raw[(u * 2 + 1) * 32]);
          else shift();
          const int64_t o = t + u - H;
          if (o >= t_lo && o < t_hi) derive(o);
        }
      }
      op += kQuad * ch;
    }
    if (in) {   // rows at the end of all, with none behind them
      for (int64_t t = (t_end - t_lo + kQuad - 1) / kQuad * kQuad + t_lo; t - H < t_hi; ++t) {
        shift();
        derive(t - H);
      }
    }
  }
  // parts [run of CTAs][W + 1][Ch] of the sums
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < VEC; ++e) s_sum[warp][lane * VEC + e] = j < W ? dw[j < W ? j : 0][e] : db[e];
    __syncthreads();
    for (int k = tid; k < 32 * VEC; k += kBackThreads) {
      const int64_t cc = (int64_t)blockIdx.x * 32 * VEC + k;
      float sum = 0.f;
#pragma unroll
      for (int q = 0; q < kBackWarps; ++q) sum += s_sum[q][k];
      if (cc < ch) part[((int64_t)blockIdx.y * (W + 1) + j) * ch + cc] = sum;
    }
  }
  KDA_DEBUG_FOLD(status);
}

// The sequence of each row (-1: none that is valid; the last one that holds it where lengths run
// backwards), the status word, and the derivatives by the states of sequences without tokens (dfinal) and of
// invalid ones (0).
template <typename T>
__global__ void __launch_bounds__(1024)
conv_back_plan_kernel(const int32_t* __restrict__ cu, int N, int64_t total, uint32_t* __restrict__ status,
                      int32_t* __restrict__ seq, const T* __restrict__ dfinal, T* __restrict__ dstate, int64_t row) {
  __shared__ int s_seq[1024];
  const int tid = threadIdx.x;
  tc::grid_dep_launch_dependents();
  if (blockIdx.x == 0) check_all(status, cu, nullptr, N, total, total, 0);
  for (int64_t t0 = (int64_t)blockIdx.x * 1024; t0 < total; t0 += (int64_t)gridDim.x * 1024) {
    sequences_of<1024>(s_seq, cu, nullptr, 0, N, total, t0);
    if (t0 + tid < total) seq[t0 + tid] = s_seq[tid];
    __syncthreads();
  }
  if (dstate) rows_without_tokens(cu, N, total, dfinal, dstate, row, true);
}

// The tiles' parts of the sums, added in a fixed order.
__global__ void __launch_bounds__(256)
conv_sum_kernel(const float* __restrict__ part, int64_t tiles, int ch, int W, float* __restrict__ dw,
                float* __restrict__ db) {
  __shared__ float s[8][32];
  tc::grid_dep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = blockIdx.y;
  const int c = blockIdx.x * 32 + lane;
  float sum = 0.f;
  if (c < ch) {
#pragma unroll 8
    for (int64_t k = warp; k < tiles; k += 8) sum += part[(k * (W + 1) + j) * ch + c];
  }
  s[warp][lane] = sum;
  __syncthreads();
  if (warp != 0 || c >= ch) return;
#pragma unroll
  for (int q = 1; q < 8; ++q) sum += s[q][lane];
  if (j < W) dw[(int64_t)c * W + j] = sum;
  else if (db) db[c] = sum;
}

// Rows that start on a boundary of 4 elements.
bool rows4(const void* p, int64_t pitch, int size) {
  return !p || ((uintptr_t)p % (4 * size) == 0 && pitch % 4 == 0);
}

template <typename T, int VEC, int W, int kStrip>
cudaError_t launch_strips(const ConvArgs& a, cudaStream_t st) {
  const int ch = a.d.channels;
  const int64_t tiles = (a.d.total_tokens + kStrip * kStrips - 1) / (kStrip * kStrips);
  dim3 grid((unsigned)(tiles > 0 ? tiles : 1),  // no tokens: empty sequences may want their state
            (unsigned)((ch + kLanes * VEC - 1) / (kLanes * VEC)));
  conv_prompt_kernel<T, VEC, W, kStrip><<<grid, kConvThreads, 0, st>>>(
      (const T*)a.x, a.d.x_pitch, (const T*)a.w, (const T*)a.bias, a.cu, (const T*)a.state_in,
      a.idx, (T*)a.state_out, a.slot_stride, a.d.num_slots, (T*)a.y, a.status, a.d.num_seqs,
      a.d.total_tokens, ch, a.d.silu != 0);
  return cudaGetLastError();
}

// Long strips read fewer rows twice and set up less often; they are taken once they leave four blocks an
// SM (bf16, 12288 channels, strips of 32 against 8: 46 against 52 us for 4096 tokens, 1536 blocks, but
// 16.5 against 14.7 us for 1024, 384 blocks; 4096 channels: 12.7 against 6.2 us for 512 tokens).
template <typename T, int VEC, int W>
cudaError_t launch_prompt(const ConvArgs& a, cudaStream_t st) {
  const int64_t blocks = (a.d.total_tokens / (32 * kStrips)) * (a.d.channels / (kLanes * VEC));
  return blocks >= 4 * gpu_sms() ? launch_strips<T, VEC, W, 32>(a, st) : launch_strips<T, VEC, W, 8>(a, st);
}

template <typename T, int VEC, int W>
cudaError_t launch_token(const ConvArgs& a, cudaStream_t st) {
  const int ch = a.d.channels;
  dim3 grid((unsigned)a.d.num_seqs, (unsigned)((ch + 128 * VEC - 1) / (128 * VEC)));
  conv_token_kernel<T, VEC, W><<<grid, 128, 0, st>>>(
      (const T*)a.x, a.d.x_pitch, (const T*)a.w, (const T*)a.bias, a.cu, (T*)a.state_out, a.idx,
      a.slot_stride, a.d.num_slots, (T*)a.y, a.status, a.d.num_seqs, a.d.total_tokens, ch,
      a.d.silu != 0, (T*)a.cache, a.cache_pitch, a.max_steps, a.update_pool);
  return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t by_width(const ConvArgs& a, cudaStream_t st, bool token) {
  switch (a.d.width) {
    case 2: return token ? launch_token<T, VEC, 2>(a, st) : launch_prompt<T, VEC, 2>(a, st);
    case 3: return token ? launch_token<T, VEC, 3>(a, st) : launch_prompt<T, VEC, 3>(a, st);
    default: return token ? launch_token<T, VEC, 4>(a, st) : launch_prompt<T, VEC, 4>(a, st);
  }
}

template <typename T>
cudaError_t by_type(const ConvArgs& a, cudaStream_t st, bool token) {
  constexpr int VEC = 4;
  const int64_t ch = a.d.channels, e = sizeof(T);
  const bool wide = rows4(a.x, a.d.x_pitch, e) && rows4(a.y, ch, e) && rows4(a.w, ch, e) &&
                    rows4(a.bias, ch, e) &&
                    rows4(a.state_in, ch, e) && rows4(a.state_in, a.slot_stride, e) &&
                    rows4(a.state_out, ch, e) && rows4(a.cache, a.cache_pitch, e) && ch % VEC == 0;
  return wide ? by_width<T, VEC>(a, st, token) : by_width<T, 1>(a, st, token);
}

// CTAs a channel block, of runs of 32 rows at least a warp: as many as fit the GPU at two an SM, or, where
// that leaves a fifth of it without work, as many as fill it two to four times over (8192 rows in bf16: 10240
// channels by one round, 240 CTAs of 304 places, 135 us, by two 131; but 8192 channels, 256 places of 304, 105 by
// one, 113 by two; one CTA an SM: 224 against 135 us for 12288 channels).
struct BackShape {
  int64_t run, ctas;
};
BackShape back_shape(const kda_conv_desc_t& d, int vec) {
  const int64_t blocks = (d.channels + 32 * vec - 1) / (32 * vec), T = d.total_tokens, room = 2ll * gpu_sms();
  int64_t ctas = 1, best = 0;   // of 1024 places, those with work
  for (int rounds = 1; rounds <= 4 && best < 820; ++rounds) {
    const int64_t n = rounds * room / blocks, used = n * blocks * 1024 / (rounds * room);
    if (used > best) {
      ctas = n;
      best = used;
    }
  }
  const int64_t most = (T + 32 * kBackWarps - 1) / (32 * kBackWarps);
  ctas = ctas < most ? ctas : most;
  ctas = ctas > 0 ? ctas : 1;
  int64_t run = (T + ctas * kBackWarps - 1) / (ctas * kBackWarps);
  run = (run + 15) / 16 * 16;
  return {run > 0 ? run : 16, ctas};
}
size_t back_part(const kda_conv_desc_t& d) {   // behind the header: the rows' sequences, then the sums
  return kWsPayload + ((size_t)d.total_tokens * 4 + 255) / 256 * 256;
}

template <typename T, int VEC, int W>
cudaError_t launch_back(const ConvBackArgs& a, cudaStream_t st) {
  const int ch = a.d.channels;
  const BackShape s = back_shape(a.d, VEC);
  int32_t* seq = reinterpret_cast<int32_t*>(a.ws + kWsPayload);
  float* part = reinterpret_cast<float*>(a.ws + back_part(a.d));
  uint32_t* status = &reinterpret_cast<WsHeader*>(a.ws)->status;
  int64_t plan = (a.d.total_tokens + 1023) / 1024, most = 2ll * gpu_sms();
  if (a.dstate) plan += row_blocks(a.d.num_seqs, (int64_t)(W - 1) * ch, most);
  plan = plan < 1 ? 1 : plan > most ? most : plan;
  conv_back_plan_kernel<T><<<(unsigned)plan, 1024, 0, st>>>(a.cu, a.d.num_seqs, a.d.total_tokens, status, seq,
                                                          (const T*)a.dfinal, (T*)a.dstate, (int64_t)(W - 1) * ch);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  dim3 grid((unsigned)((ch + 32 * VEC - 1) / (32 * VEC)), (unsigned)s.ctas);
  const int bytes = kBackThreads * (back_depth<T, VEC>() * kQuad * 2 * (int)sizeof(typename Row<T, VEC>::Raw) +
                                    (W - 1) * VEC * 4);
  auto* kernel = conv_back_kernel<T, VEC, W>;
  if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) != cudaSuccess) return e;
  e = launch_behind(
      kernel, grid, dim3(kBackThreads), bytes, st, (const T*)a.dy, a.dy_pitch,
      (const T*)a.x, a.d.x_pitch, (const T*)a.w, (const T*)a.bias, a.cu, seq,
      (const T*)a.state, (const T*)a.dfinal, (T*)a.dx, (T*)a.dstate, part, status, a.d.total_tokens, s.run, ch,
      a.d.silu != 0, a.db != nullptr);
  if (e != cudaSuccess) return e;
  return launch_behind(conv_sum_kernel, dim3((unsigned)((ch + 31) / 32), W + 1), dim3(256), 0, st, part, s.ctas, ch, W,
                       a.dw, a.db);
}

template <typename T, int VEC>
cudaError_t back_by_width(const ConvBackArgs& a, cudaStream_t st) {
  switch (a.d.width) {
    case 2: return launch_back<T, VEC, 2>(a, st);
    case 3: return launch_back<T, VEC, 3>(a, st);
    default: return launch_back<T, VEC, 4>(a, st);
  }
}

template <typename T>
cudaError_t back_by_type(const ConvBackArgs& a, cudaStream_t st) {
  constexpr int VEC = 4;
  const int64_t ch = a.d.channels, e = sizeof(T);
  const bool wide = rows4(a.x, a.d.x_pitch, e) && rows4(a.dy, a.dy_pitch, e) && rows4(a.w, ch, e) &&
                    rows4(a.bias, ch, e) && rows4(a.state, ch, e) && rows4(a.dfinal, ch, e) &&
                    rows4(a.dx, ch, e) && rows4(a.dstate, ch, e) && ch % VEC == 0;
  return wide ? back_by_width<T, VEC>(a, st) : back_by_width<T, 1>(a, st);
}

}  // namespace

size_t conv_back_workspace(const kda_conv_desc_t& d) {
  const int64_t four = back_shape(d, 4).ctas, one = back_shape(d, 1).ctas;   // either form may be taken
  return back_part(d) + (size_t)(four > one ? four : one) * (d.width + 1) * d.channels * 4;
}

cudaError_t launch_conv_back(const ConvBackArgs& a, cudaStream_t st) {
  return a.d.dtype == KDA_BF16 ? back_by_type<__nv_bfloat16>(a, st) : back_by_type<float>(a, st);
}

cudaError_t launch_conv(const ConvArgs& a, cudaStream_t st) {
  return a.d.dtype == KDA_BF16 ? by_type<__nv_bfloat16>(a, st, false) : by_type<float>(a, st, false);
}

cudaError_t launch_conv_decode(const ConvArgs& a, cudaStream_t st) {
  return a.d.dtype == KDA_BF16 ? by_type<__nv_bfloat16>(a, st, true) : by_type<float>(a, st, true);
}

}  // namespace kda
