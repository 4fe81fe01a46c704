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

}  // namespace

cudaError_t launch_conv(const ConvArgs& a, cudaStream_t st) {
  return a.d.dtype == KDA_BF16 ? by_type<__nv_bfloat16>(a, st, false) : by_type<float>(a, st, false);
}

cudaError_t launch_conv_decode(const ConvArgs& a, cudaStream_t st) {
  return a.d.dtype == KDA_BF16 ? by_type<__nv_bfloat16>(a, st, true) : by_type<float>(a, st, true);
}

}  // namespace kda
