// kda_gated.cu -- gated linear recurrence, per channel, of packed sequences: prompts, their backward
// pass, tokens and drafts.
//
//   s = sigmoid(r_t)   g = -exp(A_log) s   a = e^g   m = sqrt(1 - a^2)   u = sigmoid(i_t) x_t
//   h_t = a h_{t-1} + m u        y_t = h_t
//
// and backward, with l_t the loss's derivative by h_t and e_t = a_t l_t what of it reaches h_{t-1}:
//
//   l_t = dy_t + e_{t+1}         dx = m sigmoid(i) l    di = m l u (1 - sigmoid(i))
//   p = g a l h_{t-1} - a^2 (g / m) u l                 dr = p (1 - s)      dA_log = sum of p
//
// (g / m goes to 0 with g, so p needs no case for closed gates; 1 - a^2 is -expm1(2 g), whose digits
// a subtraction would lose.)
//
// Both passes are bound by HBM if their arithmetic (five or six special functions an element) hides behind
// it, so each reads its inputs once. The packed rows, whatever sequences they belong to, are cut into
// tiles of kWarps * S rows by 32 * V channels; a warp takes S rows of a tile, a lane V channels. What a
// run of rows does to the state is h -> A h + H, so
//   1. each warp forms a and m u of its rows in registers, and their (A, H);
//   2. the tile's (A, H) goes to global memory for the tiles after it, and the state before the tile is
//      put together from those of the tiles before it: the state at the start of its group of kGroup
//      tiles, then the tiles of the group in order;
//   3. each warp runs through its rows again, from registers, and writes them.
// Tiles are handed out by a counter, earlier rows first, so a tile waits only for tiles that run already.
// The state at a group's start comes from the group before it, one wait for kGroup tiles. The order of all
// sums is fixed, whichever tile comes first: results are bit-identical from run to run. A sequence's first
// row starts from its own state, and no product carries the state before it (which may be no number).
//
// The backward pass runs over the tiles from the last to the first, e in the place of h. It needs
// h_{t-1} as well; the forward pass left the state before each kCarryRows rows for it.
#include "kda_internal.cuh"
#include "tc_ptx.cuh"

namespace kda {
namespace {

KDA_DEBUG_FLAG_DEFINE();

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kGroup = 16;
constexpr int kPlanRows = 1024;   // rows a block of the planning kernel
constexpr float kLog2e = 1.4426950408889634f;

// Workspace behind the header: the sequence of each row, each tile's flag, each group's flag, each
// tile's (A, H) and each group's state, all channels; the backward pass's parts of dA_log.
struct Layout {
  int64_t tiles, groups;
  int32_t blocks;               // channel blocks
  size_t seq, flag, gflag, agg_a, agg_h, group, part, total;
};
__host__ __device__ inline Layout layout_of(int64_t T, int32_t ch, int rows, int lane_ch, bool back) {
  Layout l;
  l.tiles = (T + rows - 1) / rows;
  l.groups = (l.tiles + kGroup - 1) / kGroup;
  l.blocks = (ch + 32 * lane_ch - 1) / (32 * lane_ch);
  size_t at = kWsPayload;
  auto take = [&](size_t bytes) {
    const size_t was = at;
    at += (bytes + 255) / 256 * 256;
    return was;
  };
  l.flag = take((size_t)l.tiles * l.blocks * 4);
  l.gflag = take((size_t)l.groups * l.blocks * 4);
  l.seq = take((size_t)T * 4);
  l.agg_a = take((size_t)l.tiles * ch * 4);
  l.agg_h = take((size_t)l.tiles * ch * 4);
  l.group = take((size_t)l.groups * ch * 4);
  l.part = take(back ? (size_t)l.tiles * ch * 4 : 0);
  l.total = at;
  return l;
}

// ---- channels of a lane -------------------------------------------------------------------
template <int V> struct Ch { float f[V]; };
template <int V> __device__ __forceinline__ Ch<V> all(float x) {
  Ch<V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.f[i] = x;
  return r;
}
template <int V> __device__ __forceinline__ Ch<V> mul(Ch<V> a, const Ch<V>& b) {
  if constexpr (V == 2) mul2(a.f[0], a.f[1], b.f[0], b.f[1]);
  else a.f[0] *= b.f[0];
  return a;
}
template <int V> __device__ __forceinline__ Ch<V> add(Ch<V> a, const Ch<V>& b) {
  if constexpr (V == 2) add2(a.f[0], a.f[1], b.f[0], b.f[1]);
  else a.f[0] += b.f[0];
  return a;
}
template <int V> __device__ __forceinline__ Ch<V> fma(Ch<V> a, const Ch<V>& b, const Ch<V>& c) {
  if constexpr (V == 2) fma2(a.f[0], a.f[1], b.f[0], b.f[1], c.f[0], c.f[1]);
  else a.f[0] = fmaf(a.f[0], b.f[0], c.f[0]);
  return a;
}
template <int V> __device__ __forceinline__ Ch<V> neg(Ch<V> a) {
#pragma unroll
  for (int i = 0; i < V; ++i) a.f[i] = -a.f[i];
  return a;
}

// V elements of a row as one access.
template <typename T, int V> struct Pack;
template <typename T> struct Pack<T, 1> {
  using Raw = T;
  static __device__ __forceinline__ Ch<1> open(Raw r) { return {{to_f32(r)}}; }
  static __device__ __forceinline__ Raw close(const Ch<1>& c) { return from_f32<T>(c.f[0]); }
};
template <> struct Pack<float, 2> {
  using Raw = float2;
  static __device__ __forceinline__ Ch<2> open(Raw r) { return {{r.x, r.y}}; }
  static __device__ __forceinline__ Raw close(const Ch<2>& c) { return make_float2(c.f[0], c.f[1]); }
};
template <> struct Pack<__nv_bfloat16, 2> {
  using Raw = uint32_t;
  static __device__ __forceinline__ Ch<2> open(Raw r) {
    return {{__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u)}};
  }
  static __device__ __forceinline__ Raw close(const Ch<2>& c) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(c.f[0], c.f[1]);
    return *reinterpret_cast<const uint32_t*>(&b);
  }
};
template <typename T, int V> __device__ __forceinline__ typename Pack<T, V>::Raw load(const T* p) {
  return *reinterpret_cast<const typename Pack<T, V>::Raw*>(p);
}
template <typename T, int V> __device__ __forceinline__ void store(T* p, const Ch<V>& c) {
  *reinterpret_cast<typename Pack<T, V>::Raw*>(p) = Pack<T, V>::close(c);
}
// What other tiles write while this one runs is read past the L1.
template <int V> __device__ __forceinline__ Ch<V> load_shared_state(const float* p) {
  if constexpr (V == 2) {
    const float2 r = __ldcg(reinterpret_cast<const float2*>(p));
    return {{r.x, r.y}};
  } else {
    return {{__ldcg(p)}};
  }
}

// ---- gates ----------------------------------------------------------------------------------
// e^-v, kept below 1e37, and sigmoid(v) = 1 / (1 + e^-v), so that both sigmoid(v) and e^-v sigmoid(v) =
// 1 - sigmoid(v) keep their leading digits at either end. bf16 inputs take the fast exponential and
// reciprocal, good to 2^-21 and |v| 2^-24: far below those inputs' own rounding, and what is fp32 of the
// results (states, dA_log) keeps 2^-19.
template <bool kFast, int V> __device__ __forceinline__ Ch<V> exp_neg(const Ch<V>& v) {
  Ch<V> e;
  if constexpr (kFast) e = mul(v, all<V>(-kLog2e));
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (kFast) asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.f[i]));
    else e.f[i] = expf(-v.f[i]);
    e.f[i] = e.f[i] > 1e37f ? 1e37f : e.f[i];  // NaN stays
  }
  return e;
}
template <bool kFast, int V> __device__ __forceinline__ Ch<V> one_over(Ch<V> e) {  // 1 / (1 + e)
  e = add(e, all<V>(1.f));
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (kFast) asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.f[i]));
    else e.f[i] = 1.f / e.f[i];
  }
  return e;
}
template <bool kFast, int V> __device__ __forceinline__ Ch<V> sigmoid(const Ch<V>& v) {
  return one_over<kFast>(exp_neg<kFast>(v));
}

// Decay rates of a lane's channels, -exp(A_log), finite.
template <int V> __device__ __forceinline__ Ch<V> rates(const float* a_log, int c, int ch) {
  Ch<V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.f[i] = c + i < ch ? ssm_rate(a_log[c + i]) : 0.f;
  return r;
}

template <bool kFast, int V> __device__ __forceinline__ Ch<V> decay(const Ch<V>& g) {  // e^g
  Ch<V> a;
  if constexpr (kFast) {
    a = mul(g, all<V>(kLog2e));
#pragma unroll
    for (int i = 0; i < V; ++i) asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a.f[i]));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) a.f[i] = expf(g.f[i]);
  }
  return a;
}

// 1 - a^2 of a = e^g, g <= 0: above -0.175 the series of -expm1(2 g) (its next term is 2^-26 of it there),
// below it the difference, which has lost at most two bits.
template <int V> __device__ __forceinline__ Ch<V> loss(const Ch<V>& g, const Ch<V>& a) {
  const Ch<V> z = add(g, g);
  Ch<V> p = fma(z, all<V>(1.f / 5040.f), all<V>(1.f / 720.f));
  p = fma(p, z, all<V>(1.f / 120.f));
  p = fma(p, z, all<V>(1.f / 24.f));
  p = fma(p, z, all<V>(1.f / 6.f));
  p = fma(p, z, all<V>(0.5f));
  p = fma(p, z, all<V>(1.f));
  p = mul(p, neg(z));
  Ch<V> d = fma(neg(a), a, all<V>(1.f));
#pragma unroll
  for (int i = 0; i < V; ++i) d.f[i] = z.f[i] > -0.35f ? p.f[i] : d.f[i];
  return d;
}

template <bool kFast> __device__ __forceinline__ float root(float w) {
  if constexpr (kFast) {
    asm("sqrt.approx.ftz.f32 %0, %0;" : "+f"(w));
    return w;
  } else {
    return sqrtf(w);
  }
}
template <bool kFast, int V> __device__ __forceinline__ Ch<V> root(Ch<V> w) {
#pragma unroll
  for (int i = 0; i < V; ++i) w.f[i] = root<kFast>(w.f[i]);
  return w;
}

// ---- planning -------------------------------------------------------------------------------
// The sequence of each row (-1: none that is valid; the last one that holds it where lengths run
// backwards), flags cleared, rows of the sequences without tokens written: to <- from (zeros if null).
__global__ void __launch_bounds__(1024)
gated_plan_kernel(const int32_t* __restrict__ cu, const int32_t* __restrict__ idx, int N, int64_t T,
                  int64_t num_slots, WsHeader* hdr, int32_t* __restrict__ seq, uint32_t* __restrict__ flags,
                  int64_t num_flags, const float* from, float* to, int ch, bool zero_bad) {
  __shared__ int s_seq[kPlanRows];
  const int tid = threadIdx.x;
  if (blockIdx.x == 0) {
    check_all(&hdr->status, cu, idx, N, T, T, idx ? num_slots : 0);
    if (tid == 0) {
      hdr->next_item = 0;
      hdr->num_entries = 0;
    }
  }
  for (int64_t i = blockIdx.x * 1024ll + tid; i < num_flags; i += gridDim.x * 1024ll) flags[i] = 0;
  for (int64_t t0 = (int64_t)blockIdx.x * kPlanRows; t0 < T; t0 += (int64_t)gridDim.x * kPlanRows) {
    s_seq[tid] = -1;
    __syncthreads();
    for (int base = 0; base < N; base += 1024) {
      const int n = base + tid;
      int64_t a = 0, b = 0;
      bool hit = n < N && seq_bounds(cu, n, T, &a, &b) && a < t0 + kPlanRows && b > t0 && a < b;
      if (hit && idx) hit = resolve_slot(idx, n, num_slots) >= 0;
      unsigned m = __ballot_sync(0xffffffffu, hit);
      while (m) {
        const int src = __ffs(m) - 1;
        m &= m - 1;
        const int64_t sa = __shfl_sync(0xffffffffu, a, src), sb = __shfl_sync(0xffffffffu, b, src);
        const int sn = __shfl_sync(0xffffffffu, n, src);
        const int lo = (int)(sa > t0 ? sa - t0 : 0), hi = (int)(sb < t0 + kPlanRows ? sb - t0 : kPlanRows);
        for (int i = lo + (tid & 31); i < hi; i += 32) atomicMax(&s_seq[i], sn);
      }
    }
    __syncthreads();
    if (t0 + tid < T) seq[t0 + tid] = s_seq[tid];
    __syncthreads();
  }
  if (!to) return;
  for (int64_t n = blockIdx.x * 32ll + (tid >> 5); n < N; n += gridDim.x * 32ll) {
    int64_t a, b;
    const bool ok = seq_bounds(cu, (int)n, T, &a, &b);
    if (ok ? a != b : !zero_bad) continue;
    for (int c = tid & 31; c < ch; c += 32) to[n * ch + c] = ok && from ? from[n * ch + c] : 0.f;
  }
}

struct Plan {
  const int32_t* seq;
  uint32_t *flag, *gflag;
  float *agg_a, *agg_h, *group;
  int64_t tiles;
  int32_t blocks;
};

// ---- waits between tiles --------------------------------------------------------------------
__device__ __forceinline__ uint32_t load_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void store_release(uint32_t* p, uint32_t v) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
// Waits until *p is set, or until another tile has given up, or for limit_ns; 0 if it gave up.
__device__ __noinline__ uint32_t wait_flag_slow(const uint32_t* p, WsHeader* hdr, uint64_t limit_ns) {
  const uint64_t t0 = tc::globaltimer_ns();
  for (;;) {
    for (int i = 0; i < 64; ++i) {
      const uint32_t v = load_acquire(p);
      if (v) return v;
    }
    if (load_acquire(&hdr->num_entries)) return 0;
    if (tc::globaltimer_ns() - t0 > limit_ns) {
      raise_status(&hdr->status, KDA_DEVICE_PIPE_TIMEOUT);
      store_release(&hdr->num_entries, 1);
      return 0;
    }
  }
}
__device__ __forceinline__ uint32_t wait_flag(const uint32_t* p, WsHeader* hdr, uint64_t limit_ns) {
  const uint32_t v = load_acquire(p);
  return v ? v : wait_flag_slow(p, hdr, limit_ns);
}

// What is shared by the warps of a tile: each warp's (A, H) and whether a sequence begins in it, and
// those of the tiles before it in its group.
template <int V> struct Shared {
  Ch<V> a[kWarps][32], h[kWarps][32];
  Ch<V> ga[kGroup][32], gh[kGroup][32];
  uint32_t cut[kWarps], gcut[kGroup];
  int64_t tile;
};

template <int V>
__device__ __forceinline__ void fold(Ch<V>& h, const Ch<V>& A, const Ch<V>& H, bool cut) {
  const Ch<V> n = fma(A, h, H);
#pragma unroll
  for (int i = 0; i < V; ++i) h.f[i] = cut ? H.f[i] : n.f[i];
}

// The state that reaches tile `pos` (counted in the order of the pass) of channel block cb, of the
// channels of this lane, for warp `rank` of it (warps counted in that order too).
template <int V>
__device__ __forceinline__ Ch<V> enter(Shared<V>& s, const Plan& p, int64_t pos, int cb, int c, int ch,
                                       int warp, int lane, int rank, WsHeader* hdr, uint64_t limit_ns) {
  const int before = (int)(pos % kGroup);
  const int64_t g = pos / kGroup, first = g * kGroup;
  const bool in = c < ch;
  if (warp == 0) {  // the whole tile's
    Ch<V> A = s.a[0][lane], H = s.h[0][lane];
    // warps in the order of the pass: rank 0 is stored first
    uint32_t cut = s.cut[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      fold(H, s.a[w][lane], s.h[w][lane], s.cut[w] != 0);
      A = mul(A, s.a[w][lane]);
      cut |= s.cut[w];
    }
    if (before < kGroup - 1 && pos + 1 < p.tiles) {
      if (in) {
        store<float, V>(p.agg_a + pos * ch + c, A);
        store<float, V>(p.agg_h + pos * ch + c, H);
      }
      __syncwarp();
      if (lane == 0) {
        __threadfence();
        store_release(p.flag + pos * p.blocks + cb, cut ? 2u : 1u);
      }
    }
    s.ga[before][lane] = A;
    s.gh[before][lane] = H;
    if (lane == 0) s.gcut[before] = cut;
  }
  for (int j = warp; j < before; j += kWarps) {
    uint32_t v = 0;
    if (lane == 0) v = wait_flag(p.flag + (first + j) * p.blocks + cb, hdr, limit_ns);
    v = __shfl_sync(0xffffffffu, v, 0);
    if (in) {
      s.ga[j][lane] = load_shared_state<V>(p.agg_a + (first + j) * ch + c);
      s.gh[j][lane] = load_shared_state<V>(p.agg_h + (first + j) * ch + c);
    }
    if (lane == 0) s.gcut[j] = v == 2;
  }
  Ch<V> h = all<V>(0.f);
  if (g > 0) {
    if (lane == 0) wait_flag(p.gflag + g * p.blocks + cb, hdr, limit_ns);
    __syncwarp();
    if (in) h = load_shared_state<V>(p.group + g * ch + c);
  }
  __syncthreads();
  for (int j = 0; j < before; ++j) fold(h, s.ga[j][lane], s.gh[j][lane], s.gcut[j] != 0);
  if (warp == 0 && before == kGroup - 1 && pos + 1 < p.tiles) {
    Ch<V> n = h;
    fold(n, s.ga[before][lane], s.gh[before][lane], s.gcut[before] != 0);
    if (in) store<float, V>(p.group + (g + 1) * ch + c, n);
    __syncwarp();
    if (lane == 0) {
      __threadfence();
      store_release(p.gflag + (g + 1) * p.blocks + cb, 1u);
    }
  }
  for (int w = 0; w < rank; ++w) fold(h, s.a[w][lane], s.h[w][lane], s.cut[w] != 0);
  return h;
}

// Bits of a warp's S rows: valid ones, first and last ones of a sequence; lane j holds row j's sequence.
struct Rows {
  uint32_t valid, first, last;
  int seq;
};
template <int S>
__device__ __forceinline__ Rows rows_of(const int32_t* seq, int64_t t0, int64_t T, int lane) {
  Rows r;
  const int64_t t = t0 + lane;
  r.seq = lane < S && t < T ? seq[t] : -1;
  const int before = lane < S && t < T && t > 0 ? seq[t - 1] : -1;
  const int after = lane < S && t + 1 < T ? seq[t + 1] : -1;
  r.valid = __ballot_sync(0xffffffffu, r.seq >= 0);
  r.first = __ballot_sync(0xffffffffu, r.seq >= 0 && before != r.seq);
  r.last = __ballot_sync(0xffffffffu, r.seq >= 0 && after != r.seq);
  return r;
}

// ---- forward --------------------------------------------------------------------------------
template <typename T, int V, bool kGate, int S>
__global__ void __launch_bounds__(kThreads, 2)
gated_scan_kernel(const T* __restrict__ x, int64_t x_pitch, const T* __restrict__ r, int64_t r_pitch,
                  const T* __restrict__ ig, int64_t i_pitch, const float* __restrict__ a_log,
                  const float* state, const int32_t* __restrict__ idx, int64_t num_slots, int64_t stride,
                  float* final_state, T* __restrict__ y, float* __restrict__ carries, Plan plan, WsHeader* hdr,
                  int64_t total, int ch, uint64_t limit_ns) {
  constexpr bool kFast = sizeof(T) == 2;
  using P = Pack<T, V>;
  __shared__ Shared<V> s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) s.tile = atomicAdd(&hdr->next_item, 1u);
  __syncthreads();
  const int64_t k = s.tile / plan.blocks;
  const int cb = (int)(s.tile % plan.blocks);
  const int64_t t0 = (k * kWarps + warp) * S;
  const int c = (cb * 32 + lane) * V;
  const bool in = c < ch;

  typename P::Raw xr[S], rr[S], ir[S];
#pragma unroll
  for (int j = 0; j < S; ++j) {
    const bool ok = in && t0 + j < total;
    xr[j] = ok ? load<T, V>(x + (t0 + j) * x_pitch + c) : P::close(all<V>(0.f));
    rr[j] = ok ? load<T, V>(r + (t0 + j) * r_pitch + c) : P::close(all<V>(0.f));
    if (kGate) ir[j] = ok ? load<T, V>(ig + (t0 + j) * i_pitch + c) : P::close(all<V>(0.f));
  }
  const Ch<V> rate = rates<V>(a_log, c, ch);
  const Rows rows = rows_of<S>(plan.seq, t0, total, lane);

  Ch<V> a[S], b[S];
  Ch<V> A = all<V>(1.f), H = all<V>(0.f);
#pragma unroll
  for (int j = 0; j < S; ++j) {
    const Ch<V> g = mul(rate, sigmoid<kFast>(P::open(rr[j])));
    a[j] = decay<kFast>(g);
    b[j] = mul(root<kFast>(loss(g, a[j])), P::open(xr[j]));
    if (kGate) b[j] = mul(b[j], sigmoid<kFast>(P::open(ir[j])));
    if ((rows.first >> j) & 1) {  // the sequence's own state instead of what came before
      const int n = __shfl_sync(0xffffffffu, rows.seq, j);
      const int64_t slot = idx ? resolve_slot(idx, n, num_slots) : n;
      Ch<V> h0 = all<V>(0.f);
      if (state && in && KDA_CHECK(slot >= 0)) h0 = Pack<float, V>::open(load<float, V>(state + slot * stride + c));
      b[j] = fma(a[j], h0, b[j]);
      H = b[j];
    } else {
      H = fma(a[j], H, b[j]);
    }
    A = mul(A, a[j]);
  }
  s.a[warp][lane] = A;
  s.h[warp][lane] = H;
  if (lane == 0) s.cut[warp] = rows.first != 0;
  __syncthreads();
  Ch<V> h = enter(s, plan, k, cb, c, ch, warp, lane, warp, hdr, limit_ns);
  if (carries && t0 % KDA_GATED_CARRY_ROWS == 0 && t0 < total && in)
    store<float, V>(carries + t0 / KDA_GATED_CARRY_ROWS * ch + c, h);
#pragma unroll
  for (int j = 0; j < S; ++j) {
    if ((rows.first >> j) & 1) h = b[j];
    else h = fma(a[j], h, b[j]);
    if (((rows.valid >> j) & 1) && in && KDA_CHECK(t0 + j < total && c + V <= ch))
      store<T, V>(y + (t0 + j) * ch + c, h);
    if (((rows.last >> j) & 1) && final_state) {
      const int n = __shfl_sync(0xffffffffu, rows.seq, j);
      const int64_t slot = idx ? resolve_slot(idx, n, num_slots) : n;
      if (in && KDA_CHECK(slot >= 0)) store<float, V>(final_state + slot * stride + c, h);
    }
  }
  KDA_DEBUG_FOLD(&hdr->status);
}

// ---- backward -------------------------------------------------------------------------------
template <typename T, int V, bool kGate, int S>
__global__ void __launch_bounds__(kThreads, 2)
gated_back_kernel(const T* __restrict__ dy, int64_t dy_pitch, const T* __restrict__ x, int64_t x_pitch,
                  const T* __restrict__ r, int64_t r_pitch, const T* __restrict__ ig, int64_t i_pitch,
                  const float* __restrict__ a_log, const float* __restrict__ carries,
                  const float* __restrict__ state, const float* __restrict__ dfinal, T* __restrict__ dx,
                  T* __restrict__ dr, T* __restrict__ di, float* __restrict__ dstate, float* __restrict__ part,
                  Plan plan, WsHeader* hdr, int64_t total, int ch, uint64_t limit_ns) {
  constexpr bool kFast = sizeof(T) == 2;
  static_assert(S * kWarps == KDA_GATED_CARRY_ROWS, "a tile starts where a carry was left");
  using P = Pack<T, V>;
  __shared__ Shared<V> s;
  __shared__ Ch<V> s_fa[kWarps][32], s_fh[kWarps][32];  // the state's own (A, H)
  __shared__ uint32_t s_first[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) s.tile = atomicAdd(&hdr->next_item, 1u);
  __syncthreads();
  const int64_t pos = s.tile / plan.blocks;          // tiles from the last one on
  const int64_t k = plan.tiles - 1 - pos;
  const int cb = (int)(s.tile % plan.blocks);
  const int64_t t0 = (k * kWarps + warp) * S;
  const int c = (cb * 32 + lane) * V;
  const bool in = c < ch;

  typename P::Raw xr[S], rr[S], ir[S], gr[S];
#pragma unroll
  for (int j = 0; j < S; ++j) {
    const bool ok = in && t0 + j < total;
    xr[j] = ok ? load<T, V>(x + (t0 + j) * x_pitch + c) : P::close(all<V>(0.f));
    rr[j] = ok ? load<T, V>(r + (t0 + j) * r_pitch + c) : P::close(all<V>(0.f));
    if (kGate) ir[j] = ok ? load<T, V>(ig + (t0 + j) * i_pitch + c) : P::close(all<V>(0.f));
    gr[j] = ok ? load<T, V>(dy + (t0 + j) * dy_pitch + c) : P::close(all<V>(0.f));
  }
  const Ch<V> rate = rates<V>(a_log, c, ch);
  const Rows rows = rows_of<S>(plan.seq, t0, total, lane);
  Ch<V> h = in ? Pack<float, V>::open(load<float, V>(carries + k * ch + c)) : all<V>(0.f);

  // the rows' decays and the state's (A, H), then what they do to e, from the last row to the first
  Ch<V> a[S], er[S], ei[S], hp[S];
  Ch<V> A = all<V>(1.f), H = all<V>(0.f);
#pragma unroll
  for (int j = 0; j < S; ++j) {
    er[j] = exp_neg<kFast>(P::open(rr[j]));
    const Ch<V> g = mul(rate, one_over<kFast>(er[j]));
    a[j] = decay<kFast>(g);
    Ch<V> b = mul(root<kFast>(loss(g, a[j])), P::open(xr[j]));
    if (kGate) {
      ei[j] = exp_neg<kFast>(P::open(ir[j]));
      b = mul(b, one_over<kFast>(ei[j]));
    }
    if ((rows.first >> j) & 1) {
      const int n = __shfl_sync(0xffffffffu, rows.seq, j);
      Ch<V> h0 = all<V>(0.f);
      if (state && in) h0 = Pack<float, V>::open(load<float, V>(state + (int64_t)n * ch + c));
      hp[j] = h0;
      H = fma(a[j], h0, b);
    } else {
      hp[j] = H;               // within the warp; what reaches it is added below
      H = fma(a[j], H, b);
    }
    A = mul(A, a[j]);
  }
  s_fa[warp][lane] = A;
  s_fh[warp][lane] = H;
  if (lane == 0) s_first[warp] = rows.first != 0;
  Ch<V> E = all<V>(0.f);
#pragma unroll
  for (int j = S - 1; j >= 0; --j) {
    Ch<V> l = P::open(gr[j]);
    if ((rows.last >> j) & 1) {
      const int n = __shfl_sync(0xffffffffu, rows.seq, j);
      if (dfinal && in) l = add(l, Pack<float, V>::open(load<float, V>(dfinal + (int64_t)n * ch + c)));
    } else {
      l = add(l, E);
    }
    E = mul(a[j], l);
  }
  const int rank = kWarps - 1 - warp;
  s.a[rank][lane] = A;
  s.h[rank][lane] = E;
  if (lane == 0) s.cut[rank] = rows.last != 0;
  __syncthreads();
  Ch<V> e = enter(s, plan, pos, cb, c, ch, warp, lane, rank, hdr, limit_ns);
  for (int w = 0; w < warp; ++w) fold(h, s_fa[w][lane], s_fh[w][lane], s_first[w] != 0);
  {
    Ch<V> q = h;               // decayed from row to row until a sequence begins
#pragma unroll
    for (int j = 0; j < S; ++j) {
      if ((rows.first >> j) & 1) break;
      hp[j] = add(hp[j], q);
      q = mul(q, a[j]);
    }
  }
  Ch<V> sum = all<V>(0.f);
#pragma unroll
  for (int j = S - 1; j >= 0; --j) {
    const bool valid = (rows.valid >> j) & 1;
    Ch<V> l = P::open(gr[j]);
    if ((rows.last >> j) & 1) {
      const int n = __shfl_sync(0xffffffffu, rows.seq, j);
      if (dfinal && in) l = add(l, Pack<float, V>::open(load<float, V>(dfinal + (int64_t)n * ch + c)));
    } else {
      l = add(l, e);
    }
    e = mul(a[j], l);
    const Ch<V> sr = one_over<kFast>(er[j]), g = mul(rate, sr);
    const Ch<V> m = root<kFast>(loss(g, a[j]));
    Ch<V> q;
#pragma unroll
    for (int i = 0; i < V; ++i) q.f[i] = m.f[i] == 0.f ? 0.f : kFast ? __fdividef(g.f[i], m.f[i]) : g.f[i] / m.f[i];
    Ch<V> u = P::open(xr[j]), ml = mul(m, l), si;
    if (kGate) {
      si = one_over<kFast>(ei[j]);
      u = mul(u, si);
    }
    // p = e (g h_{t-1} - a (g / m) u)
    const Ch<V> p = mul(e, fma(g, hp[j], neg(mul(mul(a[j], q), u))));
    if (in && t0 + j < total && KDA_CHECK(c + V <= ch)) {
      const int64_t at = (t0 + j) * ch + c;
      const Ch<V> zero = all<V>(0.f);
      store<T, V>(dx + at, !valid ? zero : kGate ? mul(ml, si) : ml);
      store<T, V>(dr + at, valid ? mul(p, mul(er[j], sr)) : zero);
      if (kGate) store<T, V>(di + at, valid ? mul(mul(ml, u), mul(ei[j], si)) : zero);
    }
    if (valid) sum = add(sum, p);
    if (((rows.first >> j) & 1) && dstate) {
      const int n = __shfl_sync(0xffffffffu, rows.seq, j);
      if (in) store<float, V>(dstate + (int64_t)n * ch + c, e);
    }
  }
  __syncthreads();
  s.a[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && in) {
#pragma unroll
    for (int w = 1; w < kWarps; ++w) sum = add(sum, s.a[w][lane]);
    store<float, V>(part + k * ch + c, sum);
  }
  KDA_DEBUG_FOLD(&hdr->status);
}

// dA_log: the tiles' parts of a channel, added up in a fixed order.
__global__ void __launch_bounds__(256)
gated_sum_kernel(const float* __restrict__ part, int64_t tiles, int ch, float* __restrict__ da) {
  __shared__ float s[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float sum = 0.f;
  if (c < ch)
    for (int64_t k = warp; k < tiles; k += 8) sum += part[k * ch + c];
  s[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && c < ch) {
#pragma unroll
    for (int w = 1; w < 8; ++w) sum += s[w][lane];
    da[c] = sum;
  }
}

// ---- tokens ---------------------------------------------------------------------------------
// One token, or a few drafted ones, a row.
template <typename T, int V, bool kGate>
__global__ void __launch_bounds__(128)
gated_token_kernel(const T* __restrict__ x, int64_t x_pitch, const T* __restrict__ r, int64_t r_pitch,
                   const T* __restrict__ ig, int64_t i_pitch, const float* __restrict__ a_log,
                   const int32_t* __restrict__ cu, float* pool, const int32_t* __restrict__ idx,
                   int64_t num_slots, int64_t stride, T* __restrict__ y, uint32_t* status, int N,
                   int64_t total, int ch, float* __restrict__ cache, int64_t cache_pitch, int max_steps,
                   bool update_pool) {
  constexpr bool kFast = sizeof(T) == 2;
  using P = Pack<T, V>;
  if (blockIdx.x == 0 && blockIdx.y == 0) check_all(status, cu, idx, N, total, max_steps, num_slots);
  const int n = blockIdx.x;
  const int c = (blockIdx.y * 128 + threadIdx.x) * V;
  if (c >= ch) return;
  int64_t bos = n, eos = n + 1;
  if (cu && (!seq_bounds(cu, n, total, &bos, &eos) || eos - bos > max_steps)) return;
  const int64_t slot = idx ? resolve_slot(idx, n, num_slots) : (n < num_slots ? n : -1);
  if (slot < 0) return;
  float* so = pool + slot * stride + c;
  Ch<V> h = Pack<float, V>::open(load<float, V>(so));
  const Ch<V> rate = rates<V>(a_log, c, ch);
  for (int64_t t = bos; t < eos; ++t) {
    const typename P::Raw xr = load<T, V>(x + t * x_pitch + c), rr = load<T, V>(r + t * r_pitch + c);
    Ch<V> u = P::open(xr);
    if (kGate) u = mul(u, sigmoid<kFast>(P::open(load<T, V>(ig + t * i_pitch + c))));
    const Ch<V> g = mul(rate, sigmoid<kFast>(P::open(rr))), a = decay<kFast>(g);
    h = fma(a, h, mul(root<kFast>(loss(g, a)), u));
    if (KDA_CHECK(t >= 0 && t < total && c + V <= ch)) store<T, V>(y + t * ch + c, h);
    if (cache) store<float, V>(cache + n * cache_pitch + (t - bos) * ch + c, h);
  }
  if (update_pool) store<float, V>(so, h);
  KDA_DEBUG_FOLD(status);
}

// ---- launches -------------------------------------------------------------------------------
constexpr int kRows = 16;      // rows a warp, forward
constexpr int kBackRows = 8;   // and backward

bool pairs(const void* p, int64_t pitch, int size) {
  return !p || ((uintptr_t)p % (2 * size) == 0 && pitch % 2 == 0);
}

Plan plan_of(const Layout& l, uint8_t* ws) {
  Plan p;
  p.seq = reinterpret_cast<int32_t*>(ws + l.seq);
  p.flag = reinterpret_cast<uint32_t*>(ws + l.flag);
  p.gflag = reinterpret_cast<uint32_t*>(ws + l.gflag);
  p.agg_a = reinterpret_cast<float*>(ws + l.agg_a);
  p.agg_h = reinterpret_cast<float*>(ws + l.agg_h);
  p.group = reinterpret_cast<float*>(ws + l.group);
  p.tiles = l.tiles;
  p.blocks = l.blocks;
  return p;
}

cudaError_t launch_plan(const GatedArgs& a, const Layout& l, const float* from, float* to, bool zero_bad,
                        cudaStream_t st) {
  const int64_t most = 4ll * gpu_sms();
  int64_t blocks = (a.d.total_tokens + kPlanRows - 1) / kPlanRows;
  if (to) blocks = blocks > (a.d.num_seqs + 31) / 32 ? blocks : (a.d.num_seqs + 31) / 32;
  blocks = blocks < 1 ? 1 : blocks > most ? most : blocks;
  gated_plan_kernel<<<(unsigned)blocks, 1024, 0, st>>>(
      a.cu, a.idx, a.d.num_seqs, a.d.total_tokens, a.d.num_slots, reinterpret_cast<WsHeader*>(a.ws),
      reinterpret_cast<int32_t*>(a.ws + l.seq), reinterpret_cast<uint32_t*>(a.ws + l.flag),
      (int64_t)((l.seq - l.flag) / 4), from, to, a.d.channels, zero_bad);
  return cudaGetLastError();
}

template <typename T, int V, bool kGate>
cudaError_t run_scan(const GatedArgs& a, cudaStream_t st) {
  const Layout l = layout_of(a.d.total_tokens, a.d.channels, kRows * kWarps, V, false);
  const bool dense = !a.idx && a.state_out && a.state_out != a.state_in;
  cudaError_t e = launch_plan(a, l, a.state_in, dense ? a.state_out : nullptr, false, st);
  if (e != cudaSuccess || l.tiles == 0) return e;
  gated_scan_kernel<T, V, kGate, kRows><<<(unsigned)(l.tiles * l.blocks), kThreads, 0, st>>>(
      (const T*)a.x, a.d.x_pitch, (const T*)a.r, a.d.r_pitch, (const T*)a.i, a.d.i_pitch, a.a_log, a.state_in,
      a.idx, a.d.num_slots, a.slot_stride, a.state_out, (T*)a.y, a.carries, plan_of(l, a.ws),
      reinterpret_cast<WsHeader*>(a.ws), a.d.total_tokens, a.d.channels, pipeline_wait_limit_ns());
  return cudaGetLastError();
}

template <typename T, int V, bool kGate>
cudaError_t run_back(const GatedArgs& a, cudaStream_t st) {
  const Layout l = layout_of(a.d.total_tokens, a.d.channels, kBackRows * kWarps, V, true);
  cudaError_t e = launch_plan(a, l, a.dfinal, a.dstate, true, st);
  if (e != cudaSuccess) return e;
  float* part = reinterpret_cast<float*>(a.ws + l.part);
  if (l.tiles > 0) {
    gated_back_kernel<T, V, kGate, kBackRows><<<(unsigned)(l.tiles * l.blocks), kThreads, 0, st>>>(
        (const T*)a.dy, a.dy_pitch, (const T*)a.x, a.d.x_pitch, (const T*)a.r, a.d.r_pitch, (const T*)a.i,
        a.d.i_pitch, a.a_log, a.carries, a.state_in, a.dfinal, (T*)a.dx, (T*)a.dr, (T*)a.di, a.dstate, part,
        plan_of(l, a.ws), reinterpret_cast<WsHeader*>(a.ws), a.d.total_tokens, a.d.channels,
        pipeline_wait_limit_ns());
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  gated_sum_kernel<<<(unsigned)((a.d.channels + 31) / 32), 256, 0, st>>>(part, l.tiles, a.d.channels, a.da_log);
  return cudaGetLastError();
}

template <typename T, int V, bool kGate>
cudaError_t run_token(const GatedArgs& a, cudaStream_t st) {
  dim3 grid((unsigned)a.d.num_seqs, (unsigned)((a.d.channels + 128 * V - 1) / (128 * V)));
  gated_token_kernel<T, V, kGate><<<grid, 128, 0, st>>>(
      (const T*)a.x, a.d.x_pitch, (const T*)a.r, a.d.r_pitch, (const T*)a.i, a.d.i_pitch, a.a_log, a.cu,
      a.state_out, a.idx, a.d.num_slots, a.slot_stride, (T*)a.y, &reinterpret_cast<WsHeader*>(a.ws)->status,
      a.d.num_seqs, a.d.total_tokens, a.d.channels, a.cache, a.cache_pitch, a.max_steps, a.update_pool);
  return cudaGetLastError();
}

enum class Pass { kScan, kBack, kToken };

template <typename T, int V>
cudaError_t by_gate(const GatedArgs& a, cudaStream_t st, Pass pass) {
  switch (pass) {
    case Pass::kScan: return a.i ? run_scan<T, V, true>(a, st) : run_scan<T, V, false>(a, st);
    case Pass::kBack: return a.i ? run_back<T, V, true>(a, st) : run_back<T, V, false>(a, st);
    default: return a.i ? run_token<T, V, true>(a, st) : run_token<T, V, false>(a, st);
  }
}

// Two channels a lane where every row starts on a boundary of two elements, else one.
template <typename T>
cudaError_t by_type(const GatedArgs& a, cudaStream_t st, Pass pass) {
  const int e = sizeof(T);
  const int64_t ch = a.d.channels;
  const bool wide = ch % 2 == 0 && pairs(a.x, a.d.x_pitch, e) && pairs(a.r, a.d.r_pitch, e) &&
                    pairs(a.i, a.d.i_pitch, e) && pairs(a.dy, a.dy_pitch, e) && pairs(a.y, ch, e) &&
                    pairs(a.dx, ch, e) && pairs(a.dr, ch, e) && pairs(a.di, ch, e) &&
                    pairs(a.state_in, a.slot_stride, 4) && pairs(a.state_out, a.slot_stride, 4) &&
                    pairs(a.cache, a.cache_pitch, 4) && pairs(a.carries, ch, 4) && pairs(a.dfinal, ch, 4) &&
                    pairs(a.dstate, ch, 4);
  return wide ? by_gate<T, 2>(a, st, pass) : by_gate<T, 1>(a, st, pass);
}

cudaError_t launch(const GatedArgs& a, cudaStream_t st, Pass pass) {
  return a.d.dtype == KDA_BF16 ? by_type<__nv_bfloat16>(a, st, pass) : by_type<float>(a, st, pass);
}

}  // namespace

// One channel a lane is the form with the most channel blocks.
size_t gated_scan_workspace(const kda_gated_desc_t& d) {
  return layout_of(d.total_tokens, d.channels, kRows * kWarps, 1, false).total;
}
size_t gated_back_workspace(const kda_gated_desc_t& d) {
  return layout_of(d.total_tokens, d.channels, kBackRows * kWarps, 1, true).total;
}
bool gated_fits(const kda_gated_desc_t& d) {  // tiles are counted in 32 bits, by the smaller tile
  const Layout l = layout_of(d.total_tokens, d.channels, kBackRows * kWarps, 1, true);
  return l.tiles * l.blocks <= 0x7fffffffll;
}
cudaError_t launch_gated_scan(const GatedArgs& a, cudaStream_t st) { return launch(a, st, Pass::kScan); }
cudaError_t launch_gated_back(const GatedArgs& a, cudaStream_t st) { return launch(a, st, Pass::kBack); }
cudaError_t launch_gated_token(const GatedArgs& a, cudaStream_t st) { return launch(a, st, Pass::kToken); }

}  // namespace kda
