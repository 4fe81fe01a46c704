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
// Both passes are bound by HBM if their arithmetic (six special functions an element with an input gate, eleven
// backward, whose last step forms the gates again) hides behind it, so each reads its inputs once. The packed rows,
// whatever sequences they belong to, are cut into tiles of kWarps * S rows by 32 * V channels; a warp takes S rows of a
// tile, a lane V channels. What a run of rows does to the state is h -> A h + H, so
//   1. each warp forms a and m u of its rows, which it keeps in shared memory, and their (A, H);
//   2. the tile's (A, H) goes to global memory for the tiles after it, and the state before the tile is
//      put together from those of the tiles before it: the state at the start of its group of kGroup
//      tiles, then the tiles of the group in order;
//   3. each warp runs through its rows again, from shared memory, and writes them.
// Ten warps a CTA: eight run; one takes tiles by a counter (earlier rows first, so a tile waits only for tiles that
// are done or in work), has their rows fetched by TMA and publishes the tile's run; one puts the state together. The
// eight are a tile ahead of themselves: step 1 of the next tile comes before step 3 of this one, so that the trip to
// other tiles' runs is behind arithmetic. The state at a group's start comes from the group before it, one
// wait for kGroup tiles. What tiles tell each other is valid when it is seen: A's place, or a tag beside the
// state, holds a pattern no result has until its 8 bytes are written at once, so a wait is one trip to the
// L2 and no fence. The order of all sums is fixed, whichever tile comes first: results are bit-identical
// from run to run. A sequence's first row starts from its own state, and no product carries the state before
// it (which may be no number).
//
// The backward pass runs over the tiles from the last to the first, e in the place of h. It needs
// h_{t-1} as well; the forward pass left the state before each KDA_GATED_CARRY_ROWS rows for it. Its gates are formed
// again from x, r and i, which it reads anyway (a and m u, left by the forward pass, would be 8 bytes an element more
// to write and to read).
//
// Measured: forward, 32768 x 4096 bf16 (16 sequences, input gate, states of a pool) 269 us, 4.0 TB/s, 59 % of the
// copy rate; 177 with a state that waits for nobody and gates of two multiplications, 245 with the gates as they
// are, so the special functions bound it, then the state's trips. Groups of 4 tiles 267 but slower where channels
// are few, 16: 279. Four warps a CTA 353 us, eight rows a warp 416, two states put together in turns 324. Backward,
// 16384 x 4096 bf16: 305 us, 3.1 TB/s; its special functions alone take 160 at 16 a cycle and SM, and with 57 % of
// the issue slots and 36 % of HBM in use what is left is latency, of 20 warps an SM. Both in fp32, 65536 x 320, one
// sequence: 265 us.
#include <cudaTypedefs.h>

#include <algorithm>
#include <type_traits>

#include "kda_internal.cuh"
#include "tc_ptx.cuh"

namespace kda {
namespace {

KDA_DEBUG_FLAG_DEFINE();

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kScanCtas = 2, kBackCtas = 2;   // CTAs an SM
constexpr int kGroup = 8;                     // tiles between states that are told
constexpr int kPlanRows = 1024;   // rows a block of the planning kernel
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kUnset = 0xffffffffu;
constexpr int kInfos = 8;         // tiles of a CTA from the ones taken ahead back to the one whose sums are added up

// Workspace behind the header: each tile's (A, H) and each group's (state, tag) of all channels, which the
// planning kernel sets to kUnset; the sequence of each row; the backward pass's parts of dA_log.
struct Layout {
  int64_t tiles, groups;
  int32_t blocks;               // channel blocks
  size_t agg, group, seq, part, total;
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
  l.agg = take((size_t)l.tiles * ch * 8);
  l.group = take((size_t)l.groups * ch * 8);
  l.seq = take((size_t)T * 4);
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
// ---- gates ----------------------------------------------------------------------------------
// e^-v and sigmoid(v) = 1 / (1 + e^-v). Where e^-v is kept at 3e38 at most, e^-v sigmoid(v) = 1 - sigmoid(v) has its
// leading digits at either end, unless sigmoid(v) is below 2^-126 and counts as 0: such a gate has no derivative (and
// the Newton step has no infinity to meet). bf16 inputs take the fast exponential
// and reciprocal, good to 2^-21 and |v| 2^-24: far below those inputs' own rounding, and what is fp32 of the results
// (states, dA_log) keeps 2^-18 of a step's terms for |v| up to 8. fp32 inputs take CUDA's exponential and a Newton step
// behind the reciprocal.
template <bool kFast, bool kBounded, int V> __device__ __forceinline__ Ch<V> exp_neg(const Ch<V>& v) {
  Ch<V> e;
  if constexpr (kFast) e = mul(v, all<V>(-kLog2e));
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (kFast) asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.f[i]));
    else e.f[i] = expf(-v.f[i]);
    if constexpr (kBounded) asm("min.NaN.f32 %0, %0, 0f7f61b1e6;" : "+f"(e.f[i]));  // 3e38; NaN stays
  }
  return e;
}
template <bool kFast, int V> __device__ __forceinline__ Ch<V> one_over(Ch<V> e) {  // 1 / (1 + e)
  e = add(e, all<V>(1.f));
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e.f[i]));
    e.f[i] = kFast ? r : fmaf(r, fmaf(-e.f[i], r, 1.f), r);
  }
  return e;
}
template <bool kFast, int V> __device__ __forceinline__ Ch<V> sigmoid(const Ch<V>& v) {
  return one_over<kFast>(exp_neg<kFast, !kFast>(v));
}

// Decay rates of a lane's channels, -exp(A_log), finite.
template <int V> __device__ __forceinline__ Ch<V> rates(const float* a_log, int c, int ch) {
  Ch<V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.f[i] = c + i < ch ? ssm_rate(a_log[c + i]) : 0.f;
  return r;
}

// a = e^g and a^2 - 1 of a log-decay g <= 0. Above -0.175 by the series of e = e^g - 1 (its next term is 2^-27
// of it there): a = 1 + e is rounded once, which long memories need (a decay off by 2^-22, as the fast
// exponential's, is a state off by that times the tokens it remembers), and a^2 - 1 = e (2 + e) keeps its
// digits. Below it the difference, which has lost at most two bits. (The backward pass has a already.)
constexpr float kSeries = -0.175f;
template <int V> __device__ __forceinline__ Ch<V> series(const Ch<V>& g) {
  Ch<V> p = fma(g, all<V>(1.f / 720.f), all<V>(1.f / 120.f));
  p = fma(p, g, all<V>(1.f / 24.f));
  p = fma(p, g, all<V>(1.f / 6.f));
  p = fma(p, g, all<V>(0.5f));
  p = fma(p, g, all<V>(1.f));
  return mul(p, g);
}
template <int V> __device__ __forceinline__ Ch<V> lost(const Ch<V>& g, const Ch<V>& e, const Ch<V>& a) {
  const Ch<V> near = mul(e, add(e, all<V>(2.f)));
  Ch<V> w = fma(a, a, all<V>(-1.f));
#pragma unroll
  for (int i = 0; i < V; ++i) w.f[i] = g.f[i] > kSeries ? near.f[i] : w.f[i];
  return w;
}
template <bool kFast, int V> __device__ __forceinline__ Ch<V> decay(const Ch<V>& g, Ch<V>& w) {
  Ch<V> a;
  if constexpr (kFast) {
    a = mul(g, all<V>(kLog2e));
#pragma unroll
    for (int i = 0; i < V; ++i) asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a.f[i]));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) a.f[i] = expf(g.f[i]);
  }
  const Ch<V> e = series(g), near = add(e, all<V>(1.f));
  w = lost(g, e, a);
#pragma unroll
  for (int i = 0; i < V; ++i) a.f[i] = g.f[i] > kSeries ? near.f[i] : a.f[i];
  return a;
}

// sqrt(-w), to 2^-23
template <int V> __device__ __forceinline__ Ch<V> root(Ch<V> w) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    w.f[i] = -w.f[i];
    asm("sqrt.approx.ftz.f32 %0, %0;" : "+f"(w.f[i]));
  }
  return w;
}
// -1 over sqrt(-w) and sqrt(-w), to 2^-22; both 0 where that is.
template <int V> __device__ __forceinline__ void over_root(const Ch<V>& w, Ch<V>& k, Ch<V>& m) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(k.f[i]) : "f"(-w.f[i]));
    k.f[i] = w.f[i] > -1e-37f ? 0.f : -k.f[i];
  }
  m = mul(w, k);
}

// ---- planning -------------------------------------------------------------------------------
// The sequence of each row (-1: none that is valid; the last one that holds it where lengths run
// backwards), what tiles tell each other unset, rows of the sequences without tokens written: to <- from
// (zeros if null).
__global__ void __launch_bounds__(1024)
gated_plan_kernel(const int32_t* __restrict__ cu, const int32_t* __restrict__ idx, int N, int64_t T,
                  int64_t num_slots, WsHeader* hdr, int32_t* __restrict__ seq, uint4* __restrict__ unset,
                  int64_t num_unset, const float* from, float* to, int ch, bool zero_bad) {
  __shared__ int s_seq[kPlanRows];
  const int tid = threadIdx.x;
  tc::grid_dep_launch_dependents();
  if (blockIdx.x == 0) {
    check_all(&hdr->status, cu, idx, N, T, T, idx ? num_slots : 0);
    if (tid == 0) {
      hdr->next_item = 0;
      hdr->num_entries = 0;
    }
  }
  for (int64_t i = blockIdx.x * 1024ll + tid; i < num_unset; i += gridDim.x * 1024ll)
    unset[i] = make_uint4(kUnset, kUnset, kUnset, kUnset);
  for (int64_t t0 = (int64_t)blockIdx.x * kPlanRows; t0 < T; t0 += (int64_t)gridDim.x * kPlanRows) {
    sequences_of<kPlanRows>(s_seq, cu, idx, num_slots, N, T, t0);
    if (t0 + tid < T) seq[t0 + tid] = s_seq[tid];
    __syncthreads();
  }
  if (to) rows_without_tokens(cu, N, T, from, to, ch, zero_bad);
}

struct Plan {
  const int32_t* seq;
  float *agg, *group;
  int64_t tiles;
  int32_t blocks;
  uint32_t items;      // tiles of all channel blocks
};

// ---- what tiles tell each other ---------------------------------------------------------------
// Two 32-bit values of each of a lane's channels, 8 bytes a channel, each written and read at once.
template <int V> struct Pair { float a[V], h[V]; };
template <int V> __device__ __forceinline__ void tell(float* at, const Pair<V>& p) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    asm volatile("{\n .reg .b64 t;\n mov.b64 t, {%1, %2};\n st.relaxed.gpu.global.b64 [%0], t;\n}\n" ::"l"(at + 2 * i),
                 "f"(p.a[i]), "f"(p.h[i])
                 : "memory");
  }
}
template <int V> __device__ __forceinline__ bool hear(const float* at, Pair<V>& p) {
  bool set = true;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    asm volatile("{\n .reg .b64 t;\n ld.relaxed.gpu.global.b64 t, [%2];\n mov.b64 {%0, %1}, t;\n}\n"
                 : "=f"(p.a[i]), "=f"(p.h[i])
                 : "l"(at + 2 * i)
                 : "memory");
    set = set && __float_as_uint(p.a[i]) != kUnset;
  }
  return set;
}
// Whether a warp that waits for other tiles should go on: until one of them has given up, or for limit_ns. It asks
// at each 64th try, which is nothing beside seconds; where the limit is shorter than 64 trips take, at each.
constexpr uint64_t kTriesNs = 100000;
struct Patience {
  uint64_t t0 = 0;
  int tries = 0;
  __device__ __forceinline__ bool more(WsHeader* hdr, uint64_t limit_ns) {
    if (++tries % 64 && limit_ns >= kTriesNs) return true;
    if (*(volatile uint32_t*)&hdr->num_entries) return false;
    const uint64_t now = __shfl_sync(0xffffffffu, tc::globaltimer_ns(), 0);
    if (t0 == 0) t0 = now;
    if (now - t0 <= limit_ns) return true;
    raise_status(&hdr->status, KDA_DEVICE_PIPE_TIMEOUT);
    atomicExch(&hdr->num_entries, 1u);
    return false;
  }
};

// h <- A h + H; a run in which a sequence begins has A = -1 and forgets h.
template <int V> __device__ __forceinline__ void fold(Ch<V>& h, const Ch<V>& A, const Ch<V>& H) {
  const Ch<V> n = fma(A, h, H);
#pragma unroll
  for (int i = 0; i < V; ++i) h.f[i] = A.f[i] < 0.f ? H.f[i] : n.f[i];
}
// The run (A, H) followed by (B, G), as one in (A, H).
template <int V> __device__ __forceinline__ void join(Ch<V>& A, Ch<V>& H, const Ch<V>& B, const Ch<V>& G) {
  fold(H, B, G);
  const Ch<V> n = mul(A, B);
#pragma unroll
  for (int i = 0; i < V; ++i) A.f[i] = A.f[i] < 0.f || B.f[i] < 0.f ? -1.f : n.f[i];
}

// What the warps of a CTA share. Tiles of a CTA are counted by `n`.
struct Info {
  int64_t t0;        // the tile's first row; -1: no tile
  int64_t pos;       // its number in the order of the pass
  int c0;            // its first channel
  int plain;         // its rows, and one on either side, are of one sequence, its channels all there
};
template <int V> struct Shared {
  Ch<V> a[2][kWarps][32], h[2][kWarps][32];   // each warp's run of tile n & 1, in the order of the pass
  Ch<V> carry[2][kWarps][32];                 // the state that reaches it
  Info info[kInfos];                          // of tile n % kInfos
  uint64_t full;                              // the next tile's rows are there
};
// Named barriers, two each, by n & 1: the warps' runs of a tile are there (for the warp that fetches), the
// tile's run is published (for the one that carries), the state that reaches the warps is there (for them).
enum : uint32_t { kRan = 1, kPublished = 3, kCarried = 5 };
constexpr uint32_t kAll = kThreads + 64;   // with the warp that fetches and the one that carries
constexpr uint32_t kMeet = kThreads + 32;    // the warps that run and one of the others
__device__ __forceinline__ void bar_arrive(uint32_t id, uint32_t threads = kMeet) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_sync(uint32_t id, uint32_t threads = kMeet) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// The warp that takes tiles: the counter and the rows' sequences are asked for ahead of where they are needed.
template <int V, int S, bool kBack> struct Taker {
  static constexpr int kRowsTile = kWarps * S, kLoads = (kRowsTile + 2 + 31) / 32;
  uint32_t item, next;
  int seq[kLoads];
  __device__ __forceinline__ int64_t first_row(const Plan& p) const {
    const int64_t pos = item / p.blocks;
    return (kBack ? p.tiles - 1 - pos : pos) * kRowsTile;
  }
  __device__ __forceinline__ void start(WsHeader* hdr, int lane) {
    next = lane == 0 ? atomicAdd(&hdr->next_item, 1u) : 0u;
  }
  // the next tile, and the sequences of its rows and of one on either side, on their way
  __device__ __forceinline__ void ask(const Plan& p, WsHeader* hdr, int64_t total, int lane) {
    item = __shfl_sync(0xffffffffu, next, 0);
    next = lane == 0 ? atomicAdd(&hdr->next_item, 1u) : 0u;
    if (item >= p.items) return;
    const int64_t t0 = first_row(p) - 1 + lane;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int64_t t = t0 + j * 32;
      seq[j] = -1;
      if (j * 32 + lane >= kRowsTile + 2) seq[j] = -2;    // none of the rows asked for
      else if (t >= 0 && t < total) seq[j] = p.seq[t];
    }
  }
  __device__ __forceinline__ void tell_all(Info& to, const Plan& p, int64_t total, int ch, int lane) const {
    Info o;
    o.t0 = -1;
    o.pos = item / p.blocks;
    o.c0 = (int)(item % p.blocks) * 32 * V;
    o.plain = 0;
    if (item < p.items) {
      o.t0 = first_row(p);
      const int own = __shfl_sync(0xffffffffu, seq[0], 0);
      bool same = own >= 0 && o.c0 + 32 * V <= ch;
#pragma unroll
      for (int j = 0; j < kLoads; ++j) same = same && (seq[j] == own || seq[j] == -2);
      o.plain = __all_sync(0xffffffffu, same);
    }
    if (lane == 0) to = o;
    __syncwarp();
  }
};

// Step 2 of a tile: its run for the tiles after it (one warp),
template <int V>
__device__ __forceinline__ void publish(const Shared<V>& s, int n, const Plan& p, int ch, int lane) {
  const int64_t pos = s.info[n % kInfos].pos;
  const int c = s.info[n % kInfos].c0 + lane * V;
  if (pos % kGroup == kGroup - 1 || pos + 1 >= p.tiles) return;
  const Ch<V>(*ra)[32] = s.a[n & 1], (*rh)[32] = s.h[n & 1];
  Ch<V> A = ra[0][lane], H = rh[0][lane];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) join(A, H, ra[w][lane], rh[w][lane]);
  if (c >= ch) return;
  Pair<V> o;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    o.a[i] = A.f[i] != A.f[i] ? __uint_as_float(0x7fc00000u) : A.f[i];
    o.h[i] = H.f[i];
  }
  tell(p.agg + (pos * ch + c) * 2, o);
}
// and the state that reaches each of its warps (another). What is there already of the tiles before it is asked
// for while its warps still run.
template <int V> struct Carrier {
  int64_t pos, g;
  int c, before;
  bool in;
  const float *at, *at_start;
  int64_t step;
  uint32_t need;                    // tiles of the group, and its start, that were not there yet
  Pair<V> t[kGroup - 1], start;

  __device__ __forceinline__ void ask() {   // all at once
    uint32_t not_yet = 0;
#pragma unroll
    for (int j = 0; j < kGroup - 1; ++j)
      if (((need >> j) & 1) && in && !hear(at + j * step, t[j])) not_yet |= 1u << j;
    if ((need >> (kGroup - 1)) && in && !hear(at_start, start)) not_yet |= 1u << (kGroup - 1);
    need = __reduce_or_sync(0xffffffffu, not_yet);
  }
  __device__ __forceinline__ void begin(const Info& o, const Plan& p, int ch, int lane) {
    pos = o.pos;
    g = pos / kGroup;
    c = o.c0 + lane * V;
    before = (int)(pos % kGroup);
    in = c < ch;
    at = p.agg + (g * kGroup * ch + c) * 2;
    at_start = p.group + (g * ch + c) * 2;
    step = (int64_t)ch * 2;
    need = (1u << before) - 1 | (g > 0 ? 1u << (kGroup - 1) : 0u);
    ask();
  }
  __device__ __forceinline__ void end(Shared<V>& s, int n, const Plan& p, int ch, int lane, WsHeader* hdr,
                                      uint64_t limit_ns) {
    const Ch<V>(*ra)[32] = s.a[n & 1], (*rh)[32] = s.h[n & 1];
    Patience wait;
    while (need && wait.more(hdr, limit_ns)) ask();
    Ch<V> h = all<V>(0.f);
    if (g > 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) h.f[i] = start.h[i];
    }
#pragma unroll
    for (int j = 0; j < kGroup - 1; ++j) {
      if (j >= before) continue;
      Ch<V> A, H;
#pragma unroll
      for (int i = 0; i < V; ++i) A.f[i] = t[j].a[i], H.f[i] = t[j].h[i];
      fold(h, A, H);
    }
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      s.carry[n & 1][w][lane] = h;
      fold(h, ra[w][lane], rh[w][lane]);
    }
    if (before == kGroup - 1 && pos + 1 < p.tiles && in) {  // the next group's start
      Pair<V> o;
#pragma unroll
      for (int i = 0; i < V; ++i) o.a[i] = 1.f, o.h[i] = h.f[i];
      tell(p.group + ((g + 1) * ch + c) * 2, o);
    }
  }
};

// Bits of a warp's S rows: valid ones, first and last ones of a sequence; lane j holds row j's sequence.
struct Rows {
  uint32_t valid, first, last;
  int seq;
};
template <int S>
__device__ __forceinline__ Rows rows_of(const int32_t* seq, int64_t t0, int64_t T, int lane) {
  const int64_t t = t0 + lane;
  Rows r;
  r.seq = lane < S && t < T ? seq[t] : -1;
  const int before = lane < S && t < T && t > 0 ? seq[t - 1] : -1;
  const int after = lane < S && t + 1 < T ? seq[t + 1] : -1;
  r.valid = __ballot_sync(0xffffffffu, r.seq >= 0);
  r.first = __ballot_sync(0xffffffffu, r.seq >= 0 && before != r.seq);
  r.last = __ballot_sync(0xffffffffu, r.seq >= 0 && after != r.seq);
  return r;
}

// Rows of the inputs on their way into shared memory, [row][lane], zeros where there is nothing: where rows
// allow, a tile of each by TMA; else a warp's own S rows, a lane its own elements. (Rows as bulk copies of their
// own, 288 of 128 bytes a tile, took 10 us a tile.)
struct Maps { CUtensorMap m[4]; };
template <typename T, int V, int S>
__device__ __forceinline__ void fetch_own(typename Pack<T, V>::Raw* to, const T* p, int64_t pitch, int64_t t0,
                                          int64_t total, int c, int ch, int lane) {
  constexpr int kBytes = sizeof(T) * V;
  const T* src = p + t0 * pitch + c;
#pragma unroll
  for (int j = 0; j < S; ++j) {
    const bool ok = c < ch && t0 + j < total;
    if constexpr (kBytes >= 4) {
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(tc::smem_u32(to + j * 32 + lane)),
                   "l"(ok ? src : p), "n"(kBytes), "r"(ok ? kBytes : 0)
                   : "memory");
    } else {
      to[j * 32 + lane] = ok ? load<T, V>(src) : Pack<T, V>::close(all<V>(0.f));
    }
    src += pitch;
  }
}
__device__ __forceinline__ void fetch_own_done() {
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
}
// ---- forward --------------------------------------------------------------------------------
template <typename T, int V, bool kGate, int S>
__global__ void __launch_bounds__(kAll, kScanCtas)
gated_scan_kernel(const __grid_constant__ Maps maps, const T* __restrict__ x, int64_t x_pitch,
                  const T* __restrict__ r, int64_t r_pitch,
                  const T* __restrict__ ig, int64_t i_pitch, const float* __restrict__ a_log,
                  const float* state, const int32_t* __restrict__ idx, int64_t num_slots, int64_t stride,
                  float* final_state, T* __restrict__ y, float* __restrict__ carries, Plan plan, WsHeader* hdr,
                  int64_t total, int ch, bool wide, uint64_t limit_ns) {
  constexpr bool kFast = sizeof(T) == 2;
  constexpr int kInputs = kGate ? 3 : 2, kRowsTile = kWarps * S;
  using P = Pack<T, V>;
  using Raw = typename P::Raw;
  using Kept = typename std::conditional<V == 2, float4, float2>::type;
  extern __shared__ __align__(1024) uint8_t s_raw[];   // [input][row][lane], then a and m u of the tile before
  __shared__ Shared<V> s;
  Raw* const raw = reinterpret_cast<Raw*>(s_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    tc::mbar_init(&s.full, 1);
    tc::fence_mbar_init();
  }
  tc::grid_dep_wait();
  Taker<V, S, false> taker;
  if (warp == kWarps) {
    taker.start(hdr, lane);
    for (int n = 0; n < 2; ++n) {
      taker.ask(plan, hdr, total, lane);
      taker.tell_all(s.info[n], plan, total, ch, lane);
    }
    taker.ask(plan, hdr, total, lane);
  }
  __syncthreads();

  if (warp == kWarps) {   // this warp takes tiles and fetches their rows
    auto fetch = [&](int n) {
      const Info& o = s.info[n % kInfos];
      if (!wide || o.t0 < 0 || lane != 0) return;
      tc::mbar_expect_tx(&s.full, kInputs * kRowsTile * 32 * (uint32_t)sizeof(Raw));
#pragma unroll
      for (int q = 0; q < kInputs; ++q) tc::tma_load_2d(raw + q * kRowsTile * 32, &maps.m[q], &s.full, o.c0, (int)o.t0);
    };
    fetch(0);
    for (int n = 0; s.info[n % kInfos].t0 >= 0; ++n) {
      taker.tell_all(s.info[(n + 2) % kInfos], plan, total, ch, lane);
      taker.ask(plan, hdr, total, lane);
      bar_sync(kRan + (n & 1));
      fetch(n + 1);
      publish(s, n, plan, ch, lane);
      bar_arrive(kPublished + (n & 1), 64);
    }
    return;
  }
  if (warp > kWarps) {    // and this one carries the state
    Carrier<V> carrier;
    for (int n = 0; s.info[n % kInfos].t0 >= 0; ++n) {
      carrier.begin(s.info[n % kInfos], plan, ch, lane);
      bar_sync(kPublished + (n & 1), 64);
      carrier.end(s, n, plan, ch, lane, hdr, limit_ns);
      bar_arrive(kCarried + (n & 1));
    }
    return;
  }

  const Raw* const mine = raw + warp * S * 32 + lane;
  Kept* const kept = reinterpret_cast<Kept*>(s_raw + kInputs * kRowsTile * 32 * sizeof(Raw)) + warp * S * 32 + lane;
  auto fetch = [&](int n) {   // where the other warp does not
    const Info& o = s.info[n % kInfos];
    if (wide || o.t0 < 0) return;
    const int64_t t0 = o.t0 + warp * S;
    const int c = o.c0 + lane * V;
    Raw* const to = raw + warp * S * 32;
    fetch_own<T, V, S>(to, x, x_pitch, t0, total, c, ch, lane);
    fetch_own<T, V, S>(to + kRowsTile * 32, r, r_pitch, t0, total, c, ch, lane);
    if (kGate) fetch_own<T, V, S>(to + 2 * kRowsTile * 32, ig, i_pitch, t0, total, c, ch, lane);
  };
  auto unkeep = [&](int j, Ch<V>& a, Ch<V>& b) {
    const Kept q = kept[j * 32];
    if constexpr (V == 2) a = {{q.x, q.y}}, b = {{q.z, q.w}};
    else a = {{q.x}}, b = {{q.y}};
  };
  // step 3 of tile n
  auto finish = [&](int n) {
    const Info& o = s.info[n % kInfos];
    const int64_t t0 = o.t0 + warp * S;
    const int c = o.c0 + lane * V;
    const bool in = c < ch;
    Ch<V> h = s.carry[n & 1][warp][lane];
    T* yp = y + t0 * ch + c;
    const bool marked = carries && t0 % KDA_GATED_CARRY_ROWS == 0;
    static_assert(KDA_GATED_CARRY_ROWS % S == 0, "carries are left where a warp starts");
    if (marked && in && t0 < total) store<float, V>(carries + t0 / KDA_GATED_CARRY_ROWS * ch + c, h);
    if (o.plain) {
#pragma unroll
      for (int j = 0; j < S; ++j) {
        Ch<V> a, b;
        unkeep(j, a, b);
        h = fma(a, h, b);
        if (KDA_CHECK(t0 + j < total)) store<T, V>(yp, h);
        yp += ch;
      }
    } else {
      const Rows rows = rows_of<S>(plan.seq, t0, total, lane);
#pragma unroll 1
      for (int j = 0; j < S; ++j) {
        Ch<V> a, b;
        unkeep(j, a, b);
        if ((rows.first >> j) & 1) h = b;
        else h = fma(a, h, b);
        if (((rows.valid >> j) & 1) && in && KDA_CHECK(t0 + j < total && c + V <= ch)) store<T, V>(yp, h);
        yp += ch;
        if (((rows.last >> j) & 1) && final_state) {
          const int q = __shfl_sync(0xffffffffu, rows.seq, j);
          const int64_t slot = idx ? resolve_slot(idx, q, num_slots) : q;
          if (in && KDA_CHECK(slot >= 0)) store<float, V>(final_state + slot * stride + c, h);
        }
      }
    }
  };

  fetch(0);
  int n = 0;
  for (; s.info[n % kInfos].t0 >= 0; ++n) {
    const Info& o = s.info[n % kInfos];
    const int c = o.c0 + lane * V;
    Ch<V> rate;
#pragma unroll
    for (int i = 0; i < V; ++i) rate.f[i] = c + i < ch ? ssm_rate(a_log[c + i]) : 0.f;
    if (!wide) fetch_own_done();
    else if (!tc::mbar_wait(&s.full, n & 1)) raise_status(&hdr->status, KDA_DEVICE_PIPE_TIMEOUT);

    Ch<V> a[S], b[S];
#pragma unroll
    for (int j = 0; j < S; ++j) {
      Ch<V> w;
      a[j] = decay<kFast>(mul(rate, sigmoid<kFast>(P::open(mine[(kRowsTile + j) * 32]))), w);
      b[j] = mul(root(w), P::open(mine[j * 32]));
      if (kGate) b[j] = mul(b[j], sigmoid<kFast>(P::open(mine[(2 * kRowsTile + j) * 32])));
    }
    Ch<V> A = a[0], H = b[0];
    if (o.plain) {
#pragma unroll
      for (int j = 1; j < S; ++j) {
        H = fma(a[j], H, b[j]);
        A = mul(A, a[j]);
      }
    } else {
      const Rows rows = rows_of<S>(plan.seq, o.t0 + warp * S, total, lane);
      if (rows.first) A = all<V>(-1.f);
#pragma unroll
      for (int j = 0; j < S; ++j) {
        if ((rows.first >> j) & 1) {  // the sequence's own state instead of what came before
          const int q = __shfl_sync(0xffffffffu, rows.seq, j);
          const int64_t slot = idx ? resolve_slot(idx, q, num_slots) : q;
          Ch<V> h0 = all<V>(0.f);
          if (state && c < ch && KDA_CHECK(slot >= 0))
            h0 = Pack<float, V>::open(load<float, V>(state + slot * stride + c));
          b[j] = fma(a[j], h0, b[j]);
          H = b[j];
        } else if (j > 0) {
          H = fma(a[j], H, b[j]);
        }
        if (j > 0 && !rows.first) A = mul(A, a[j]);
      }
    }
    s.a[n & 1][warp][lane] = A;
    s.h[n & 1][warp][lane] = H;
    bar_arrive(kRan + (n & 1));
    if (n > 0) {
      bar_sync(kCarried + ((n - 1) & 1));
      fetch(n + 1);
      finish(n - 1);
    } else {
      fetch(1);
    }
#pragma unroll
    for (int j = 0; j < S; ++j) {
      if constexpr (V == 2) kept[j * 32] = make_float4(a[j].f[0], a[j].f[1], b[j].f[0], b[j].f[1]);
      else kept[j * 32] = make_float2(a[j].f[0], b[j].f[0]);
    }
  }
  if (n > 0) {
    bar_sync(kCarried + ((n - 1) & 1));
    finish(n - 1);
  }
  KDA_DEBUG_FOLD(&hdr->status);
}

// ---- backward -------------------------------------------------------------------------------
template <int V> struct BackShared : Shared<V> {
  Ch<V> fa[2][kWarps][32], fh[2][kWarps][32];   // the state's own runs, from the first row on
  Ch<V> state[2][kWarps][32];                   // the state that reaches each warp
  Ch<V> sum[2][kWarps][32];                     // each warp's part of dA_log
};

template <typename T, int V, bool kGate, int S>
__global__ void __launch_bounds__(kAll, kBackCtas)
gated_back_kernel(const __grid_constant__ Maps maps, const T* __restrict__ dy, int64_t dy_pitch,
                  const T* __restrict__ x, int64_t x_pitch,
                  const T* __restrict__ r, int64_t r_pitch, const T* __restrict__ ig, int64_t i_pitch,
                  const float* __restrict__ a_log, const float* __restrict__ carries,
                  const float* __restrict__ state, const float* __restrict__ dfinal, T* __restrict__ dx,
                  T* __restrict__ dr, T* __restrict__ di, float* __restrict__ dstate, float* __restrict__ part,
                  Plan plan, WsHeader* hdr, int64_t total, int ch, bool wide, uint64_t limit_ns) {
  constexpr bool kFast = sizeof(T) == 2;
  constexpr int kInputs = kGate ? 4 : 3, kRowsTile = kWarps * S;
  static_assert(kRowsTile == KDA_GATED_CARRY_ROWS, "a tile starts where a carry was left");
  using P = Pack<T, V>;
  using Raw = typename P::Raw;
  struct alignas(4 * sizeof(Raw)) Row4 { Raw x, r, g, i; };
  using Kept = typename std::conditional<V == 2, float4, float2>::type;
  extern __shared__ __align__(1024) uint8_t s_raw[];   // [input][row][lane], then what is kept of the tile before
  __shared__ BackShared<V> s;
  Raw* const raw = reinterpret_cast<Raw*>(s_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    tc::mbar_init(&s.full, 1);
    tc::fence_mbar_init();
  }
  tc::grid_dep_wait();
  Taker<V, S, true> taker;
  if (warp == kWarps) {
    taker.start(hdr, lane);
    for (int n = 0; n < 2; ++n) {
      taker.ask(plan, hdr, total, lane);
      taker.tell_all(s.info[n], plan, total, ch, lane);
    }
    taker.ask(plan, hdr, total, lane);
  }
  __syncthreads();

  if (warp == kWarps) {   // this warp takes tiles and fetches their rows
    auto fetch = [&](int n) {
      const Info& o = s.info[n % kInfos];
      if (!wide || o.t0 < 0 || lane != 0) return;
      tc::mbar_expect_tx(&s.full, kInputs * kRowsTile * 32 * (uint32_t)sizeof(Raw));
#pragma unroll
      for (int q = 0; q < kInputs; ++q) tc::tma_load_2d(raw + q * kRowsTile * 32, &maps.m[q], &s.full, o.c0, (int)o.t0);
    };
    auto add_up = [&](int n) {   // dA_log's part of tile n, which all warps are done with
      if (n < 0) return;
      const int c = s.info[n % kInfos].c0 + lane * V;
      Ch<V> sum = s.sum[n & 1][0][lane];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) sum = add(sum, s.sum[n & 1][w][lane]);
      if (c < ch) store<float, V>(part + s.info[n % kInfos].t0 / kRowsTile * ch + c, sum);
    };
    fetch(0);
    int n = 0;
    for (; s.info[n % kInfos].t0 >= 0; ++n) {
      taker.tell_all(s.info[(n + 2) % kInfos], plan, total, ch, lane);
      taker.ask(plan, hdr, total, lane);
      bar_sync(kRan + (n & 1));
      fetch(n + 1);
      publish<V>(s, n, plan, ch, lane);
      add_up(n - 2);
      bar_arrive(kPublished + (n & 1), 64);
    }
    bar_sync(kRan + (n & 1));
    add_up(n - 2);
    add_up(n - 1);
    return;
  }
  if (warp > kWarps) {    // and this one carries state and e
    Carrier<V> carrier;
    int n = 0;
    for (; s.info[n % kInfos].t0 >= 0; ++n) {
      const int c = s.info[n % kInfos].c0 + lane * V;
      Ch<V> h = all<V>(0.f);
      if (c < ch) h = Pack<float, V>::open(load<float, V>(carries + s.info[n % kInfos].t0 / kRowsTile * ch + c));
      carrier.begin(s.info[n % kInfos], plan, ch, lane);
      bar_sync(kPublished + (n & 1), 64);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        s.state[n & 1][w][lane] = h;
        fold(h, s.fa[n & 1][w][lane], s.fh[n & 1][w][lane]);
      }
      carrier.end(s, n, plan, ch, lane, hdr, limit_ns);
      bar_arrive(kCarried + (n & 1));
    }
    return;
  }

  const Raw* const mine = raw + warp * S * 32 + lane;
  Kept* const kept = reinterpret_cast<Kept*>(s_raw + kInputs * kRowsTile * 32 * sizeof(Raw)) + warp * S * 32 + lane;
  Row4* const kept_rows = reinterpret_cast<Row4*>(s_raw + kRowsTile * 32 * (kInputs * sizeof(Raw) + sizeof(Kept))) +
                          warp * S * 32 + lane;
  const int rank = kWarps - 1 - warp;
  auto fetch = [&](int n) {   // where the other warp does not
    const Info& o = s.info[n % kInfos];
    if (wide || o.t0 < 0) return;
    const int64_t t0 = o.t0 + warp * S;
    const int c = o.c0 + lane * V;
    Raw* const to = raw + warp * S * 32;
    fetch_own<T, V, S>(to, x, x_pitch, t0, total, c, ch, lane);
    fetch_own<T, V, S>(to + kRowsTile * 32, r, r_pitch, t0, total, c, ch, lane);
    fetch_own<T, V, S>(to + 2 * kRowsTile * 32, dy, dy_pitch, t0, total, c, ch, lane);
    if (kGate) fetch_own<T, V, S>(to + 3 * kRowsTile * 32, ig, i_pitch, t0, total, c, ch, lane);
  };
  // dfinal of a sequence whose last row is row j
  auto at_end = [&](const Rows& rows, int j, int c) {
    Ch<V> l = all<V>(0.f);
    const int q = __shfl_sync(0xffffffffu, rows.seq, j);
    if (dfinal && c < ch) l = Pack<float, V>::open(load<float, V>(dfinal + (int64_t)q * ch + c));
    return l;
  };
  // step 3 of tile n, from its last row to its first
  auto finish = [&](int n) {
    const Info& o = s.info[n % kInfos];
    const int64_t t0 = o.t0 + warp * S, at0 = t0 * ch + o.c0 + lane * V;
    const int c = o.c0 + lane * V;
    const bool in = c < ch;
    Ch<V> rate;
#pragma unroll
    for (int i = 0; i < V; ++i) rate.f[i] = c + i < ch ? ssm_rate(a_log[c + i]) : 0.f;
    Ch<V> e = s.carry[n & 1][rank][lane], sum = all<V>(0.f);
    const Ch<V> h0 = s.state[n & 1][warp][lane];
    auto one = [&](int j, const Ch<V>& reach, Ch<V> l, Ch<V>& ox, Ch<V>& orr, Ch<V>& oi) {
      const Kept q = kept[j * 32];
      const Row4 row = kept_rows[j * 32];
      Ch<V> a, hp;
      if constexpr (V == 2) a = {{q.x, q.y}}, hp = {{q.z, q.w}};
      else a = {{q.x}}, hp = {{q.y}};
      hp = add(hp, reach);
      l = add(l, P::open(row.g));
      e = mul(a, l);
      const Ch<V> er = exp_neg<kFast, true>(P::open(row.r)), sr = one_over<kFast>(er), g = mul(rate, sr);
      Ch<V> m, k, u = P::open(row.x);
      over_root(lost(g, series(g), a), k, m);
      const Ch<V> ml = mul(m, l);
      ox = ml;
      if (kGate) {
        const Ch<V> ei = exp_neg<kFast, true>(P::open(row.i)), si = one_over<kFast>(ei);
        u = mul(u, si);
        ox = mul(ml, si);
        oi = mul(mul(ml, u), mul(ei, si));
      }
      // p = e g h_{t-1} - e a (g / m) u, by e g: where g is large e is small or 0, but g h_{t-1} may pass fp32's range
      const Ch<V> eg = mul(e, g), p = fma(mul(mul(eg, k), a), u, mul(eg, hp));
      orr = mul(p, mul(er, sr));
      return p;
    };
    if (o.plain) {
      // what reaches row j of the warp's state: h0 decayed by the rows before it
      Ch<V> reach[S];
      reach[0] = h0;
#pragma unroll
      for (int j = 1; j < S; ++j) {
        const Kept q = kept[(j - 1) * 32];
        Ch<V> a;
        if constexpr (V == 2) a = {{q.x, q.y}};
        else a = {{q.x}};
        reach[j] = mul(reach[j - 1], a);
      }
#pragma unroll
      for (int j = S - 1; j >= 0; --j) {
        Ch<V> ox, orr, oi;
        sum = add(sum, one(j, reach[j], e, ox, orr, oi));
        if (KDA_CHECK(t0 + j < total && c + V <= ch)) {
          store<T, V>(dx + at0 + (int64_t)j * ch, ox);
          store<T, V>(dr + at0 + (int64_t)j * ch, orr);
          if (kGate) store<T, V>(di + at0 + (int64_t)j * ch, oi);
        }
      }
    } else {
      const Rows rows = rows_of<S>(plan.seq, t0, total, lane);
      const int until = rows.first ? __ffs(rows.first) - 1 : S;   // rows that h0 reaches
#pragma unroll 1
      for (int j = S - 1; j >= 0; --j) {
        Ch<V> reach = all<V>(0.f), ox, orr, oi;
        if (j < until) {
          reach = h0;
          for (int i = 0; i < j; ++i) {
            const Kept q = kept[i * 32];
            Ch<V> a;
            if constexpr (V == 2) a = {{q.x, q.y}};
            else a = {{q.x}};
            reach = mul(reach, a);
          }
        }
        const Ch<V> p = one(j, reach, (rows.last >> j) & 1 ? at_end(rows, j, c) : e, ox, orr, oi);
        const int64_t at = at0 + (int64_t)j * ch;
        if ((rows.valid >> j) & 1) {
          sum = add(sum, p);
          if (((rows.first >> j) & 1) && dstate) {
            const int q = __shfl_sync(0xffffffffu, rows.seq, j);
            if (in) store<float, V>(dstate + (int64_t)q * ch + c, e);
          }
        } else {
          ox = orr = oi = all<V>(0.f);
        }
        if (in && t0 + j < total && KDA_CHECK(c + V <= ch)) {
          store<T, V>(dx + at, ox);
          store<T, V>(dr + at, orr);
          if (kGate) store<T, V>(di + at, oi);
        }
      }
    }
    s.sum[n & 1][warp][lane] = sum;
  };

  fetch(0);
  int n = 0;
  for (; s.info[n % kInfos].t0 >= 0; ++n) {
    const Info& o = s.info[n % kInfos];
    const int c = o.c0 + lane * V;
    Ch<V> rate;
#pragma unroll
    for (int i = 0; i < V; ++i) rate.f[i] = c + i < ch ? ssm_rate(a_log[c + i]) : 0.f;
    if (!wide) fetch_own_done();
    else if (!tc::mbar_wait(&s.full, n & 1)) raise_status(&hdr->status, KDA_DEVICE_PIPE_TIMEOUT);

    // the rows' decays and what they add to the state; hp becomes the state before each row, without what
    // reaches the warp
    Row4 row[S];
    Ch<V> a[S], hp[S];
#pragma unroll
    for (int j = 0; j < S; ++j) {
      row[j].x = mine[j * 32];
      row[j].r = mine[(kRowsTile + j) * 32];
      row[j].g = mine[(2 * kRowsTile + j) * 32];
      if (kGate) row[j].i = mine[(3 * kRowsTile + j) * 32];
      Ch<V> w;
      a[j] = decay<kFast>(mul(rate, one_over<kFast>(exp_neg<kFast, true>(P::open(row[j].r)))), w);
      hp[j] = mul(root(w), P::open(row[j].x));
      if (kGate) hp[j] = mul(hp[j], sigmoid<kFast>(P::open(row[j].i)));
    }
    Ch<V> A = a[0], H = all<V>(0.f), E = all<V>(0.f);
#pragma unroll
    for (int j = 1; j < S; ++j) A = mul(A, a[j]);
    Ch<V> EA = A;
    if (o.plain) {
#pragma unroll
      for (int j = 0; j < S; ++j) {
        const Ch<V> b = hp[j];
        hp[j] = H;
        H = j > 0 ? fma(a[j], H, b) : b;
      }
#pragma unroll
      for (int j = S - 1; j >= 0; --j) E = mul(a[j], add(P::open(row[j].g), E));
    } else {
      const Rows rows = rows_of<S>(plan.seq, o.t0 + warp * S, total, lane);
      if (rows.first) A = all<V>(-1.f);
      if (rows.last) EA = all<V>(-1.f);
#pragma unroll
      for (int j = 0; j < S; ++j) {
        const Ch<V> b = hp[j];
        if ((rows.first >> j) & 1) {
          const int q = __shfl_sync(0xffffffffu, rows.seq, j);
          H = all<V>(0.f);
          if (state && c < ch) H = Pack<float, V>::open(load<float, V>(state + (int64_t)q * ch + c));
        }
        hp[j] = H;
        H = fma(a[j], H, b);
      }
#pragma unroll
      for (int j = S - 1; j >= 0; --j)
        E = mul(a[j], add(P::open(row[j].g), (rows.last >> j) & 1 ? at_end(rows, j, c) : E));
    }
    s.fa[n & 1][warp][lane] = A;
    s.fh[n & 1][warp][lane] = H;
    s.a[n & 1][rank][lane] = EA;
    s.h[n & 1][rank][lane] = E;
    bar_arrive(kRan + (n & 1));
    if (n > 0) {
      bar_sync(kCarried + ((n - 1) & 1));
      fetch(n + 1);
      finish(n - 1);
    } else {
      fetch(1);
    }
#pragma unroll
    for (int j = 0; j < S; ++j) {
      if constexpr (V == 2) kept[j * 32] = make_float4(a[j].f[0], a[j].f[1], hp[j].f[0], hp[j].f[1]);
      else kept[j * 32] = make_float2(a[j].f[0], hp[j].f[0]);
      kept_rows[j * 32] = row[j];
    }
  }
  if (n > 0) {
    bar_sync(kCarried + ((n - 1) & 1));
    finish(n - 1);
  }
  bar_arrive(kRan + (n & 1));
  KDA_DEBUG_FOLD(&hdr->status);
}

// dA_log: the tiles' parts of a channel, added up in a fixed order (9 us for 342 x 4096 parts: as many loads in flight as
// 1024 threads a CTA have).
__global__ void __launch_bounds__(1024)
gated_sum_kernel(const float* __restrict__ part, int64_t tiles, int ch, float* __restrict__ da) {
  __shared__ float s[32][33];
  tc::grid_dep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float sum = 0.f;
  if (c < ch) {
#pragma unroll 8
    for (int64_t k = warp; k < tiles; k += 32) sum += part[k * ch + c];
  }
  s[warp][lane] = sum;
  __syncthreads();
  sum = s[lane][warp];          // the warps' sums of channel `warp` of the block
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0 && blockIdx.x * 32 + warp < ch) da[blockIdx.x * 32 + warp] = sum;
}

// ---- tokens ---------------------------------------------------------------------------------
// One token, or a few drafted ones, a row: the states are read and written once, whatever the number of drafts, and
// the launch bounds the smallest calls. 64 x 4096 bf16 4.4 us; 512 x 5 x 2560 bf16 with the state after each kept 15 us,
// 4.5 TB/s.
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
    Ch<V> w;
    const Ch<V> a = decay<kFast>(mul(rate, sigmoid<kFast>(P::open(rr))), w);
    h = fma(a, h, mul(root(w), u));
    if (KDA_CHECK(t >= 0 && t < total && c + V <= ch)) store<T, V>(y + t * ch + c, h);
    if (cache) store<float, V>(cache + n * cache_pitch + (t - bos) * ch + c, h);
  }
  if (update_pool) store<float, V>(so, h);
  KDA_DEBUG_FOLD(status);
}

// ---- launches -------------------------------------------------------------------------------
constexpr int kRows = 12;      // rows a warp, forward
constexpr int kBackRows = 6;   // and backward

bool pairs(const void* p, int64_t pitch, int size) {
  return !p || ((uintptr_t)p % (2 * size) == 0 && pitch % 2 == 0);
}

Plan plan_of(const Layout& l, uint8_t* ws) {
  Plan p;
  p.seq = reinterpret_cast<int32_t*>(ws + l.seq);
  p.agg = reinterpret_cast<float*>(ws + l.agg);
  p.group = reinterpret_cast<float*>(ws + l.group);
  p.tiles = l.tiles;
  p.blocks = l.blocks;
  p.items = (uint32_t)(l.tiles * l.blocks);
  return p;
}

cudaError_t launch_plan(const GatedArgs& a, const Layout& l, const float* from, float* to, bool zero_bad,
                        cudaStream_t st) {
  const int64_t most = 2ll * gpu_sms(), unset = (int64_t)((l.seq - l.agg) / 16);
  int64_t blocks = (a.d.total_tokens + kPlanRows - 1) / kPlanRows;
  blocks = std::max(blocks, (unset + 4095) / 4096);
  if (to) blocks += row_blocks(a.d.num_seqs, a.d.channels, most);
  blocks = blocks < 1 ? 1 : blocks > most ? most : blocks;
  gated_plan_kernel<<<(unsigned)blocks, 1024, 0, st>>>(
      a.cu, a.idx, a.d.num_seqs, a.d.total_tokens, a.d.num_slots, reinterpret_cast<WsHeader*>(a.ws),
      reinterpret_cast<int32_t*>(a.ws + l.seq), reinterpret_cast<uint4*>(a.ws + l.agg), unset, from, to,
      a.d.channels, zero_bad);
  return cudaGetLastError();
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// Maps of [T, ch] rows, boxes of `cols` channels x `rows`.  False where the rows allow none (TMA wants them
// on 16-byte boundaries): the kernel then fetches them by elements.
template <typename T>
bool maps_of(Maps* m, const void* const* base, const int64_t* pitch, int count, int64_t total, int ch, int cols, int rows) {
  auto enc = encoder();
  if (!enc) return false;
  for (int q = 0; q < count; ++q) {
    if ((uintptr_t)base[q] % 16 != 0 || pitch[q] * (int64_t)sizeof(T) % 16 != 0) return false;
    cuuint64_t dims[2] = {(cuuint64_t)ch, (cuuint64_t)total};
    cuuint64_t strides[1] = {(cuuint64_t)pitch[q] * sizeof(T)};
    cuuint32_t box[2] = {(cuuint32_t)cols, (cuuint32_t)rows};
    cuuint32_t es[2] = {1u, 1u};
    if (enc(&m->m[q], sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
            const_cast<void*>(base[q]), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  }
  return true;
}

// CTAs that stay: as many as fit, or one a tile.
template <typename K>
cudaError_t stay(K* kernel, const Plan& p, int ctas, int bytes, unsigned* grid) {
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  const unsigned most = (unsigned)(ctas * gpu_sms());
  *grid = p.items < most ? p.items : most;
  return e;
}

template <typename T, int V, bool kGate>
cudaError_t run_scan(const GatedArgs& a, cudaStream_t st) {
  const Layout l = layout_of(a.d.total_tokens, a.d.channels, kRows * kWarps, V, false);
  const bool dense = !a.idx && a.state_out && a.state_out != a.state_in;
  cudaError_t e = launch_plan(a, l, a.state_in, dense ? a.state_out : nullptr, false, st);
  if (e != cudaSuccess || l.tiles == 0) return e;
  const Plan p = plan_of(l, a.ws);
  auto* kernel = gated_scan_kernel<T, V, kGate, kRows>;
  const int bytes = kRows * kThreads * V * ((kGate ? 3 : 2) * (int)sizeof(T) + 8);
  unsigned grid;
  if ((e = stay(kernel, p, kScanCtas, bytes, &grid)) != cudaSuccess) return e;
  Maps maps;
  const void* base[] = {a.x, a.r, a.i};
  const int64_t pitch[] = {a.d.x_pitch, a.d.r_pitch, a.d.i_pitch};
  const bool wide = maps_of<T>(&maps, base, pitch, kGate ? 3 : 2, a.d.total_tokens, a.d.channels, 32 * V, kRows * kWarps);
  return launch_behind(
      kernel, dim3(grid), dim3(kAll), bytes, st, maps, (const T*)a.x, a.d.x_pitch,
      (const T*)a.r, a.d.r_pitch, (const T*)a.i, a.d.i_pitch, a.a_log, a.state_in,
      a.idx, a.d.num_slots, a.slot_stride, a.state_out, (T*)a.y, a.carries, p,
      reinterpret_cast<WsHeader*>(a.ws), a.d.total_tokens, a.d.channels, wide, pipeline_wait_limit_ns());
}

template <typename T, int V, bool kGate>
cudaError_t run_back(const GatedArgs& a, cudaStream_t st) {
  const Layout l = layout_of(a.d.total_tokens, a.d.channels, kBackRows * kWarps, V, true);
  cudaError_t e = launch_plan(a, l, a.dfinal, a.dstate, true, st);
  if (e != cudaSuccess) return e;
  float* part = reinterpret_cast<float*>(a.ws + l.part);
  if (l.tiles > 0) {
    const Plan p = plan_of(l, a.ws);
    auto* kernel = gated_back_kernel<T, V, kGate, kBackRows>;
    const int bytes = kBackRows * kThreads * V * (((kGate ? 4 : 3) + 4) * (int)sizeof(T) + 8);
    unsigned grid;
    if ((e = stay(kernel, p, kBackCtas, bytes, &grid)) != cudaSuccess) return e;
    Maps maps;
    const void* base[] = {a.x, a.r, a.dy, a.i};
    const int64_t pitch[] = {a.d.x_pitch, a.d.r_pitch, a.dy_pitch, a.d.i_pitch};
    const bool wide = maps_of<T>(&maps, base, pitch, kGate ? 4 : 3, a.d.total_tokens, a.d.channels, 32 * V,
                                 kBackRows * kWarps);
    e = launch_behind(
        kernel, dim3(grid), dim3(kAll), bytes, st, maps, (const T*)a.dy, a.dy_pitch,
        (const T*)a.x, a.d.x_pitch, (const T*)a.r, a.d.r_pitch, (const T*)a.i,
        a.d.i_pitch, a.a_log, a.carries, a.state_in, a.dfinal, (T*)a.dx, (T*)a.dr, (T*)a.di, a.dstate, part, p,
        reinterpret_cast<WsHeader*>(a.ws), a.d.total_tokens, a.d.channels, wide,
        pipeline_wait_limit_ns());
    if (e != cudaSuccess) return e;
  }
  return launch_behind(gated_sum_kernel, dim3((unsigned)((a.d.channels + 31) / 32)), dim3(1024), 0, st, part, l.tiles,
                       a.d.channels, a.da_log);
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
  if (pass == Pass::kScan) return a.i ? run_scan<T, V, true>(a, st) : run_scan<T, V, false>(a, st);
  return a.i ? run_back<T, V, true>(a, st) : run_back<T, V, false>(a, st);
}
template <typename T, int V>
cudaError_t token_by_gate(const GatedArgs& a, cudaStream_t st) {
  return a.i ? run_token<T, V, true>(a, st) : run_token<T, V, false>(a, st);
}

// Four bytes of a row a lane: two channels in bf16 where every row starts on a boundary of two elements, else
// one (forward, 8192 x 4096 bf16: 80 us, 90 with one; 4095 channels, fetched by elements: 123). Tokens take two in fp32
// as well.
template <typename T>
cudaError_t by_type(const GatedArgs& a, cudaStream_t st, Pass pass) {
  const int e = sizeof(T);
  const int64_t ch = a.d.channels;
  const bool wide = (e == 2 || pass == Pass::kToken) && ch % 2 == 0 && pairs(a.x, a.d.x_pitch, e) &&
                    pairs(a.r, a.d.r_pitch, e) && pairs(a.i, a.d.i_pitch, e) && pairs(a.dy, a.dy_pitch, e) &&
                    pairs(a.y, ch, e) && pairs(a.dx, ch, e) && pairs(a.dr, ch, e) && pairs(a.di, ch, e) &&
                    pairs(a.state_in, a.slot_stride, 4) && pairs(a.state_out, a.slot_stride, 4) &&
                    pairs(a.cache, a.cache_pitch, 4) && pairs(a.carries, ch, 4) && pairs(a.dfinal, ch, 4) &&
                    pairs(a.dstate, ch, 4);
  if (pass == Pass::kToken) return wide ? token_by_gate<T, 2>(a, st) : token_by_gate<T, 1>(a, st);
  if constexpr (sizeof(T) == 2) {
    if (wide) return by_gate<T, 2>(a, st, pass);
  }
  return by_gate<T, 1>(a, st, pass);
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
