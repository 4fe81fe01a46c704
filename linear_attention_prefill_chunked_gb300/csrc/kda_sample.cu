// kda_sample.cu -- tokens, or probabilities, from logits under a temperature, top-k, top-p and min-p.
//
// With the entries of a row ordered by value, then index, p_i = exp((z_i - max) / T):
//   top-k  the first k of the order stand; top-p of these the first whose sum reaches top_p of it (what is
//          before an entry is below top_p of the whole); min-p those with p_i >= min_p
//   token = argmax p_i / noise_i over what stands (a draw in proportion to p for noise ~ Exp(1))
//   probabilities = p_i / their sum over what stands, 0 elsewhere
//
// All filters keep a prefix of one order, so all that is sought is its last entry, by count or by mass. A row
// is read once, into the shared memory of a cluster of CTAs (a slice each); no row is sorted. A histogram over
// the distance from the maximum (2048 bins of counts and masses) gives the bin the last entry lies in; the few
// entries of that bin are ranked against each other. Where a bin holds too many (equal values, as bf16 logits
// have them), further digits of the distance, then of the value, then of the index split it.
//
// An entry next to top-p's border stands or falls with the last digits of a sum over the row, so masses
// are whole numbers, p in units of 2^-44, whose sums do not depend on their order: results are bit-identical
// from run to run, whichever CTA adds first. p itself is 2^-n 2^(-j/64) 2^-r from a table and four terms of the
// exponential series, the distance carried as two floats: good to 2^-31, where a float's sum of a
// vocabulary would be off by more than the smallest entries that stand.
//
// Bound by HBM in principle (the row, and noise or probabilities), by the arithmetic of p and the cluster's
// exchanges (two to four a row) in practice.
#include <cooperative_groups.h>

#include "kda_internal.cuh"

namespace cg = cooperative_groups;

namespace kda {
namespace {

KDA_DEBUG_FLAG_DEFINE();

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kPer = kBins / kThreads;     // bins a thread looks after
constexpr int kList = 1024;                // entries that are ranked against each other
constexpr int kMaxRanks = 8;
constexpr int kSliceMax = 43008;           // floats of a row a CTA can hold beside the rest
constexpr int kPasses = 7;                 // digits: two of the distance, three of the value, two of the index
constexpr int kOneBits = 44;
constexpr unsigned long long kOne = 1ull << kOneBits;
constexpr float kMaskedOut = -__builtin_huge_valf();
using u64 = unsigned long long;

// 2^(-j/64) in units of 2^-44
__constant__ u64 c_pow[64] = {
    17592186044416ull, 17402683248456ull, 17215221774115ull, 17029779632301ull,
    16846335070792ull, 16664866571680ull, 16485352848846ull, 16307772845465ull,
    16132105731538ull, 15958330901445ull, 15786427971528ull, 15616376777705ull,
    15448157373097ull, 15281750025697ull, 15117135216047ull, 14954293634955ull,
    14793206181226ull, 14633853959423ull, 14476218277651ull, 14320280645363ull,
    14166022771192ull, 14013426560807ull, 13862474114787ull, 13713147726524ull,
    13565429880144ull, 13419303248457ull, 13274750690919ull, 13131755251623ull,
    12990300157313ull, 12850368815412ull, 12711944812080ull, 12575011910285ull,
    12439554047902ull, 12305555335825ull, 12173000056107ull, 12041872660113ull,
    11912157766698ull, 11783840160404ull, 11656904789672ull, 11531336765078ull,
    11407121357589ull, 11284243996830ull, 11162690269381ull, 11042445917079ull,
    10923496835354ull, 10805829071568ull, 10689428823381ull, 10574282437131ull,
    10460376406236ull, 10347697369602ull, 10236232110063ull, 10125967552830ull,
    10016890763953ull, 9908988948806ull, 9802249450589ull, 9696659748838ull,
    9592207457961ull, 9488880325783ull, 9386666232110ull, 9285553187305ull,
    9185529330885ull, 9086582930126ull, 8988702378691ull, 8891876195264ull
};

struct Item {
  uint32_t nk;   // descending values are ascending nk
  int idx;
  u64 w;
};
struct Best {
  float v;
  int idx;
};
__device__ __forceinline__ Best better(Best a, Best b) {  // of equal values the lower index
  return b.v > a.v || (b.v == a.v && b.idx < a.idx) ? b : a;
}

struct alignas(16) Shared {
  uint32_t cnt[kBins], lo[kBins], hi[kBins];
  Item list[kList];      // this CTA's entries of the bin
  Item all[kList];       // the cluster's
  u64 pow[64];
  Best warp_best[kWarps], best[kMaxRanks];
  float warp_low[kWarps], low[kMaxRanks];
  u64 warp_cnt[kWarps], warp_mass[kWarps], sum[kMaxRanks];
  u64 cnt_before, mass_before, cnt_in, mass_in;   // of the bin that was found
  int bin, n;
  uint32_t nk;
  int idx;
  u64 mass_incl;
};

static_assert(sizeof(Shared) % 16 == 0 && sizeof(Shared) + kSliceMax * 4 <= 232448, "227 KB a CTA");

// A row's parameters and what follows from them.
struct Row {
  float top, ch, cl, fx;   // the maximum; log2(e) / T as two floats; bins by distance
  bool inf;                // the maximum is infinite: its entries alone count
};

__device__ __forceinline__ uint32_t down_key(float z) {
  const uint32_t b = __float_as_uint(z);
  return ~((b >> 31) ? ~b : b | 0x80000000u);
}
// The distance from the maximum in octaves of p; infinite for masked entries.
__device__ __forceinline__ float octaves(const Row& r, float z) {
  const float d = r.top - z;
  return z == kMaskedOut ? __builtin_huge_valf() : r.inf ? (z == r.top ? 0.f : __builtin_huge_valf()) : d * r.ch;
}
__device__ __forceinline__ int distance(const Row& r, float z) {  // 22 bits, never falling as z falls
  const float y = octaves(r, z) * r.fx;
  return y < 4194303.f ? (int)y : 4194303;
}
// p, and p in units of 2^-44.
__device__ __forceinline__ float weight(const Row& r, float z, const u64* pow, u64& w) {
  const float yh = octaves(r, z);
  if (!(yh < 126.f)) {
    w = 0;
    return 0.f;
  }
  float yl = 0.f;
  if (!r.inf) {
    const float d = r.top - z, b = d - r.top, dl = (r.top - (d - b)) - (z + b);
    yl = fmaf(d, r.ch, -yh) + fmaf(d, r.cl, dl * r.ch);
  }
  const float n = floorf(yh), f = yh - n;
  const int j = (int)(f * 64.f);
  const float t = (f - (float)j * (1.f / 64.f) + yl) * -0.69314718055994531f;
  const float e = t * fmaf(t, fmaf(t, fmaf(t, 1.f / 24.f, 1.f / 6.f), 0.5f), 1.f);
  const u64 whole = pow[j];
  const float h = (float)(uint32_t)(whole >> 20) * 5.9604644775390625e-8f;  // of 2^24
  const int ni = (int)n;
  const long long fine = (long long)__float2int_rn(h * e * 137438953472.f) << 7;  // of 2^37
  w = ni < 64 ? (whole + (u64)fine) >> ni : 0;
  return fmaf(h, e, h) * __uint_as_float((uint32_t)(127 - ni) << 23);
}

// Sum over the threads before this one, of two numbers.
__device__ __forceinline__ void before_me(u64 c, u64 m, Shared& s, u64& bc, u64& bm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 ic = c, im = m;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 a = __shfl_up_sync(0xffffffffu, ic, o), b = __shfl_up_sync(0xffffffffu, im, o);
    if (lane >= o) {
      ic += a;
      im += b;
    }
  }
  if (lane == 31) {
    s.warp_cnt[warp] = ic;
    s.warp_mass[warp] = im;
  }
  __syncthreads();
  bc = ic - c;
  bm = im - m;
  for (int w = 0; w < warp; ++w) {
    bc += s.warp_cnt[w];
    bm += s.warp_mass[w];
  }
  __syncthreads();
}

// The cluster's histogram: this thread's bins and what lies in the bins before them.
struct Bins {
  uint32_t c[kPer];
  u64 m[kPer], before_c, before_m, total_m;
};

// One row a cluster. kProbs: probabilities, else a token.
template <typename T, bool kProbs>
__global__ void __launch_bounds__(kThreads)
sample_kernel(const T* __restrict__ logits, int64_t pitch, const float* __restrict__ noise, int64_t noise_pitch,
              const float* __restrict__ temperature, const int32_t* __restrict__ top_k,
              const float* __restrict__ top_p, const float* __restrict__ min_p, float temperature_all,
              int top_k_all, float top_p_all, float min_p_all, int32_t* __restrict__ token,
              float* __restrict__ probs, uint32_t* __restrict__ status, int rows, int vocab, int slice) {
  extern __shared__ __align__(16) uint8_t s_raw[];
  Shared& s = *reinterpret_cast<Shared*>(s_raw);
  float* s_z = reinterpret_cast<float*>(s_raw + sizeof(Shared));   // this CTA's slice of the row
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), ranks = (int)cl.num_blocks(), tid = threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
  const int row = (int)(blockIdx.x / ranks) - 1;

  auto bad_params = [&](int n) {
    const float t = temperature ? temperature[n] : temperature_all;
    const float p = top_p ? top_p[n] : top_p_all, m = min_p ? min_p[n] : min_p_all;
    return !(t >= 0.f) || p != p || m != m;
  };
  if (row < 0) {  // the first cluster's: the status word
    if (rank != 0) return;
    int bad = 0;
    for (int n = tid; n < rows; n += kThreads) bad |= bad_params(n);
    bad = __syncthreads_or(bad);
    if (tid == 0) set_status(status, bad ? KDA_DEVICE_BAD_PARAM : 0u);
    return;
  }
  const int v0 = rank * slice, v1 = vocab - v0 < slice ? (vocab > v0 ? vocab : v0) : v0 + slice;
  const int mine = v1 - v0;
  auto nothing = [&] {  // no entry stands
    if (kProbs) {
      for (int i = tid; i < mine; i += kThreads) probs[(int64_t)row * vocab + v0 + i] = 0.f;
    } else if (rank == 0 && tid == 0) {
      token[row] = -1;
    }
  };
  if (bad_params(row)) {  // the whole cluster, as at each return below
    nothing();
    return;
  }
  const float temp = temperature ? temperature[row] : temperature_all;
  const int k = top_k ? top_k[row] : top_k_all;
  const float tp = top_p ? top_p[row] : top_p_all;
  const float mp = fminf(min_p ? min_p[row] : min_p_all, 1.f);

  // every CTA of the cluster has to have started before another writes into its shared memory
  auto started = cl.barrier_arrive();
  if (tid < 64) s.pow[tid] = c_pow[tid];
  Best top{kMaskedOut, 0x7fffffff};
  float low = __builtin_huge_valf();
  const T* z = logits + (int64_t)row * pitch + v0;
  for (int i = tid; i < mine; i += kThreads) {
    float x = to_f32(z[i]) + 0.f;         // -0 counts as 0
    if (x != x) x = kMaskedOut;           // and what is no number as masked
    s_z[i] = x;
    top = better(top, Best{x, v0 + i});
    if (x > kMaskedOut) low = fminf(low, x);
  }
  auto across = [&](Best b) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
      b = better(b, Best{__shfl_xor_sync(0xffffffffu, b.v, o), __shfl_xor_sync(0xffffffffu, b.idx, o)});
    return b;
  };
  // joins the cluster's best entries (every CTA has them all then)
  auto join = [&](Best b) {
    b = across(b);
    if (lane == 0) s.warp_best[warp] = b;
    __syncthreads();
    if (warp == 0) {
      b = across(lane < kWarps ? s.warp_best[lane] : Best{kMaskedOut, 0x7fffffff});
      if (lane < ranks) cl.map_shared_rank(s.best, lane)[rank] = b;
    }
    cl.sync();
    b = s.best[0];
    for (int q = 1; q < ranks; ++q) b = better(b, s.best[q]);
    return b;
  };
#pragma unroll
  for (int o = 16; o; o >>= 1) low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
  if (lane == 0) s.warp_low[warp] = low;
  cl.barrier_wait(std::move(started));
  __syncthreads();
  if (warp == 0) {
    low = lane < kWarps ? s.warp_low[lane] : __builtin_huge_valf();
#pragma unroll
    for (int o = 16; o; o >>= 1) low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
    if (lane < ranks) cl.map_shared_rank(s.low, lane)[rank] = low;
  }
  top = join(top);
  for (int q = 0; q < ranks; ++q) low = fminf(q ? low : s.low[0], s.low[q]);
  if (top.v == kMaskedOut) {
    nothing();
    return;
  }
  if (temp == 0.f || k == 1 || tp <= 0.f) {  // the first entry alone
    if (kProbs) {
      for (int i = tid; i < mine; i += kThreads) probs[(int64_t)row * vocab + v0 + i] = v0 + i == top.idx ? 1.f : 0.f;
    } else if (rank == 0 && tid == 0) {
      token[row] = top.idx;
    }
    return;
  }
  Row r;
  r.top = top.v;
  r.inf = top.v == __builtin_huge_valf();
  const double c = fmin(1.4426950408889634074 / (double)temp, 1e38);
  r.ch = (float)c;
  r.cl = (float)(c - (double)r.ch);
  r.fx = 1.f;
  {  // bins over the row's range, of 64 octaves at most
    const float range = fminf(octaves(r, low), 64.f);
    r.fx = 4194304.f / fmaxf(range, 1e-30f);
  }
  const bool by_count = k > 0 && k < vocab, by_mass = tp < 1.f;
  const u64 least = mp > 0.f ? (u64)ceil((double)mp * (double)kOne) : 0;

  // the entries whose digits before `depth` are p[]
  int p[kPasses];
  auto digit = [&](int d, int i, float x) -> int {
    const uint32_t nk = down_key(x);
    switch (d) {
      case 0: return distance(r, x) >> 11;
      case 1: return distance(r, x) & 2047;
      case 2: return (int)(nk >> 21);
      case 3: return (int)((nk >> 10) & 2047);
      case 4: return (int)(nk & 1023);
      case 5: return (v0 + i) >> 9;
      default: return (v0 + i) & 511;
    }
  };
  auto member = [&](int depth, int i, float x) {
    for (int d = 0; d < depth; ++d)
      if (digit(d, i, x) != p[d]) return false;
    return true;
  };
  auto histogram = [&](int depth, Bins& b) {
    for (int i = tid; i < kBins; i += kThreads) s.cnt[i] = s.lo[i] = s.hi[i] = 0;
    __syncthreads();
    for (int i = tid; i < mine; i += kThreads) {
      const float x = s_z[i];
      if (!member(depth, i, x)) continue;
      const int at = digit(depth, i, x);
      u64 w;
      weight(r, x, s.pow, w);
      if (!KDA_CHECK(at >= 0 && at < kBins)) continue;
      atomicAdd(&s.cnt[at], 1u);
      if (w) {
        const uint32_t lo = (uint32_t)w, was = atomicAdd(&s.lo[at], lo);
        const uint32_t hi = (uint32_t)(w >> 32) + (was + lo < was ? 1u : 0u);
        if (hi) atomicAdd(&s.hi[at], hi);
      }
    }
    cl.sync();
    u64 c = 0, m = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) b.c[j] = 0, b.m[j] = 0;
    for (int q = 0; q < ranks; ++q) {
      const Shared* o = cl.map_shared_rank(&s, q);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        b.c[j] += o->cnt[tid * kPer + j];
        b.m[j] += (u64)o->hi[tid * kPer + j] << 32 | o->lo[tid * kPer + j];
      }
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) c += b.c[j], m += b.m[j];
    before_me(c, m, s, b.before_c, b.before_m);
    if (tid == kThreads - 1) s.mass_incl = b.before_m + m;
    __syncthreads();
    b.total_m = s.mass_incl;
    __syncthreads();
  };
  // the bin where the count (or mass) of the order reaches `target`
  auto find = [&](const Bins& b, bool mass, u64 target) {
    u64 bc = b.before_c, bm = b.before_m;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const u64 was = mass ? bm : bc, v = mass ? b.m[j] : b.c[j];
      if (was < target && target <= was + v) {
        s.bin = tid * kPer + j;
        s.cnt_before = bc;
        s.mass_before = bm;
        s.cnt_in = b.c[j];
        s.mass_in = b.m[j];
      }
      bc += b.c[j];
      bm += b.m[j];
    }
    __syncthreads();
  };
  // The last entry that stands, in s.nk and s.idx, and the mass up to and with it, in s.mass_incl.
  auto last = [&](const Bins& first, bool mass, u64 target) {
    find(first, mass, target);
    int depth = 1;
    p[0] = s.bin;
    u64 cb = s.cnt_before, mb = s.mass_before, in = s.cnt_in;
    while (in > kList && depth < kPasses) {
      cl.sync();   // everyone has read the histogram before
      Bins b;
      histogram(depth, b);
      find(b, mass, target - (mass ? mb : cb));
      p[depth++] = s.bin;
      cb += s.cnt_before;
      mb += s.mass_before;
      in = s.cnt_in;
    }
    cl.sync();     // everyone has read the histogram, and the lists of a search before
    if (tid == 0) s.n = 0;
    __syncthreads();
    for (int i = tid; i < mine; i += kThreads) {
      const float x = s_z[i];
      if (!member(depth, i, x)) continue;
      Item it;
      it.nk = down_key(x);
      it.idx = v0 + i;
      weight(r, x, s.pow, it.w);
      const int at = atomicAdd(&s.n, 1);
      if (KDA_CHECK(at < kList)) s.list[at] = it;
    }
    cl.sync();
    int n = 0;
    for (int q = 0; q < ranks; ++q) {
      const Shared* o = cl.map_shared_rank(&s, q);
      const int m = o->n;
      for (int i = tid; i < m; i += kThreads)
        if (KDA_CHECK(n + i < kList)) s.all[n + i] = o->list[i];
      n += m;
    }
    __syncthreads();
    const u64 want = target - (mass ? mb : cb);
    for (int i = tid; i < n; i += kThreads) {
      const Item it = s.all[i];
      u64 c = 0, m = 0;
      for (int j = 0; j < n; ++j) {
        const Item o = s.all[j];
        if (o.nk < it.nk || (o.nk == it.nk && o.idx < it.idx)) {
          ++c;
          m += o.w;
        }
      }
      const u64 was = mass ? m : c, v = mass ? it.w : 1;
      if (was < want && want <= was + v) {
        s.nk = it.nk;
        s.idx = it.idx;
        s.mass_incl = mb + m + it.w;
      }
    }
    __syncthreads();
  };

  bool cut = false;
  u64 sum = 0;
  if (by_count || by_mass) {
    Bins b;
    histogram(0, b);
    sum = b.total_m;
    if (by_count) {
      last(b, false, (u64)k);
      sum = s.mass_incl;
      cut = true;
    }
    if (by_mass) {
      const double x = ceil((double)tp * (double)sum);
      u64 target = x < 1. ? 1 : (u64)x;
      if (target > sum) target = sum;
      __syncthreads();
      last(b, true, target);
      sum = s.mass_incl;
      cut = true;
    }
  }
  const uint32_t nk = cut ? s.nk : 0xffffffffu;
  const int at = cut ? s.idx : 0x7fffffff;
  auto stands = [&](int i, float x, u64 w) {
    const uint32_t key = down_key(x);
    return w >= least && (key < nk || (key == nk && v0 + i <= at));
  };
  if (kProbs) {
    if (least || !(by_count || by_mass)) {  // what min-p leaves is not known yet
      u64 part = 0;
      for (int i = tid; i < mine; i += kThreads) {
        u64 w;
        const float x = s_z[i];
        weight(r, x, s.pow, w);
        if (stands(i, x, w)) part += w;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
      __syncthreads();
      if (lane == 0) s.warp_mass[warp] = part;
      __syncthreads();
      if (tid < ranks) {
        u64 all = 0;
        for (int q = 0; q < kWarps; ++q) all += s.warp_mass[q];
        cl.map_shared_rank(s.sum, tid)[rank] = all;
      }
      cl.sync();
      sum = 0;
      for (int q = 0; q < ranks; ++q) sum += s.sum[q];
    } else {
      cl.sync();  // no CTA leaves while another reads its lists
    }
    const float inv = (float)((double)kOne / (double)sum);
    for (int i = tid; i < mine; i += kThreads) {
      u64 w;
      const float x = s_z[i], pr = weight(r, x, s.pow, w);
      probs[(int64_t)row * vocab + v0 + i] = stands(i, x, w) ? pr * inv : 0.f;
    }
  } else {
    Best best{-1.f, 0x7fffffff};
    for (int i = tid; i < mine; i += kThreads) {
      u64 w;
      const float x = s_z[i], pr = weight(r, x, s.pow, w);
      if (pr > 0.f && stands(i, x, w))
        best = better(best, Best{pr / noise[(int64_t)row * noise_pitch + v0 + i], v0 + i});
    }
    cl.sync();     // everyone has read s.best, and the lists
    best = join(best);
    if (rank == 0 && tid == 0) token[row] = best.v < 0.f ? -1 : best.idx;
  }
  KDA_DEBUG_FOLD(status);
}

template <typename T, bool kProbs>
cudaError_t launch(const SampleArgs& a, cudaStream_t st) {
  const int sms = gpu_sms(), vocab = a.d.vocab, rows = a.d.num_rows;
  // a slice has to fit; below two CTAs an SM the row is shared by more
  int ranks = 1;
  while (ranks < kMaxRanks && ((vocab + ranks - 1) / ranks > 16384 ||
                               ((int64_t)rows * ranks < 2 * sms && vocab / ranks > 4096)))
    ranks *= 2;
  const int slice = ((vocab + ranks - 1) / ranks + 7) / 8 * 8;
  auto* kernel = sample_kernel<T, kProbs>;
  const int bytes = (int)sizeof(Shared) + slice * 4;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)sizeof(Shared) + kSliceMax * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((rows + 1) * ranks));  // (num_rows is at most 2^27)
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)ranks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, (const T*)a.logits, a.d.logits_pitch, a.noise, a.d.noise_pitch,
                            a.temperature, a.top_k, a.top_p, a.min_p, a.d.temperature, a.d.top_k, a.d.top_p,
                            a.d.min_p, a.token, a.probs, a.status, rows, vocab, slice);
}

}  // namespace

bool sample_fits(const kda_sample_desc_t& d) {
  return d.vocab <= kMaxRanks * kSliceMax && d.num_rows <= (1 << 27);
}

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t st) {
  if (a.probs) return a.d.dtype == KDA_BF16 ? launch<__nv_bfloat16, true>(a, st) : launch<float, true>(a, st);
  return a.d.dtype == KDA_BF16 ? launch<__nv_bfloat16, false>(a, st) : launch<float, false>(a, st);
}

}  // namespace kda
