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
// the distance from the maximum (1024 bins of counts and masses) gives the bin the last entry lies in; the few
// entries of that bin are ranked against each other. Where a bin holds too many (equal values, as bf16 logits
// have them), further digits of the distance, then of the value, then of the index split it.
//
// An entry next to top-p's border stands or falls with the last digits of a sum over the row, so masses
// are whole numbers, p in units of 2^-44, whose sums do not depend on their order: results are bit-identical
// from run to run, whichever CTA adds first. p itself is 2^-n 2^(-j/32) 2^-r from a table, an entry a lane, and four
// terms of the exponential series, the distance carried as two floats: good to 2^-28 (2^-31 on average), where a
// float's sum of a vocabulary would be off by more than the smallest entries that stand.
//
// Bound by HBM in principle (the row, and noise or probabilities), by the arithmetic of p, the histogram's shared
// atomics and the cluster's exchanges (three to six a row) in practice: 64 x 131072 fp32, all filters,
// 53 us (0.63 TB/s); 1 x 32003 bf16 17 us; probabilities under top-p, 320 x 131072 fp32, 260 us (1.29 TB/s; without the
// histogram's atomics 35 less; masses as one 64-bit atomic instead of three of 32 bits 333 against 296 at that step).
#include <cooperative_groups.h>

#include <type_traits>

#include "kda_internal.cuh"
#include "tc_ptx.cuh"

namespace cg = cooperative_groups;

namespace kda {
namespace {

KDA_DEBUG_FLAG_DEFINE();

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kFine = 32, kCoarse = kBins / kFine;   // bins are looked through in two steps
constexpr int kList = 1024;                // entries that are ranked against each other
constexpr int kFew = 512;                  // entries up to the k-th that are ranked by number and mass at once,
constexpr int kPairs = 64;                 // pairs of them a thread
constexpr int kMaxRanks = 8;
constexpr int kMostQuads = 22;             // fours of entries a thread looks after at most
constexpr int kPasses = 7;                 // digits: the distance, four of the value, two of the index
constexpr int kOneBits = 44;
constexpr unsigned long long kOne = 1ull << kOneBits;
constexpr float kMaskedOut = -__builtin_huge_valf();
using u64 = unsigned long long;

// 2^(-j/32) in units of 2^-44
__constant__ u64 c_pow[32] = {
    17592186044416ull, 17215221774115ull, 16846335070792ull, 16485352848846ull,
    16132105731538ull, 15786427971528ull, 15448157373097ull, 15117135216047ull,
    14793206181226ull, 14476218277651ull, 14166022771192ull, 13862474114787ull,
    13565429880144ull, 13274750690919ull, 12990300157313ull, 12711944812080ull,
    12439554047902ull, 12173000056107ull, 11912157766698ull, 11656904789672ull,
    11407121357589ull, 11162690269381ull, 10923496835354ull, 10689428823381ull,
    10460376406236ull, 10236232110063ull, 10016890763953ull, 9802249450589ull,
    9592207457961ull, 9386666232110ull, 9185529330885ull, 8988702378691ull
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
  union {
    struct {
      uint32_t cnt[kBins], part[3][kBins];   // of masses, 16 bits and 16 and the rest: sums of a CTA fit 32 bits
    };
    Item all[kList];     // the cluster's entries of the bin
  };
  Item list[kList];      // this CTA's entries of the bin
  Best warp_best[kWarps], best[2][kMaxRanks];
  float warp_low[kWarps], low[kMaxRanks];
  u64 coarse[kMaxRanks][kCoarse], fine[kMaxRanks][kFine];   // each CTA's sums, of its bins by 32 and of 32 of its bins
  u64 warp_mass[kWarps], sum[kMaxRanks];
  int n, counts[kMaxRanks];             // entries of the bin, here and in each CTA
  uint32_t nk;                          // the entry that was sought,
  int idx;
  u64 mass_incl, kth_mass;              // and the mass up to and with it; the same of the k-th
  float ch, cl, mp, inv;                    // what is worked out in 64 bits, by one thread
  u64 target;
};

static_assert(kMostQuads * 4 * kThreads < 65536, "sums of 16 bits");
static_assert(sizeof(Shared) + kMostQuads * kThreads * 16 <= 232448, "227 KB a CTA");

// A row's parameters and what follows from them.
struct Row {
  float top, ch, cl, fx;   // the maximum; log2(e) / T as two floats; bins by distance
};

__device__ __forceinline__ uint32_t down_key(float z) {
  const uint32_t b = __float_as_uint(z);
  return (b >> 31) ? b : ~(b | 0x80000000u);
}
// The bin of an entry by its distance from the maximum, never falling as z falls (1.5 * 2^23 rounds to whole
// numbers).
constexpr float kRound = 12582912.f;
constexpr int kRoundBits = 0x4b400000;
__device__ __forceinline__ int distance(const Row& r, float z) {
  return __float_as_int(fminf((r.top - z) * r.ch * r.fx, (float)(kBins - 1)) + kRound) - kRoundBits;
}
// Adds v to a word of shared memory kOff bytes behind `at`, unless it is 0 (without a branch).
template <int kOff> __device__ __forceinline__ void add_shared(uint32_t at, uint32_t v) {
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %1, 0;\n @p red.shared.add.u32 [%0 + %2], %1;\n}\n" ::"r"(at), "r"(v),
               "n"(kOff)
               : "memory");
}
// The distance from the maximum in octaves of p, as two floats.
__device__ __forceinline__ void octaves(const Row& r, float z, float& yh, float& yl) {
  const float d = r.top - z, b = d - r.top, dl = (r.top - (d - b)) - (z + b);
  yh = d * r.ch;
  yl = fmaf(d, r.ch, -yh) + fmaf(d, r.cl, dl * r.ch);
}
// p = 2^-n 2^(-j/32) (1 + e).  `whole` is p 2^n in units of 2^-44, good to 2^-28 however small p is: min-p is
// compared with it.  units() is p in units of 2^-44 (0 for masked entries), whose sums are exact.  Of a whole warp,
// whose lanes hold the table between them (reads of shared memory at 32 places take several times as long), or of
// some of its lanes.
struct Table {
  uint32_t lo, hi;
  float f;
  __device__ __forceinline__ explicit Table(int lane)
      : lo((uint32_t)c_pow[lane]), hi((uint32_t)(c_pow[lane] >> 32)),
        f((float)(uint32_t)(c_pow[lane] >> 20) * 5.9604644775390625e-8f) {}  // 2^-24
};
struct Mass {
  u64 whole;
  float yh;
  int n;
  __device__ __forceinline__ u64 units() const { return yh < 45.f ? whole >> n : 0; }
  __device__ __forceinline__ bool reaches(float p) const {   // p <= 1
    return yh < 127.f && whole >= (u64)(fminf(p * __int_as_float((n + 127) << 23), 2.f) * (float)kOne);
  }
};
template <bool kWarp> __device__ __forceinline__ Mass mass_of(const Row& r, float z, const Table& table) {
  float yh, yl;
  octaves(r, z, yh, yl);
  const float m = fmaf(yh, 32.f, kRound);
  const int k = __float_as_int(m) - kRoundBits, n = k >> 5, j = k & 31;
  const float t = (fmaf(m - kRound, -1.f / 32.f, yh) + yl) * -0.69314718055994531f;
  const float e = t * fmaf(t, fmaf(t, fmaf(t, 1.f / 24.f, 1.f / 6.f), 0.5f), 1.f);   // |e| < 0.011
  u64 whole;
  float f;
  if constexpr (kWarp) {
    whole = (u64)__shfl_sync(0xffffffffu, table.hi, j) << 32 | __shfl_sync(0xffffffffu, table.lo, j);
    f = __shfl_sync(0xffffffffu, table.f, j);
  } else {
    whole = c_pow[j];
    f = (float)(uint32_t)(whole >> 20) * 5.9604644775390625e-8f;
  }
  const int fine = __float2int_rn(f * e * 68719476736.f);    // of 2^36
  asm("mad.wide.s32 %0, %1, 256, %0;" : "+l"(whole) : "r"(fine));
  return {whole, yh, n};
}
template <bool kWarp> __device__ __forceinline__ u64 mass(const Row& r, float z, const Table& table) {
  return mass_of<kWarp>(r, z, table).units();
}
// p to 2^-22
__device__ __forceinline__ float weight(const Row& r, float z) {
  float yh, yl;
  octaves(r, z, yh, yl);
  float p;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(-yh));
  return yh < 126.f ? fmaf(p, yl * -0.69314718055994531f, p) : 0.f;
}
__device__ __forceinline__ float value_of(uint32_t nk) {   // of a descending key
  return __uint_as_float((nk >> 31) ? nk : ~nk & 0x7fffffffu);
}

// One row a cluster, `quads` fours of entries a thread. kProbs: probabilities, else a token.
template <typename T, bool kProbs>
__global__ void __launch_bounds__(kThreads, 2)
sample_kernel(const T* __restrict__ logits, int64_t pitch, const float* __restrict__ noise, int64_t noise_pitch,
              const float* __restrict__ temperature, const int32_t* __restrict__ top_k,
              const float* __restrict__ top_p, const float* __restrict__ min_p, float temperature_all,
              int top_k_all, float top_p_all, float min_p_all, int32_t* __restrict__ token,
              float* __restrict__ probs, uint32_t* __restrict__ status, int rows, int vocab, int slice, int quads, bool wide) {
  extern __shared__ __align__(16) uint8_t s_raw[];
  Shared& s = *reinterpret_cast<Shared*>(s_raw);
  float4* const mine4 = reinterpret_cast<float4*>(s_raw + sizeof(Shared)) + threadIdx.x;   // fours, kThreads apart
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
  // entry e of four q is at 4 (q kThreads + tid) + e of the slice
  const int v0 = rank * slice, left = vocab - v0, mine = left < slice ? (left > 0 ? left : 0) : slice;
  auto place = [&](int q) { return 4 * (q * kThreads + tid); };
  auto get = [&](int q, float (&z)[4]) {
    const float4 v = mine4[q * kThreads];
    z[0] = v.x; z[1] = v.y; z[2] = v.z; z[3] = v.w;
  };
  float* const out = kProbs ? probs + (int64_t)row * vocab + v0 : nullptr;
  auto put = [&](int q, const float (&o)[4]) {
    const int i = place(q);
    if (wide && i + 4 <= mine) {
      *reinterpret_cast<float4*>(out + i) = make_float4(o[0], o[1], o[2], o[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e < mine) out[i + e] = o[e];
    }
  };
  auto only = [&](int idx) {  // one entry stands, or none (idx < 0)
    if (kProbs) {
      for (int q = 0; q < quads; ++q) {
        float o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = v0 + place(q) + e == idx ? 1.f : 0.f;
        put(q, o);
      }
    } else if (rank == 0 && tid == 0) {
      token[row] = idx;
    }
  };
  if (bad_params(row)) {  // the whole cluster, as at each return below
    only(-1);
    return;
  }
  const float temp = temperature ? temperature[row] : temperature_all;
  const int k = top_k ? top_k[row] : top_k_all;
  const float tp = top_p ? top_p[row] : top_p_all;
  if (tid == 0) {
    const double c = fmin(1.4426950408889634074 / (double)temp, 1e38);   // (at temperature 0 not used)
    s.ch = (float)c;
    s.cl = (float)(c - (double)s.ch);
    s.mp = fminf(min_p ? min_p[row] : min_p_all, 1.f);
  }

  // every CTA of the cluster has to have started before another writes into its shared memory
  auto started = cl.barrier_arrive();
  const Table table(lane);
  Best top{kMaskedOut, 0x7fffffff};
  float low = __builtin_huge_valf();
  const T* from = logits + (int64_t)row * pitch + v0;
#pragma unroll 8
  for (int q = 0; q < quads; ++q) {
    const int i = place(q);
    float z[4];
    if (wide && i + 4 <= mine) {
      load4(from + i, z);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] = i + e < mine ? to_f32(from[i + e]) : kMaskedOut;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      z[e] += 0.f;                              // -0 counts as 0
      z[e] = z[e] != z[e] ? kMaskedOut : z[e];  // and what is no number as masked
      if (z[e] > top.v) top = Best{z[e], v0 + i + e};
      if (z[e] > kMaskedOut) low = fminf(low, z[e]);
    }
    mine4[q * kThreads] = make_float4(z[0], z[1], z[2], z[3]);
  }
  auto across = [&](Best b) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
      b = better(b, Best{__shfl_xor_sync(0xffffffffu, b.v, o), __shfl_xor_sync(0xffffffffu, b.idx, o)});
    return b;
  };
  // joins the cluster's best entries (every CTA has them all then)
  auto join = [&](Best b, int turn) {
    b = across(b);
    if (lane == 0) s.warp_best[warp] = b;
    __syncthreads();
    if (warp == 0) {
      b = across(lane < kWarps ? s.warp_best[lane] : Best{kMaskedOut, 0x7fffffff});
      if (lane < ranks) cl.map_shared_rank(s.best[turn], lane)[rank] = b;
    }
    cl.sync();
    b = s.best[turn][0];
    for (int q = 1; q < ranks; ++q) b = better(b, s.best[turn][q]);
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
  top = join(top, 0);
  low = s.low[0];
  for (int q = 1; q < ranks; ++q) low = fminf(low, s.low[q]);
  if (top.v == kMaskedOut) {
    only(-1);
    return;
  }
  if (temp == 0.f || k == 1 || tp <= 0.f) {  // the first entry alone
    only(top.idx);
    return;
  }
  if (top.v == __builtin_huge_valf()) {      // its entries share alike, no other stands
    for (int q = 0; q < quads; ++q) {
      float z[4];
      get(q, z);
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] = z[e] == top.v ? 0.f : kMaskedOut;
      mine4[q * kThreads] = make_float4(z[0], z[1], z[2], z[3]);
    }
    top.v = low = 0.f;
  }
  Row r;
  r.top = top.v;
  r.ch = s.ch;
  r.cl = s.cl;
  r.fx = (kBins - 1) / fmaxf(fminf((top.v - low) * r.ch, 64.f), 1e-30f);  // over the row's range, 64 octaves at most
  const bool by_count = k > 0 && k < vocab, by_mass = tp < 1.f;
  const float mp = s.mp;
  const bool by_ratio = mp > 0.f;

  // What stands so far: entries above `border`, and those that equal it up to index `at`. Masked ones never do.
  float border = kMaskedOut;
  int at = -1;
  u64 sum = 0;
  auto stands = [&](int i, float x) { return (x > border) | ((x == border) & (v0 + i <= at)); };
  // Digits 1 and on, for bins with many entries: p[] are those of the entry that is sought.
  int p[kPasses];
  auto digit = [&](int d, int idx, float x) -> int {
    const uint32_t nk = down_key(x);
    return d < 5 ? (int)(nk >> (8 * (4 - d))) & 255 : d == 5 ? idx >> 10 : idx & 1023;
  };
  auto member = [&](int depth, int idx, float x) {
    for (int d = 1; d < depth; ++d)
      if (digit(d, idx, x) != p[d]) return false;
    return true;
  };
  const uint32_t hist = tc::smem_u32(s.cnt);
  auto add_count = [&](int bin, bool one) {
    if (KDA_CHECK(bin >= 0 && bin < kBins)) add_shared<0>(hist + bin * 4, one);
  };
  auto add_mass = [&](int bin, u64 w) {
    if (!KDA_CHECK(bin >= 0 && bin < kBins)) return;
    const uint32_t to = hist + bin * 4, lo = (uint32_t)w;
    add_shared<kBins * 4>(to, lo & 0xffff);
    add_shared<2 * kBins * 4>(to, lo >> 16);
    add_shared<3 * kBins * 4>(to, (uint32_t)(w >> 32));
  };
  auto clear = [&] {
    for (int i = tid; i < kBins; i += kThreads) s.cnt[i] = s.part[0][i] = s.part[1][i] = s.part[2][i] = 0;
    __syncthreads();
  };
  auto sum_of = [&](int bin, bool by) -> u64 {
    return by ? s.part[0][bin] + ((u64)s.part[1][bin] << 16) + ((u64)s.part[2][bin] << 32) : s.cnt[bin];
  };
  // the lane whose entry of sums takes what lies before it up to `target`, and what lies before that
  auto find = [&](u64 v, u64 target, u64& before, u64& total) {
    u64 up_to = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 x = __shfl_up_sync(0xffffffffu, up_to, o);
      if (lane >= o) up_to += x;
    }
    total = __shfl_sync(0xffffffffu, up_to, 31);
    const unsigned hit = __ballot_sync(0xffffffffu, up_to >= target);
    const int at = hit ? __ffs(hit) - 1 : 31;
    before = __shfl_sync(0xffffffffu, up_to - v, at);
    return at;
  };
  // The bin of the cluster's histogram (filled, in each CTA) where the count or the mass reaches `target`, and what
  // lies in it and in the bins before it; -1 if it does not. A target of 0 stands for top-p of all mass, and is
  // set. Of its two cluster barriers the second stands between the reads of `coarse` and what the other CTAs write
  // there in the next search, whose first stands behind the reads of `fine`: every way out passes both.
  u64 inside;
  auto search = [&](bool by, u64& target, u64& before) {
    __syncthreads();
    for (int g = warp; g < kCoarse; g += kWarps) {
      u64 v = sum_of(g * kFine + lane, by);
#pragma unroll
      for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane < ranks) cl.map_shared_rank(&s, lane)->coarse[rank][g] = v;
    }
    cl.sync();
    u64 v = 0, total, rest;
    for (int q = 0; q < ranks; ++q) v += s.coarse[q][lane];
    if (target == 0) {
      find(v, 0, before, total);
      if (tid == 0) {
        const double x = ceil((double)tp * (double)total);
        const u64 t = x < 1. ? 1 : (u64)x;
        s.target = t < total ? t : total;
      }
      __syncthreads();
      target = s.target;
    }
    const int g = find(v, target, before, total);
    if (total < target) {
      cl.sync();
      return -1;
    }
    if (warp < ranks) cl.map_shared_rank(&s, warp)->fine[rank][lane] = sum_of(g * kFine + lane, by);
    cl.sync();
    v = 0;
    for (int q = 0; q < ranks; ++q) v += s.fine[q][lane];
    const int b = find(v, target - before, rest, total);
    inside = __shfl_sync(0xffffffffu, v, b);
    before += rest;
    return g * kFine + b;
  };
  // The cluster's entries that are `wanted`, in bins up to `bin` (from `bin` on, if only that is), into every CTA's
  // s.all with their masses (or ones); their number, which may be too large for that.
  auto collect = [&](int bin, bool only_that, bool masses, auto wanted) {
    if (tid == 0) s.n = 0;
    __syncthreads();
#pragma unroll 2
    for (int q = 0; q < quads; ++q) {
      float z[4];
      get(q, z);
      int hits = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = distance(r, z[e]);
        hits |= (int)(only_that ? d == bin : d <= bin) << e;
      }
      while (hits) {
        const int e = __ffs(hits) - 1, i = place(q) + e;
        hits &= hits - 1;
        const float x = e == 0 ? z[0] : e == 1 ? z[1] : e == 2 ? z[2] : z[3];
        if (!stands(i, x) || !wanted(i, x)) continue;
        const int at = atomicAdd(&s.n, 1);
        if (at < kList) s.list[at] = Item{down_key(x), v0 + i, masses ? mass<false>(r, x, table) : 1};
      }
    }
    __syncthreads();
    if (tid < ranks) cl.map_shared_rank(&s, tid)->counts[rank] = s.n;
    cl.sync();
    int n = 0;
    for (int q = 0; q < ranks; ++q) n += s.counts[q];
    if (n > kList) return n;
    for (int i = tid; i < n; i += kThreads) {
      int q = 0, j = i;
      while (j >= s.counts[q]) j -= s.counts[q++];
      if (KDA_CHECK(i < kList && q < ranks)) s.all[i] = cl.map_shared_rank(&s, q)->list[j];
    }
    __syncthreads();
    return n;
  };
  // Cuts what stands off behind the entry with which its number, or its mass, reaches `target`, in bin p[0] with
  // `before` in the bins before it; the mass up to and with that entry is in `sum` then (by mass).
  auto cut = [&](bool by, u64 target, u64 before) {
    int depth = 1, n;   // before: what lies before the entries whose digits are p[0] .. p[depth - 1]
    for (;;) {
      n = collect(p[0], true, by, [&](int i, float x) { return member(depth, v0 + i, x); });
      if (n <= kList) break;
      // too many: their next digit
      clear();
      for (int q = 0; q < quads; ++q) {
        float z[4];
        get(q, z);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = place(q) + e;
          if (distance(r, z[e]) != p[0] || !stands(i, z[e]) || !member(depth, v0 + i, z[e])) continue;
          if (by) add_mass(digit(depth, v0 + i, z[e]), mass<false>(r, z[e], table));
          else add_count(digit(depth, v0 + i, z[e]), true);
        }
      }
      u64 rest = target - before, low_part;
      p[depth++] = search(by, rest, low_part);
      before += low_part;
    }
    // each CTA ranks its share of them, several lanes an entry where that is little
    const u64 want = target - before;
    const int each = (n + ranks - 1) / ranks, first = rank * each, end = first + each < n ? first + each : n;
    const int share = each <= kThreads / 16 ? 16 : each <= kThreads / 8 ? 8 : each <= kThreads / 4 ? 4 : 1;
    for (int i0 = first; i0 < end; i0 += kThreads / share) {
      const int i = i0 + tid / share;
      const Item it = s.all[i < end ? i : first];
      u64 was = 0;
#pragma unroll 4
      for (int j = tid % share; j < n; j += share) {
        const Item o = s.all[j];
        if (o.nk < it.nk || (o.nk == it.nk && o.idx < it.idx)) was += o.w;
      }
      for (int o = 1; o < share; o *= 2) was += __shfl_xor_sync(0xffffffffu, was, o);
      if (i < end && tid % share == 0 && was < want && want <= was + it.w) {
        for (int q = 0; q < ranks; ++q) {
          Shared* o = cl.map_shared_rank(&s, q);
          o->nk = it.nk;
          o->idx = it.idx;
          o->mass_incl = before + was + it.w;
        }
      }
    }
    cl.sync();
    border = value_of(s.nk);
    at = s.idx;
    sum = s.mass_incl;
  };

  // what stands into a histogram, by number or by mass (with nothing cut off yet, masked entries have none: 260 us
  // for 320 x 131072 probabilities, 265 where each entry is asked)
  auto masses = [&](auto cut_off) {
#pragma unroll 2
    for (int q = 0; q < quads; ++q) {
      float z[4];
      get(q, z);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const u64 w = mass<true>(r, z[e], table);
        add_mass(distance(r, z[e]), !cut_off || stands(place(q) + e, z[e]) ? w : 0);
      }
    }
  };
  auto histogram = [&](bool by) {
    clear();
    if (by) {
      if (border == kMaskedOut) masses(std::false_type());
      else masses(std::true_type());
    } else {
#pragma unroll 2
      for (int q = 0; q < quads; ++q) {
        float z[4];
        get(q, z);
#pragma unroll
        for (int e = 0; e < 4; ++e) add_count(distance(r, z[e]), stands(place(q) + e, z[e]));
      }
    }
  };
  const float* const draw = kProbs ? nullptr : noise + (int64_t)row * noise_pitch;
  bool known = false;    // the mass of what stands, in `sum`
  u64 target, before;
  bool mass_cut = by_mass;
  if (by_count) {
    histogram(false);
    target = (u64)k;
    p[0] = search(false, target, before);
    const u64 up_to = before + inside;
    if (p[0] >= 0 && up_to <= kFew && up_to * up_to <= (u64)kPairs * kThreads * ranks) {
      // Few entries up to that bin: they are ranked by number and mass at once, each CTA its share, an entry or less a
      // thread, and all that follows is asked of them alone. (64 x 131072: 53 us, all by histograms of masses 70. One
      // CTA a row, 320 x 1000, ranking 400 entries: 51 us, by masses 25.)
      const int n = collect(p[0], false, true, [](int, float) { return true; });
      const int each = (n + ranks - 1) / ranks, first = rank * each, end = first + each < n ? first + each : n;
      static_assert(kFew <= kThreads && kFew <= kList, "a lane an entry at least");
      const int share = each <= kThreads / 16 ? 16 : each <= kThreads / 8 ? 8 : each <= kThreads / 4 ? 4
                        : each <= kThreads / 2 ? 2 : 1;
      const int i = first + tid / share;
      const bool lead = i < end && tid % share == 0;
      const Item it = s.all[i < end ? i : 0];
      int ahead = 0;
      u64 was = 0;
#pragma unroll 4
      for (int j = tid % share; j < n; j += share) {
        const Item o = s.all[j];
        if (o.nk < it.nk || (o.nk == it.nk && o.idx < it.idx)) {
          ++ahead;
          was += o.w;
        }
      }
      for (int o = 1; o < share; o *= 2) {
        ahead += __shfl_xor_sync(0xffffffffu, ahead, o);
        was += __shfl_xor_sync(0xffffffffu, was, o);
      }
      if (lead && ahead == k - 1)
        for (int q = 0; q < ranks; ++q) cl.map_shared_rank(&s, q)->kth_mass = was + it.w;
      cl.sync();
      if (tid == 0) {
        const double x = ceil((double)tp * (double)s.kth_mass);
        const u64 t = x < 1. ? 1 : (u64)x;
        s.target = t < s.kth_mass ? t : s.kth_mass;
      }
      __syncthreads();
      // (without top-p by number alone: entries below 2^-44 of the largest add no mass, and stand all the same)
      const bool stays = lead && ahead < k && (!by_mass || was < s.target);
      if (!kProbs) {
        Best best{-1.f, 0x7fffffff};
        if (stays) {
          const float pr = weight(r, value_of(it.nk)), u = draw[it.idx];
          if (pr > 0.f && u == u && (!by_ratio || mass_of<false>(r, value_of(it.nk), table).reaches(mp)))
            best = Best{pr / u, it.idx};
        }
        best = join(best, 1);
        if (rank == 0 && tid == 0) token[row] = best.v < 0.f ? -1 : best.idx;
        return;
      }
      if (stays && (by_mass ? was + it.w >= s.target : ahead == k - 1)) {   // the last that does
        for (int q = 0; q < ranks; ++q) {
          Shared* o = cl.map_shared_rank(&s, q);
          o->nk = it.nk;
          o->idx = it.idx;
          o->mass_incl = was + it.w;
        }
      }
      cl.sync();
      border = value_of(s.nk);
      at = s.idx;
      sum = s.mass_incl;
      known = true;
      mass_cut = false;
    } else if (p[0] >= 0) {
      cut(false, target, before);
      __syncthreads();
    }
  }
  if (mass_cut) {
    histogram(true);
    target = 0;
    p[0] = search(true, target, before);
    cut(true, target, before);
    known = true;
  }
  if (kProbs) {
    if (by_ratio || !known) {
      u64 part = 0;
#pragma unroll 2
      for (int q = 0; q < quads; ++q) {
        float z[4];
        get(q, z);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const Mass w = mass_of<true>(r, z[e], table);
          if (stands(place(q) + e, z[e]) && (!by_ratio || w.reaches(mp))) part += w.units();
        }
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
    if (tid == 0) s.inv = (float)((double)kOne / (double)sum);
    __syncthreads();
    const float inv = s.inv;
#pragma unroll 2
    for (int q = 0; q < quads; ++q) {
      float z[4], o[4];
      get(q, z);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o[e] = 0.f;
        if (stands(place(q) + e, z[e]) && (!by_ratio || mass_of<false>(r, z[e], table).reaches(mp)))
          o[e] = weight(r, z[e]) * inv;
      }
      put(q, o);
    }
  } else {
    Best best{-1.f, 0x7fffffff};
    constexpr int kBatch = 4;   // fours whose noise is on its way at once
#pragma unroll 1
    for (int q0 = 0; q0 < quads; q0 += kBatch) {
      float u[kBatch][4];
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        float z[4];
        if (q0 + q < quads) get(q0 + q, z);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = place(q0 + q) + e;
          u[q][e] = __builtin_nanf("");          // a score that is no number never wins
          if (q0 + q < quads && stands(i, z[e])) u[q][e] = draw[v0 + i];
        }
      }
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        float z[4];
        if (q0 + q < quads) get(q0 + q, z);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (u[q][e] != u[q][e]) continue;
          const float pr = weight(r, z[e]);
          if (pr > 0.f && (!by_ratio || mass_of<false>(r, z[e], table).reaches(mp)))
            best = better(best, Best{pr / u[q][e], v0 + place(q0 + q) + e});
        }
      }
    }
    best = join(best, 1);
    if (rank == 0 && tid == 0) token[row] = best.v < 0.f ? -1 : best.idx;
  }
  KDA_DEBUG_FOLD(status);
}

template <typename T, bool kProbs>
cudaError_t launch(const SampleArgs& a, cudaStream_t st) {
  const int vocab = a.d.vocab, rows = a.d.num_rows, sms = gpu_sms(), e = sizeof(T);
  constexpr int kFour = 4 * kThreads;   // entries of a four a thread
  // CTAs a row: as many as leave 32 entries a thread, so that two CTAs fit an SM (320 x 131072 probabilities: 267
  // us, with 64 entries a thread 318); few rows are shared by more, as long as all CTAs fit the GPU at once
  // (64 x 20001, 4 CTAs a row: 29 us, 8: 39) and there is a four of entries for every thread (1 x 32003: 16 us, 2
  // CTAs: 23; 40 x 4000, 2 CTAs: 20 us, 4: 23).
  int ranks = 1;
  while (ranks < kMaxRanks && (vocab > ranks * 8 * kFour ||
                               ((int64_t)rows * ranks <= sms && vocab > ranks * kFour)))
    ranks *= 2;
  const int slice = ((vocab + ranks - 1) / ranks + 3) / 4 * 4, quads = (slice + kFour - 1) / kFour;
  const bool wide = (uintptr_t)a.logits % (4 * e) == 0 && a.d.logits_pitch % 4 == 0 &&
                    (!kProbs || ((uintptr_t)a.probs % 16 == 0 && vocab % 4 == 0));
  auto* kernel = sample_kernel<T, kProbs>;
  const int most = (int)sizeof(Shared) + kMostQuads * kThreads * 16;
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((rows + 1) * ranks));  // (num_rows is at most 2^27)
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared) + (size_t)quads * kThreads * 16;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)ranks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, (const T*)a.logits, a.d.logits_pitch, a.noise, a.d.noise_pitch,
                            a.temperature, a.top_k, a.top_p, a.min_p, a.d.temperature, a.d.top_k, a.d.top_p,
                            a.d.min_p, a.token, a.probs, a.status, rows, vocab, slice, quads, wide);
}

}  // namespace

bool sample_fits(const kda_sample_desc_t& d) {
  return d.vocab <= kMaxRanks * kMostQuads * 4 * kThreads && d.num_rows <= (1 << 27);
}

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t st) {
  if (a.probs) return a.d.dtype == KDA_BF16 ? launch<__nv_bfloat16, true>(a, st) : launch<float, true>(a, st);
  return a.d.dtype == KDA_BF16 ? launch<__nv_bfloat16, false>(a, st) : launch<float, false>(a, st);
}

}  // namespace kda
