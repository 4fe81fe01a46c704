// kda_ssm_tc.cu -- selective state space scan of packed prompts on the tensor cores (tcgen05 +
// TMEM + TMA), bf16 inputs.
//
// Per head, over chunks of L = 64 tokens (g_t = -exp(a_log) d_t <= 0 the log-decay, d_t the step):
//
//   M[t][s] = (c_t . b_s) exp(g_{s+1} + .. + g_t) d_s          s <= t
//   Y = M X + diag(exp(g_1 + .. + g_t)) C S + D X              S the state before the chunk
//   S <- exp(g_1 + .. + g_L) S + sum_s exp(g_{s+1} + .. + g_L) d_s b_s x_s^T
//
// Every exponent is a sum of log-decays of consecutive tokens, so none is positive. Prefixes and
// suffixes are taken over halves of 32 tokens and across halves they add up; within a half the weight of
// s for t is exp((cl_t - cl_s) + log d_s) with cl the prefixes, so that a token's own weight is its step
// however strong the decays are. A log2-decay counts as -256 at least, past which nothing is left of
// anything in fp32: cl stays within 2^13, and a difference of two is off by some 2^-12 at most. A step of
// zero (a padded token) is a zero weight.
//
// A CTA takes 128 value columns of one sequence: two 64-wide heads of a group, or one 128-wide
// head. Transposed accumulators (lanes = value columns) put both heads into one M = 128 product
// with the group's B and C as the shared other operand:
//
//   G [64 t][s]    = C B^T      A = c tile, B = b tile (M = 64: rows 16 q .. on lanes 32 q ..)  N = 64
//   YM [128][t]    = X^T M^T    A = x tile, B = M tile (two 64-wide heads: one product a head,
//                               the other head's rows of A being zeros)                  N = 64
//   YI [128][t]    = S^T C^T    A = S^T as bf16 (TMEM), B = c tile                       N = 64
//   S^T [128][k]  += X'^T B     A = x' (TMEM), B = b tile                                N = K
//
// S^T stays in TMEM in fp32 for the whole sequence. x'_s = exp(..) d_s x_s is fp32; it enters as
// the sum of three bf16 numbers, which hold all its 24 bits (two with a bf16 pool, 2^-16); b is exact in
// bf16. The accumulator cuts each sum of 16 tokens' products, in each part, off to 24 bits: a state that
// fades within some hundred tokens has fp32 accuracy, one that does not is off by up to 3 (T / 16) 2^-23
// of itself after T tokens. M and the copy of S that C reads are rounded to bf16 once each, like the
// output. (The scores as 16 x 16 warp-level products, which need no trip through TMEM, took 2100 cycles a
// chunk against some 500 of the tensor pipe.)
//
// Shared memory's bandwidth is what the products and the warps compete for (with x' as a tile there,
// and x and y read and written by TMEM lane, two bytes at a time, 3350 wavefronts a chunk): x' goes
// from registers to TMEM, and x and y move as 8 x 8 blocks transposed on the way (ldmatrix, stmatrix).
//
// Warps 0-7 (M group): M from the scores, and x'. Warps 8-15 (R group): the state's decay and bf16 copy,
// the output. Warps 16 and 19 issue the tcgen05 products, warp 17 scans the steps (its scheduler has the
// least of M; on the schedulers that have the most, 2 to 4 % slower), warp 18 claims items and moves tiles
// (TMA). What orders them are mbarriers, each wait bounded (a timeout sets KDA_DEVICE_PIPE_TIMEOUT, stops
// the loads, lets what was issued finish and returns). Only T_SU -> R -> T_S -> products of C and x' ->
// T_SU is a chain from chunk to chunk; scans, scores, M and the arithmetic of x' run ahead of it.
//
// 32768 tokens of 32 heads (V = 128) take 236 us, against 109 us for the bytes at a copy's rate: a chunk
// is ~3900 cycles, of which the products take 2100 (one M = 128, N = 64 step of 16 after the other comes
// every 52 cycles, N = 128 every 71, of which the pipe works 32 and 64) and the chain of barriers, TMEM
// reads and writes between them the rest; the schedulers issue on 59 % of the cycles.
//
// What is no number. A zero weight does not hide it in a product, so it stays out of those that would take
// it where the recurrence does not: a step goes to its own head's rows by e and dec alone (scan_steps), an x
// leaves its tile for the product with M (hide_x) and comes back as NaN for the outputs from its token on
// (spoil_x). B and C are a group's, and reach its heads alone.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstddef>
#include <cstring>

#include "kda_internal.cuh"
#include "kda_ssm_plan.cuh"
#include "tc_ptx.cuh"

namespace kda {
namespace {

KDA_DEBUG_FLAG_DEFINE();
using namespace tc;

constexpr int kL = kSsmChunk;   // tokens a chunk
constexpr int kStages = 3;      // chunks of c, b and x tiles in flight
constexpr int kMThreads = 256, kRThreads = 256;
constexpr int kTcThreads = kMThreads + kRThreads + 128;
constexpr int kFacs = 3;        // chunks of steps and decays in flight
constexpr int kItems = 4;       // claimed items in flight
constexpr int kMinPart = 8;     // chunks a sequence is cut into parts of at least, or so

// ---- shared memory (offsets from a 1024-aligned base) -----------------------------------
constexpr uint32_t kTileBytes = 16384;               // [2 halves][64 rows][128 B]
constexpr uint32_t OFF_Z0 = 0;                       // 64 rows of zeros: the half of A before x's
constexpr uint32_t OFF_ST = 8192;
constexpr uint32_t OFF_C = 0, OFF_B = kTileBytes, OFF_X = 2 * kTileBytes;  // within a stage
constexpr uint32_t kStageBytes = 3 * kTileBytes;
constexpr uint32_t OFF_Z1 = OFF_ST + kStages * kStageBytes;  // and the half after
constexpr uint32_t OFF_M = OFF_Z1 + 8192;            // [2 by chunk parity][2 heads][64 t][64 s] (K-major B)
constexpr uint32_t OFF_CTL = OFF_M + 2 * kTileBytes;

// ---- TMEM columns -------------------------------------------------------------------------
constexpr uint32_t TM_S = 0;     // S^T fp32 (128)
constexpr uint32_t TM_SB = 128;  // S^T as bf16 pairs (64)
constexpr uint32_t TM_YI = 192;  // S^T C^T (64)
constexpr uint32_t TM_YM = 256;  // X^T M^T, two buffers of 64 by chunk parity; before it the scores
constexpr uint32_t TM_XP = 384;  // x'^T as bf16 pairs of tokens, 32 columns a part

enum TcBar {
  T_FULL = 0,                    // a stage's tiles have landed
  T_EMPTY = T_FULL + kStages,    // a stage is free: its products are done, its output has left
  T_FAC = T_EMPTY + kStages,     // a chunk's factors are written
  T_FAC_FREE = T_FAC + kFacs,    // ... and read
  T_M = T_FAC_FREE + kFacs,      // M is written (and a partial chunk's rows cleared), by chunk parity
  T_EPI = T_M + 2,               // the output has read YM and YI, by parity
  T_XP = T_EPI + 2,              // x' is written, by parity
  T_S = T_XP + 2,                // S is decayed and its bf16 copy written
  T_Y, T_SU,                     // the products of C and of x' are done
  T_MX,                          // the products of M are done, by parity
  T_G = T_MX + 2,                // the scores are done, by parity
  T_ITEM_FULL = T_G + 2,
  T_ITEM_EMPTY = T_ITEM_FULL + kItems,
  T_DRAIN = T_ITEM_EMPTY + kItems,
  T_COUNT = T_DRAIN + 2
};

struct Item {
  int32_t h0, nchunks, done;
  int32_t part;       // -1: a whole sequence; else the part's slot of the split scratch
  int32_t last;       // of the sequence's parts (1 for a whole one)
  int64_t bos, eos;   // its tokens
  int64_t state;      // element offset of head h0's state in the initial and final states
};

// Steps and decays of a chunk, by [head of the item][token], logarithms to base 2; a half is 32 tokens.
struct Factors {
  alignas(16) float cl[2][kL];  // log-decay from the half's start through t
  float step[2][kL];   // log d_s: + cl_t - cl_s is the weight of s for t in its half
  float later[2][kL];  // log d_s + log-decay after s to its half's end: + cl_t for t in the next
  float e[2][kL];      // decay from the chunk's start through t
  float to_end[2][kL];  // weight of s in the state after the chunk
  float dec[2];        // decay of the chunk
};

struct Ctl {
  uint64_t bar[T_COUNT];
  Item ring[kItems];
  Factors fac[kFacs];
  uint64_t wait_limit_ns;
  uint32_t* status;
  uint32_t tmem_base;
  uint32_t abort;
  uint32_t poll;            // waits poll: the limit is below what try_wait may suspend a thread for
  alignas(16) float none[kL / 2];  // zeros: what `later` takes in the place of cl_s
  // x that is no number, by chunk parity: whether 32 value columns (a quadrant) and 32 tokens hold any (set by
  // hide_x, cleared by spoil_x), and if so each column's first of those tokens (kL: none)
  alignas(8) uint8_t odd[2][4][2];
  uint8_t first[2][2][128];
};
constexpr uint32_t kTcSmem = OFF_CTL + ((sizeof(Ctl) + 15) & ~15u);
static_assert(kStages == 3, "the loader keeps three outputs");
static_assert(kTcSmem <= 232448, "shared memory budget exceeded");

struct ScanParams {
  CUtensorMap tm_x, tm_b, tm_c, tm_y;
  const __nv_bfloat16* dt;
  int64_t dt_pitch;
  const float *a_log, *dt_bias, *d;
  const int32_t *cu, *idx;
  const void* state_in;
  void* state_out;
  __nv_bfloat16* y;
  uint32_t* status;
  uint32_t* next_item;
  const Entry* list;           // null: sequences in order
  const uint32_t* entries;     // of the list
  float* scratch;              // [part][H][K][V]: the state before each part of a cut sequence
  float* decay;                // [part][H]: a part's decay
  uint64_t wait_limit_ns;
  int32_t N, H, G, V, pairs;   // pairs: items a sequence
  int64_t T, num_slots, slot_stride;
};

__device__ __forceinline__ bool tc_aborted(const Ctl* c) {
  return *reinterpret_cast<const volatile uint32_t*>(&c->abort) != 0u;
}
extern __shared__ __align__(1024) uint8_t ssm_smem[];
__device__ __forceinline__ Ctl* ctl() { return reinterpret_cast<Ctl*>(ssm_smem + OFF_CTL); }

// Bounded wait; after a timeout anywhere in the CTA every wait gives up soon (false). A few tests catch
// what completes at once (252 -> 239 us for 32768 tokens of 32 heads, with the M blocks of 32 columns);
// then the hardware suspends the thread in try_wait until the phase completes or some microseconds have
// passed, so that a waiting warp takes few issue slots; a limit shorter than that polls instead. Out of line, as is
// what else the chunk loop runs at several places: the warps of a CTA run five programs at once, and
// their instruction cache is what they are short of (see the launch).
__device__ __noinline__ bool tc_wait_slow(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
  for (int i = 0; i < 8; ++i)
    if (mbar_test_wait(bar, parity)) return true;
  Ctl* c = ctl();
  uint64_t t0 = 0;
  for (;;) {
    if (c->poll ? mbar_test_wait(bar, parity) : mbar_try_wait_sleep(bar, parity, kSleepHintNs)) return true;
    if (tc_aborted(c)) return false;
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > c->wait_limit_ns) {
      if (atomicExch(&c->abort, 1u) == 0u) raise_status(c->status, KDA_DEVICE_PIPE_TIMEOUT);
      return false;
    }
  }
}
__device__ __forceinline__ bool tc_wait(int b, uint32_t parity) {
  uint64_t* bar = &ctl()->bar[b];
  if (mbar_test_wait(bar, parity)) return true;
  return tc_wait_slow(bar, parity);
}
// Several at once: what is usually complete already costs one test each and one branch. (None of this
// may need a stack: with 200 KB of shared memory taken, local memory is an L2 trip away.)
struct At {
  int b;
  uint32_t parity;
};
__device__ __forceinline__ bool tc_wait2(At x, At y) {
  uint64_t* bar = ctl()->bar;
  const bool a = mbar_test_wait(bar + x.b, x.parity), b = mbar_test_wait(bar + y.b, y.parity);
  if ((int)a & (int)b) return true;
  return tc_wait_slow(bar + x.b, x.parity) && tc_wait_slow(bar + y.b, y.parity);
}
__device__ __forceinline__ bool tc_wait3(At x, At y, At z) {
  uint64_t* bar = ctl()->bar;
  const bool a = mbar_test_wait(bar + x.b, x.parity), b = mbar_test_wait(bar + y.b, y.parity);
  const bool d = mbar_test_wait(bar + z.b, z.parity);
  if ((int)a & (int)b & (int)d) return true;
  return tc_wait_slow(bar + x.b, x.parity) && tc_wait_slow(bar + y.b, y.parity) &&
         tc_wait_slow(bar + z.b, z.parity);
}
// The lanes' common result: after a timeout the warp leaves as one.
__device__ __forceinline__ bool all_lanes(bool ok) { return __all_sync(0xffffffffu, ok) != 0; }
// One arrival a warp, after what its lanes wrote.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// A shared-memory descriptor as two words: tiles and k-steps differ in the low one alone, so that an
// unrolled run of products needs one addition an operand.
struct Desc {
  uint32_t lo, hi;
};
__device__ __forceinline__ Desc desc128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  const uint64_t d = sdesc_sw128(saddr, lbo, sbo);
  return {(uint32_t)d, (uint32_t)(d >> 32)};
}
// Four k-steps of a product, A and B from shared memory, their descriptors a_step and b_step apart;
// `acc`: the first step adds to D too.
__device__ __forceinline__ void issue_ss(uint32_t d, Desc a, uint32_t a_step, Desc b, uint32_t b_step,
                                      uint32_t idesc, uint32_t acc) {
#pragma unroll
  for (int ks = 0; ks < 4; ++ks)
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %6, 0;\n mov.b64 x, {%1, %2};\n"
        " mov.b64 y, {%3, %4};\n tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n}\n" ::"r"(d),
        "r"(a.lo + ks * (a_step >> 4)), "r"(a.hi), "r"(b.lo + ks * (b_step >> 4)), "r"(b.hi), "r"(idesc),
        "r"(ks ? 1u : acc)
        : "memory");
}
// The same with A in TMEM, 8 columns a k-step.
__device__ __forceinline__ void issue_ts(uint32_t d, uint32_t a_tmem, Desc b, uint32_t b_step, uint32_t idesc,
                                      uint32_t acc) {
#pragma unroll
  for (int ks = 0; ks < 4; ++ks)
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.b32 p, %5, 0;\n mov.b64 y, {%2, %3};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n}\n" ::"r"(d),
        "r"(a_tmem + ks * 8), "r"(b.lo + ks * (b_step >> 4)), "r"(b.hi), "r"(idesc), "r"(ks ? 1u : acc)
        : "memory");
}

// Four 8 x 8 blocks of 16-bit elements, transposed: lanes 8 m .. 8 m + 7 give the 16-byte rows of
// block m; lane l has elements (2 (l % 4), + 1) of the row l / 4 of each transposed block.
__device__ __forceinline__ void ldsm_x4_trans(uint32_t (&r)[4], uint32_t saddr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(saddr)
               : "memory");
}
__device__ __forceinline__ void stsm_x4(uint32_t saddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(saddr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void stsm_x4_trans(uint32_t saddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(saddr), "r"(a),
               "r"(b), "r"(c), "r"(d)
               : "memory");
}
// TMEM as the same blocks, 16 lanes at a time: 32 fp32 columns (register 4 c + 2 h + i: lane
// l / 4 + 8 h, column 8 c + 2 (l % 4) + i), or 16 columns of pairs (2 c + h: lane l / 4 + 8 h, column
// 4 c + l % 4).
__device__ __forceinline__ void tmem_ld_16x256_x4(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15},"
      " [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st_16x128_x4(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// Reads ring entry k (whole warp, uniform result) and releases it.
__device__ __forceinline__ Item tc_item_warp(const ScanParams& p, Ctl* c, uint32_t k) {
  const int slot = k % kItems;
  const bool ok = tc_wait(T_ITEM_FULL + slot, (k / kItems) & 1);
  Item it = c->ring[slot];
  const bool stop = !all_lanes(ok && it.done == 0);
  __syncwarp();
  if (ok && (threadIdx.x & 31) == 0) mbar_arrive(&c->bar[T_ITEM_EMPTY + slot]);
  it.done = stop ? 1 : 0;
  return it;
}


// ---- warp 18: items and tiles ------------------------------------------------------------
template <int K, bool kState>
__device__ void run_loader(const ScanParams& p, uint8_t* sm, Ctl* c) {
  if (!elect_one()) return;
  const uint32_t total = (p.list ? *p.entries : (uint32_t)p.N) * (uint32_t)p.pairs;
  const int rep = p.H / p.G;                       // heads a group
  const int per = p.V == 64 ? (rep + 1) / 2 : rep; // items a group
  uint32_t j = 0;                                  // chunks loaded by this CTA
  // what the chunks in the stages leave as: column, first token, halves (0: stored by the R group)
  struct Out {
    int col, t0, halves;
  } out[kStages] = {};
  // stage st (chunk i of the CTA) is done with: its output leaves, and it is free once that was read
  auto leave = [&](uint32_t i) -> bool {
    const uint32_t st = i % kStages;
    if (!tc_wait(T_EMPTY + st, (i / kStages) & 1)) return false;
    const Out o = st == 0 ? out[0] : st == 1 ? out[1] : out[2];
    if (o.halves > 0) {
      tma_store_2d(&p.tm_y, sm + OFF_ST + st * kStageBytes + OFF_X, o.col, o.t0);
      if (o.halves > 1) tma_store_2d(&p.tm_y, sm + OFF_ST + st * kStageBytes + OFF_X + 8192, o.col + 64, o.t0);
      bulk_commit();
      bulk_wait_read();
    }
    return true;
  };
  for (uint32_t k = 0;; ++k) {
    Item it{};
    for (;;) {
      const uint32_t w = tc_aborted(c) ? total : atomicAdd(p.next_item, 1u);
      if (w >= total) {
        it.done = 1;
        break;
      }
      const int e = (int)(w / (uint32_t)p.pairs), q = (int)(w % (uint32_t)p.pairs);
      Entry en{e, 0, 0, -1, 1, {0, 0, 0}};
      if (p.list) en = p.list[e];
      int64_t bos, eos;
      if (!seq_bounds(p.cu, en.n, p.T, &bos, &eos)) {
        raise_status(p.status, KDA_DEVICE_BAD_SEQLENS);
        continue;
      }
      int64_t slot = en.n;
      if (p.idx) {
        slot = resolve_slot(p.idx, en.n, p.num_slots);
        if (slot < 0) {
          raise_status(p.status, KDA_DEVICE_BAD_SLOT);
          continue;
        }
      }
      const int g = q / per, i = q % per;
      it.h0 = g * rep + (p.V == 64 ? 2 * i : i);
      it.bos = bos + (int64_t)en.chunk0 * kL;
      const int64_t end = it.bos + (int64_t)en.nchunks * kL;
      it.eos = p.list && end < eos ? end : eos;
      it.nchunks = (int)((it.eos - it.bos + kL - 1) / kL);
      it.part = en.part;
      it.last = en.last;
      it.state = slot * p.slot_stride + (int64_t)it.h0 * K * p.V;
      break;
    }
    const int slot = k % kItems;
    if (k >= (uint32_t)kItems && !tc_wait(T_ITEM_EMPTY + slot, (k / kItems - 1) & 1)) break;
    c->ring[slot] = it;
    mbar_arrive(&c->bar[T_ITEM_FULL + slot]);
    if (it.done) break;
    const int g = it.h0 / rep;
    const bool second = p.V == 128 || (it.h0 % rep) + 1 < rep;
    const uint32_t bytes = (kState ? 1u : 2u) * (K / 64) * 8192u + (second ? 16384u : 8192u);
    // a stage comes free little more than a chunk before its tiles are wanted, less than a load from
    // HBM takes: the tiles are brought into L2 kAhead chunks before
    constexpr int kAhead = 3;
    auto prefetch = [&](int i) {
      const int t0 = (int)(it.bos + (int64_t)(kState ? it.nchunks - 1 - i : i) * kL);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (half < K / 64) {
          if (!kState) tma_prefetch_2d(&p.tm_c, g * K + half * 64, t0);
          tma_prefetch_2d(&p.tm_b, g * K + half * 64, t0);
        }
        if (half == 0 || second) tma_prefetch_2d(&p.tm_x, it.h0 * p.V + half * 64, t0);
      }
    };
#pragma unroll 1
    for (int i = -kAhead; i < it.nchunks; ++i) {
      if (i + kAhead < it.nchunks) prefetch(i + kAhead);
      if (i < 0) continue;
      const int ch = kState ? it.nchunks - 1 - i : i;
      const uint32_t st = j % kStages;
      if (j >= (uint32_t)kStages && !leave(j - kStages)) break;
      if (tc_aborted(c)) break;
      uint8_t* base = sm + OFF_ST + st * kStageBytes;
      uint64_t* bar = &c->bar[T_FULL + st];
      const int t0 = (int)(it.bos + (int64_t)ch * kL);
      mbar_expect_tx(bar, bytes);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (half < K / 64) {
          if (!kState) tma_load_2d(base + OFF_C + half * 8192, &p.tm_c, bar, g * K + half * 64, t0);
          tma_load_2d(base + OFF_B + half * 8192, &p.tm_b, bar, g * K + half * 64, t0);
        }
        if (half == 0 || second)
          tma_load_2d(base + OFF_X + half * 8192, &p.tm_x, bar, it.h0 * p.V + half * 64, t0);
      }
      const Out o{it.h0 * p.V, t0, kState || it.bos + (int64_t)(ch + 1) * kL > it.eos ? 0 : second ? 2 : 1};
      if (st == 0) out[0] = o;
      else if (st == 1) out[1] = o;
      else out[2] = o;
      ++j;
    }
    if (tc_aborted(c)) break;
  }
  // the last outputs; every load that was issued has landed, and every store has been made, before
  // the CTA may leave
  for (uint32_t i = j > (uint32_t)kStages ? j - kStages : 0; i < j; ++i)
    if (!leave(i)) break;
  bulk_wait_all();
  for (uint32_t i = j > (uint32_t)kStages ? j - kStages : 0; i < j; ++i)
    mbar_wait(&c->bar[T_FULL + i % kStages], (i / kStages) & 1);
}

// Two warps issue the products, each for one loop from chunk to chunk: a thread takes ~100 cycles a
// product here, the pipe 52 to 71, and a product never waits for one of the other loop's.

// ---- warp 19: the products of the output ------------------------------------------------------
// One thread, in chunks with an x that is no number, once the product with M is done: NaN stands in the x
// tile from a column's first such token on, so that these outputs become NaN by their D x.
__device__ __noinline__ bool spoil_x(uint32_t j) {
  const uint32_t par = j & 1;
  uint8_t* x = ssm_smem + OFF_ST + j % kStages * kStageBytes + OFF_X;
  Ctl* c = ctl();
  if (!tc_wait(T_MX + (int)par, (j >> 1) & 1)) return false;
  tc_fence_after();
#pragma unroll 1
  for (int v = 0; v < 128; ++v) {
    int r = kL;
    if (c->odd[par][v >> 5][1]) r = c->first[par][1][v];
    if (c->odd[par][v >> 5][0]) r = min(r, (int)c->first[par][0][v]);
#pragma unroll 1
    for (; r < kL; ++r)
      reinterpret_cast<uint16_t*>(x + (v >> 6) * 8192 + sw128_off(r, (v & 63) >> 3))[v & 7] = 0x7fffu;
  }
  *reinterpret_cast<uint64_t*>(c->odd[par]) = 0u;
  __threadfence_block();  // before the R group can see the products of C done
  return true;
}

template <int K>
__device__ void run_output(const ScanParams& p, uint8_t* sm, Ctl* c, uint32_t tbase) {
  if (!elect_one()) return;
  const uint32_t sbase = smem_u32(sm);
  const int rep = p.H / p.G;
  const uint32_t id_m = idesc_bf16(128, kL, 1, 0), id_c = idesc_bf16(128, kL, 0, 0);
  uint32_t j = 0;
  bool ok = true;
  for (uint32_t k = 0; ok; ++k) {
    const int slot = k % kItems;
    ok = tc_wait(T_ITEM_FULL + slot, (k / kItems) & 1);
    if (!ok) break;
    const int nchunks = c->ring[slot].nchunks, done = c->ring[slot].done;
    const bool second = p.V == 64 && (c->ring[slot].h0 % rep) + 1 < rep;
    mbar_arrive(&c->bar[T_ITEM_EMPTY + slot]);
    if (done) break;
    for (int ch = 0; ch < nchunks; ++ch, ++j) {
      const uint32_t st = j % kStages, stage = sbase + OFF_ST + st * kStageBytes;
      ok = tc_wait2({T_M + (int)(j & 1), (j >> 1) & 1}, {T_FULL + (int)st, (j / kStages) & 1});
      if (!ok) break;
      tc_fence_after();
      const uint32_t ym = tbase + TM_YM + (j & 1) * 64, m = sbase + OFF_M + (j & 1) * kTileBytes;
      // the second half of A: x's, or zeros where it is another head's
      const uint32_t x0 = stage + OFF_X;
      issue_ss(ym, desc128(x0, p.V == 128 ? 8192 : sbase + OFF_Z1 - x0, 1024), 2048,
               desc128(m, 16, 1024), 32, id_m, 0);
      if (second)
        issue_ss(ym, desc128(sbase + OFF_Z0, x0 + 8192 - (sbase + OFF_Z0), 1024), 2048,
                 desc128(m + 8192, 16, 1024), 32, id_m, 1);
      mma_commit(&c->bar[T_MX + (j & 1)]);
      if (*reinterpret_cast<const uint64_t*>(c->odd[j & 1]) != 0u) ok = spoil_x(j);
      ok = ok && tc_wait(T_S, j & 1);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (uint32_t kh = 0; kh < K / 64; ++kh)
        issue_ts(tbase + TM_YI, tbase + TM_SB + kh * 32, desc128(stage + OFF_C + kh * 8192, 16, 1024), 32, id_c,
                 kh);
      mma_commit(&c->bar[T_Y]);
    }
  }
  mma_commit(&c->bar[T_DRAIN]);
  mbar_wait(&c->bar[T_DRAIN], 0);  // the full limit, aborted or not
}

// ---- warp 16: the state's product, and the scores of the chunk after next ------------------------
template <int K, int PARTS>
__device__ void run_state(uint8_t* sm, Ctl* c, uint32_t tbase) {
  if (!elect_one()) return;
  const uint32_t sbase = smem_u32(sm);
  const uint32_t id_g = idesc_bf16(64, kL, 0, 0), id_s = idesc_bf16(128, K, 0, 1);  // A in TMEM: K-major
  // The scores run up to two chunks ahead, within this item and the next: `kg`, `cg`, `jg` are the
  // item, its chunk and the CTA's chunk they come to next (ng: that item's chunks, -1: not read).
  uint32_t j = 0, kg = 0, jg = 0;
  int cg = 0, ng = -1;
  bool more = true, ok = true;
  auto scores = [&](uint32_t k, uint32_t upto) {
    while (ok && more && jg < upto) {
      if (cg >= ng) {
        if (kg > k) return;
        ok = tc_wait(T_ITEM_FULL + (kg + 1) % kItems, ((kg + 1) / kItems) & 1);
        if (!ok) return;
        ++kg;
        cg = 0;
        ng = c->ring[kg % kItems].nchunks;
        more = c->ring[kg % kItems].done == 0;
        continue;
      }
      const uint32_t st = jg % kStages, stage = sbase + OFF_ST + st * kStageBytes;
      const At full{T_FULL + (int)st, (jg / kStages) & 1};
      ok = jg < 2 ? tc_wait(full.b, full.parity)
                  : tc_wait2(full, {T_EPI + (int)(jg & 1), ((jg >> 1) - 1) & 1});
      if (!ok) return;
      tc_fence_after();
#pragma unroll
      for (uint32_t kh = 0; kh < K / 64; ++kh)
        issue_ss(tbase + TM_YM + (jg & 1) * 64, desc128(stage + OFF_C + kh * 8192, 16, 1024), 32,
                 desc128(stage + OFF_B + kh * 8192, 16, 1024), 32, id_g, kh);
      mma_commit(&c->bar[T_G + (jg & 1)]);
      ++cg;
      ++jg;
    }
  };
  for (uint32_t k = 0; ok; ++k) {
    const int slot = k % kItems;
    ok = tc_wait(T_ITEM_FULL + slot, (k / kItems) & 1);
    if (!ok) break;
    const int nchunks = c->ring[slot].nchunks, done = c->ring[slot].done;
    if (done) break;
    if (ng < 0 || kg < k) {  // nothing left to run ahead with before this item
      kg = k;
      cg = 0;
      ng = nchunks;
    }
    for (int ch = 0; ch < nchunks && ok; ++ch, ++j) {
      const uint32_t st = j % kStages, stage = sbase + OFF_ST + st * kStageBytes;
      scores(k, j + 2);  // which have seen b's tile land
      ok = ok && tc_wait2({T_XP + (int)(j & 1), (j >> 1) & 1}, {T_S, j & 1});
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (uint32_t part = 0; part < PARTS; ++part)
        issue_ts(tbase + TM_S, tbase + TM_XP + part * 32, desc128(stage + OFF_B, 8192, 1024), 2048, id_s, 1);
      mma_commit(&c->bar[T_SU]);
      mma_commit(&c->bar[T_EMPTY + st]);
    }
    mbar_arrive(&c->bar[T_ITEM_EMPTY + slot]);
  }
  mma_commit(&c->bar[T_DRAIN + 1]);
  mbar_wait(&c->bar[T_DRAIN + 1], 0);
}

// ---- warp 17: steps and decays ------------------------------------------------------------------
// softplus(x) = max(x, 0) + log(1 + e^-|x|), the logarithm as 2 atanh(u / (2 + u)) with u = e^-|x|:
// u / (2 + u) <= 1/3, so that seven terms of the series leave a relative error of 2e-8, at small u too.
// One warp makes the steps of all others' chunks, a thousand dependent cycles with the library's
// functions; good to ~4e-7 with the fast exponential and quotient. The exponent -|x| log2 e is rounded to 24
// bits, which alone would be 4e-6 at |x| = 80: u takes what the rounding left out as a factor.
__device__ __forceinline__ float softplus_fast(float x) {
  const float a = fmaxf(-fabsf(x), -150.f);  // u is zero from -88 on
  const float hi = a * 1.44269502f;
  float u = ex2(hi);
  u = fmaf(u, fmaf(hi, -0.693147182f, a), u);
  const float z = __fdividef(u, 2.f + u), q = z * z;
  float s = fmaf(q, 1.f / 13.f, 1.f / 11.f);
  s = fmaf(q, s, 1.f / 9.f);
  s = fmaf(q, s, 1.f / 7.f);
  s = fmaf(q, s, 1.f / 5.f);
  s = fmaf(q, s, 1.f / 3.f);
  s = fmaf(q, s, 1.f);
  float top;  // max(x, 0), NaN if x is
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(top) : "f"(x));
  return top + 2.f * z * s;
}

// Steps and decays of chunk j of the CTA, for kHeads heads side by side; lane l has tokens 2 l and 2 l + 1.
// They are complete in registers before their place is waited for, as the wait's end is what the M group
// waits for (243 -> 235 us for 32768 tokens of 32 heads). M has to stay finite for the other head of its
// product, whose rows meet zeros of A: a step that is no number is left out of the weights (a step of zero),
// and from its token on the outputs and the state of its own head become NaN by e and dec instead.
template <int kHeads>
__device__ __forceinline__ bool scan_steps(Ctl* c, uint32_t j, float (&d)[2][2], const float (&rate2)[2], int lane) {
  const uint32_t fi = j % kFacs;
  Factors* f = &c->fac[fi];
  float g0[kHeads], g1[kHeads], up[kHeads], dn[kHeads];
  uint32_t bad[kHeads];  // lanes with such a step
  bool bad0[kHeads];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    bad0[h] = !(d[h][0] < INFINITY);
    const bool bad1 = !(d[h][1] < INFINITY);
    bad[h] = __ballot_sync(0xffffffffu, bad0[h] || bad1);
    d[h][0] = bad0[h] ? 0.f : d[h][0];
    d[h][1] = bad1 ? 0.f : d[h][1];
    g0[h] = rate2[h] * d[h][0];  // log2-decays
    g1[h] = rate2[h] * d[h][1];
    g0[h] = fmaxf(g0[h], -256.f);
    g1[h] = fmaxf(g1[h], -256.f);
    up[h] = dn[h] = g0[h] + g1[h];  // inclusive sums over the half's 16 lanes, from either end
  }
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) {
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      const float a = __shfl_up_sync(0xffffffffu, up[h], o, 16);
      const float b = __shfl_down_sync(0xffffffffu, dn[h], o, 16);
      if ((lane & 15) >= o) up[h] += a;
      if ((lane & 15) + o < 16) dn[h] += b;
    }
  }
  float2 cl[kHeads], step[kHeads], later[kHeads], e[kHeads], to_end[kHeads];
  float dec[kHeads];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    float before = __shfl_up_sync(0xffffffffu, up[h], 1, 16);
    float after = __shfl_down_sync(0xffffffffu, dn[h], 1, 16);
    if ((lane & 15) == 0) before = 0.f;
    if ((lane & 15) == 15) after = 0.f;
    const float first = __shfl_sync(0xffffffffu, up[h], 15), second = __shfl_sync(0xffffffffu, up[h], 31);
    const float pre = lane < 16 ? 0.f : first;
    const float c0 = before + g0[h], c1 = up[h];
    const float l0 = __log2f(d[h][0]), l1 = __log2f(d[h][1]);  // -inf for a step of zero: no weight
    cl[h] = make_float2(c0, c1);
    step[h] = make_float2(l0, l1);
    later[h] = make_float2(l0 + (after + g1[h]), l1 + after);
    e[h] = make_float2((bad[h] & ((1u << lane) - 1)) || bad0[h] ? NAN : ex2(pre + c0),
                       bad[h] & ((2u << lane) - 1) ? NAN : ex2(pre + c1));
    const float then = lane < 16 ? second : 0.f;
    to_end[h] = make_float2(d[h][0] * ex2(after + g1[h] + then), d[h][1] * ex2(after + then));
    dec[h] = bad[h] ? NAN : ex2(first + second);
  }
  if (j >= (uint32_t)kFacs && !all_lanes(tc_wait(T_FAC_FREE + fi, (j / kFacs - 1) & 1))) return false;
  const int t = 2 * lane;
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    *reinterpret_cast<float2*>(&f->cl[h][t]) = cl[h];
    *reinterpret_cast<float2*>(&f->step[h][t]) = step[h];
    *reinterpret_cast<float2*>(&f->later[h][t]) = later[h];
    *reinterpret_cast<float2*>(&f->e[h][t]) = e[h];
    *reinterpret_cast<float2*>(&f->to_end[h][t]) = to_end[h];
    if (lane == 0) f->dec[h] = dec[h];
  }
  return true;
}

template <int kHeads>
__device__ void run_scan_heads(const ScanParams& p, Ctl* c) {
  const int lane = threadIdx.x & 31, rep = p.H / p.G;
  uint32_t j = 0;
  for (uint32_t k = 0;; ++k) {
    const Item it = tc_item_warp(p, c, k);
    if (it.done) return;
    const bool second = kHeads == 2 && (it.h0 % rep) + 1 < rep;
    float rate2[2] = {0.f, 0.f}, bias[2] = {0.f, 0.f};
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      if (h == 1 && !second) break;
      rate2[h] = ssm_rate(p.a_log[it.h0 + h], 1.4426950408889634f);
      bias[h] = p.dt_bias ? p.dt_bias[it.h0 + h] : 0.f;
      if (isnan(rate2[h])) {  // then no step is a number
        rate2[h] = 0.f;
        bias[h] = NAN;
      }
    }
    // the steps of a chunk are read two scans ahead; -inf: no token, a step of zero
    const __nv_bfloat16* at = p.dt + (it.bos + 2 * lane) * p.dt_pitch + it.h0;
    int left = (int)(it.eos - it.bos) - 2 * lane;
    auto read = [&](float (&n)[2][2]) {
#pragma unroll
      for (int h = 0; h < kHeads; ++h) {
        n[h][0] = left > 0 && (h == 0 || second) ? to_f32(at[h]) : -INFINITY;
        n[h][1] = left > 1 && (h == 0 || second) ? to_f32(at[p.dt_pitch + h]) : -INFINITY;
      }
      at += kL * p.dt_pitch;
      left -= kL;
    };
    float cur[2][2], nxt[2][2], d[2][2];
    read(cur);
    read(nxt);
#pragma unroll 1
    for (int ch = 0; ch < it.nchunks; ++ch, ++j) {
      const uint32_t fi = j % kFacs;
#pragma unroll
      for (int h = 0; h < kHeads; ++h) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          d[h][i] = softplus_fast(cur[h][i] + bias[h]);
          cur[h][i] = nxt[h][i];
        }
      }
      read(nxt);
      if (!scan_steps<kHeads>(c, j, d, rate2, lane)) return;
      warp_arrive(&c->bar[T_FAC + fi]);
    }
  }
}
__device__ void run_scan(const ScanParams& p, Ctl* c) {
  if (p.V == 64) run_scan_heads<2>(p, c);
  else run_scan_heads<1>(p, c);
}

// ---- warps 0-7: M and x' ------------------------------------------------------------------------
// Two values of x' as PARTS bf16 numbers each: truncated parts leave exact remainders.
template <int PARTS>
__device__ __forceinline__ void split_x(uint32_t raw, float2 w, uint32_t (&out)[PARTS]) {
  float a = bf_lo(raw), b = bf_hi(raw);
  mul2(a, b, w.x, w.y);
#pragma unroll
  for (int q = 0; q < PARTS; ++q) {
    if (q == PARTS - 1) {
      out[q] = pack_bf16x2(a, b);
    } else {
      const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
      out[q] = __byte_perm(ua, ub, 0x7632);
      // a - trunc(a), exact
      sub2(a, b, __uint_as_float(ua & 0xffff0000u), __uint_as_float(ub & 0xffff0000u));
    }
  }
}

// The lane's part of 32 value columns and 32 tokens of the x tile, as 8 x 8 blocks: columns 16 (i / 2),
// tokens 16 (i % 2).
__device__ __forceinline__ void load_x(uint32_t (&raw)[4][4], uint32_t tile, uint32_t col0) {
#pragma unroll
  for (int i = 0; i < 4; ++i) ldsm_x4_trans(raw[i], tile + (i & 1) * 2048 + ((col0 ^ (i & 2)) << 4));
}
// Whether any of those is no number: zero times it is not zero.
__device__ __forceinline__ bool not_finite(const uint32_t (&raw)[4][4]) {
  uint32_t z[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(z[i & 3]) : "r"(raw[i >> 2][i & 3]), "r"(0u));
  return ((z[0] | z[1] | z[2] | z[3]) & 0x7fff7fffu) != 0u;
}
// Its treatment in chunk j of the CTA, for the warp's 32 columns (lane: column) and 32 rows. A zero weight of
// M would not hide it from the tokens before it: zeros take its place for the product with M (x' has been
// read), then spoil_x makes up for it.
__device__ __noinline__ void hide_x(uint32_t j) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = warp & 3, th = warp >> 2;
  uint8_t* half = ssm_smem + OFF_ST + j % kStages * kStageBytes + OFF_X + (quad >> 1) * 8192;
  int first = kL;
#pragma unroll 1
  for (int r = th * 32 + 31; r >= th * 32; --r) {
    uint16_t* p = reinterpret_cast<uint16_t*>(half + sw128_off(r, (quad & 1) * 4 + (lane >> 3))) + (lane & 7);
    if ((*p & 0x7f80u) == 0x7f80u) {
      *p = 0;
      first = r;
    }
  }
  Ctl* c = ctl();
  c->first[j & 1][th][quad * 32 + lane] = (uint8_t)first;
  if (lane == 0) c->odd[j & 1][quad][th] = 1;
}
// x' of 16 of those columns, and its way to TMEM.
template <int PARTS>
__device__ __forceinline__ void split_half(const uint32_t (&a)[4], const uint32_t (&b)[4], const float2 (&w)[4],
                                           uint32_t (&parts)[PARTS][8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t o[PARTS];
    split_x<PARTS>(i < 4 ? a[i & 3] : b[i & 3], w[i >> 1], o);
#pragma unroll
    for (int q = 0; q < PARTS; ++q) parts[q][i] = o[q];
  }
}
template <int PARTS>
__device__ __forceinline__ void put_half(uint32_t taddr, const uint32_t (&parts)[PARTS][8]) {
#pragma unroll
  for (int q = 0; q < PARTS; ++q) tmem_st_16x128_x4(taddr + q * 32, parts[q]);
}

// 16 x 32 elements of M, 16 a lane: the scores times their weights, rounded into the M tile at `at0` and
// `at1` (the lane's row of the 8 x 8 blocks, of either 16 columns). `col` and `cls`: the lane's columns'
// part of the log-weights and what is taken off for them; `row`: the block's first row, from its first
// column on: columns after the row are not weighted (their weight may be anything) but zero.
__device__ __forceinline__ void weigh_block(uint32_t tmem, const float* col, const float* cls, float cl0, float cl1,
                                            int row, uint32_t at0, uint32_t at1, int lane) {
  float g[16];
  tmem_ld_16x256_x4(tmem, g);
  float w[16];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float2 q = *reinterpret_cast<const float2*>(col + c * 8);
    const float2 s = *reinterpret_cast<const float2*>(cls + c * 8);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float u = r ? cl1 : cl0, v = u;
      sub2(u, v, s.x, s.y);
      add2(u, v, q.x, q.y);
      w[4 * c + 2 * r] = ex2(u);
      w[4 * c + 2 * r + 1] = ex2(v);
    }
  }
  const int last = row + (lane >> 2) - 2 * (lane & 3);
  tmem_ld_wait();
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 16; ++i)  // column 8 (i / 4) + 2 (lane % 4) + i % 2, row lane / 4 + 8 (i / 2 % 2)
    g[i] = (i >> 2) * 8 + (i & 1) - ((i >> 1) & 1) * 8 > last ? 0.f : g[i] * w[i];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = pack_bf16x2(g[2 * i], g[2 * i + 1]);
  stsm_x4(at0, o[0], o[1], o[2], o[3]);
  stsm_x4(at1, o[4], o[5], o[6], o[7]);
}

template <int PARTS>
__device__ void run_mgroup(const ScanParams& p, uint8_t* sm, Ctl* c, uint32_t tbase) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads = p.V == 64 ? 2 : 1;
  // the columns of M after the rows' half are never written again, the zero rows never at all
  for (uint32_t i = threadIdx.x; i < kTileBytes / 16; i += kMThreads) {
    *reinterpret_cast<uint4*>(sm + OFF_M + i * 16) = make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(sm + OFF_M + kTileBytes + i * 16) = make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(sm + (i < 512 ? OFF_Z0 + i * 16 : OFF_Z1 + (i - 512) * 16)) = make_uint4(0, 0, 0, 0);
  }
  if (threadIdx.x < kL / 2) c->none[threadIdx.x] = 0.f;
  if (threadIdx.x < 2) *reinterpret_cast<uint64_t*>(c->odd[threadIdx.x]) = 0u;
  fence_async_smem();
  named_bar(1, kMThreads);

  // x' of 32 value columns (TMEM lanes of the warp's quadrant) and 32 tokens: where the lane's row of
  // the 8 x 8 blocks lies in the x tile, for tokens 0-15 and columns 0-15 of those
  // and M's rows [16 quad, + 16): one head a warp, or one half of the columns of the one head. (Two M
  // tiles in turn, so that M does not wait for the product of the chunk before: 239 -> 235 us.)
  const int quad = warp & 3, th = warp >> 2;
  const int hm = heads == 2 ? th : 0, half0 = heads == 2 ? 0 : th, halfn = heads == 2 ? 1 : 2;
  const uint32_t mrow = quad * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
  const uint32_t m0 = smem_u32(sm) + OFF_M + hm * 8192 + mrow * 128;
  const uint32_t row0 = th * 4096 + ((lane >> 4) << 10) + (lane & 7) * 128;
  const uint32_t col0 = ((quad & 1) * 4 + ((lane >> 3) & 1)) ^ (lane & 7);  // 16-byte cell
  const uint32_t xoff = OFF_X + (quad >> 1) * 8192 + row0;
  const uint32_t txp = tbase + TM_XP + th * 16 + ((uint32_t)(quad * 32) << 16);
  const int hx = heads == 2 ? quad >> 1 : 0;
  const int rep = p.H / p.G;
  uint32_t j = 0;
  for (uint32_t k = 0;; ++k) {
    const Item it = tc_item_warp(p, c, k);
    if (it.done) return;
    const bool real = hx == 0 || (it.h0 % rep) + 1 < rep;  // else its half of x's tile is nobody's
    for (int ch = 0; ch < it.nchunks; ++ch, ++j) {
      const uint32_t st = j % kStages, par = j & 1, fi = j % kFacs;
      uint8_t* stage = sm + OFF_ST + st * kStageBytes;
      const Factors* f = &c->fac[fi];
      // (the scores: their tiles have landed. j > 1: the product that read the M before last is done.)
      const At g{T_G + (int)par, (j >> 1) & 1};
      if (!all_lanes(tc_wait3({T_FAC + (int)fi, (j / kFacs) & 1}, g,
                              j > 1 ? At{T_MX + (int)par, ((j >> 1) - 1) & 1} : g) &&
                     tc_wait(T_FULL + st, (j / kStages) & 1)))
        return;
      tc_fence_after();
      // the rows after the sequence's last token are another's (or nobody's): they must not reach a
      // product, where a zero weight would not hide an infinity. Each warp clears its 32 rows and 4
      // cells of x and b.
      const int64_t left = it.eos - it.bos - (int64_t)ch * kL;
      if (left < kL) {
#pragma unroll 1
        for (int r = (int)left > th * 32 ? (int)left : th * 32; r < th * 32 + 32; ++r) {
          if (lane < 8) {
            const uint32_t at = (quad >> 1) * 8192 + sw128_off(r, (quad & 1) * 4 + (lane & 3));
            *reinterpret_cast<uint4*>(stage + (lane < 4 ? OFF_X : OFF_B) + at) = make_uint4(0, 0, 0, 0);
          }
        }
        __syncwarp();
      }
      const float cl0 = f->cl[hm][quad * 16 + (lane >> 2)], cl1 = f->cl[hm][quad * 16 + (lane >> 2) + 8];
      const uint32_t mt = m0 + par * kTileBytes, tg = tbase + TM_YM + par * 64 + ((uint32_t)(quad * 32) << 16);
#pragma unroll 1
      for (int half = half0; half <= quad >> 1; half += halfn)
        weigh_block(tg + half * 32, (half == quad >> 1 ? f->step[hm] : f->later[hm]) + half * 32 + 2 * (lane & 3),
                    (half == quad >> 1 ? f->cl[hm] + half * 32 : c->none) + 2 * (lane & 3), cl0, cl1,
                    quad * 16 - half * 32, mt + (((half * 4 + (lane >> 4)) ^ (lane & 7)) << 4),
                    mt + (((half * 4 + 2 + (lane >> 4)) ^ (lane & 7)) << 4), lane);
      uint32_t raw[4][4], parts[PARTS][8];
      load_x(raw, smem_u32(stage) + xoff, col0);
      if (__any_sync(0xffffffffu, not_finite(raw)) && real) hide_x(j);
      tc_fence_before();
      fence_async_smem();
      warp_arrive(&c->bar[T_M + par]);
      // x' into registers, and to TMEM once the product that read the last one is done
      float2 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = *reinterpret_cast<const float2*>(&f->to_end[hx][th * 32 + i * 8 + 2 * (lane & 3)]);
      split_half<PARTS>(raw[0], raw[1], w, parts);
      warp_arrive(&c->bar[T_FAC_FREE + fi]);
      if (j > 0 && !all_lanes(tc_wait(T_SU, (j - 1) & 1))) return;
      tc_fence_after();
      put_half<PARTS>(txp, parts);
      split_half<PARTS>(raw[2], raw[3], w, parts);
      put_half<PARTS>(txp + (16u << 16), parts);
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(&c->bar[T_XP + par]);
    }
  }
}

// ---- warps 8-15: the state and the output ------------------------------------------------------
// Two warps a TMEM lane quadrant: each takes half of S^T's k columns and half of the tokens.
template <typename ST, int K>
__device__ void run_rgroup(const ScanParams& p, uint8_t* sm, Ctl* c, uint32_t tbase) {
  constexpr int KH = K / 2;                      // k columns a thread
  const int rt = threadIdx.x - kMThreads, warp = rt >> 5, lane = rt & 31;
  const int quad = (threadIdx.x >> 5) & 3, hf = warp >> 2;
  const int v = quad * 32 + lane;                // value column of the item (TMEM lane)
  const uint32_t tq = tbase + ((uint32_t)(quad * 32) << 16);
  const int hd = p.V == 64 ? v >> 6 : 0;         // head of the item
  const int vh = p.V == 64 ? v & 63 : v;         // column of that head
  const int half = v >> 6;
  const int rep = p.H / p.G;
  // the output's 8 x 8 blocks, as in the M group: 32 value columns, tokens [32 hf, + 32)
  const uint32_t xoff = OFF_X + half * 8192 + hf * 4096 + ((lane >> 4) << 10) + (lane & 7) * 128;
  const uint32_t col0 = ((quad & 1) * 4 + ((lane >> 3) & 1)) ^ (lane & 7);
  uint32_t j = 0;
  for (uint32_t k = 0;; ++k) {
    const Item it = tc_item_warp(p, c, k);
    if (it.done) return;
    const bool second = p.V == 128 || (it.h0 % rep) + 1 < rep;
    const bool real = half == 0 || second;
    const int h = it.h0 + hd;
    const float dskip = p.d && real ? p.d[h] : 0.f;
    const int64_t so = (int64_t)hd * K * p.V + vh + (int64_t)hf * KH * p.V;  // within the item's state
    // A part starts from its slot of the scratch, which the combining kernel has completed.
    const int64_t whole = (int64_t)p.H * K * p.V, head = (int64_t)it.h0 * K * p.V + so;
    const ST* src = p.state_in && real && it.part < 0 ? static_cast<const ST*>(p.state_in) + it.state + so : nullptr;
    const float* fsrc = real && it.part >= 0 ? p.scratch + it.part * whole + head : nullptr;
    ST* dst = p.state_out && real && it.last ? static_cast<ST*>(p.state_out) + it.state + so : nullptr;
    if (it.nchunks == 0) {  // an empty sequence keeps its state
      if (dst && (const void*)dst != (const void*)src)
#pragma unroll 1
        for (int i = 0; i < KH; ++i)
          dst[(int64_t)i * p.V] = src ? src[(int64_t)i * p.V] : from_f32<ST>(0.f);
      continue;
    }
    // the state before the sequence or part
#pragma unroll 1
    for (int i0 = 0; i0 < KH; i0 += 16) {
      float s[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int at = (i0 + i) * p.V;
        s[i] = src ? to_f32(src[at]) : fsrc ? fsrc[at] : 0.f;
      }
      tmem_st16(tq + TM_S + hf * KH + i0, s);
    }
    tmem_st_wait();
#pragma unroll 1
    for (int ch = 0; ch < it.nchunks; ++ch, ++j) {
      const uint32_t st = j % kStages, par = j & 1, fi = j % kFacs;
      const int64_t t0 = it.bos + (int64_t)ch * kL;
      const int m = it.eos - t0 < kL ? (int)(it.eos - t0) : kL;
      // S before the chunk: its bf16 copy for the product with C, and its decay over the chunk
      const At fac{T_FAC + (int)fi, (j / kFacs) & 1};
      if (!all_lanes(tc_wait2(fac, ch > 0 ? At{T_SU, (j - 1) & 1} : fac))) return;
      tc_fence_after();
      const float dec = c->fac[fi].dec[hd];
#pragma unroll 1
      for (int i0 = 0; i0 < KH; i0 += 32) {
        float s[32], pk[16];
        tmem_ld16(tq + TM_S + hf * KH + i0, s);
        tmem_ld16(tq + TM_S + hf * KH + i0 + 16, s + 16);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) pk[i] = __uint_as_float(pack_bf16x2(s[2 * i], s[2 * i + 1]));
        tmem_st16(tq + TM_SB + (hf * KH + i0) / 2, pk);
#pragma unroll
        for (int i = 0; i < 32; i += 2) mul2(s[i], s[i + 1], dec, dec);
        tmem_st16(tq + TM_S + hf * KH + i0, s);
        tmem_st16(tq + TM_S + hf * KH + i0 + 16, s + 16);
      }
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(&c->bar[T_S]);
      // the output of tokens [32 hf, + 32), which takes the place of x in its tile
      // (T_XP: the M group has seen x land and has read it)
      if (!all_lanes(tc_wait3({T_XP + (int)par, (j >> 1) & 1}, {T_MX + (int)par, (j >> 1) & 1}, {T_Y, j & 1})))
        return;
      tc_fence_after();
      uint8_t* stage = sm + OFF_ST + st * kStageBytes;
      float2 e[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        e[i] = *reinterpret_cast<const float2*>(&c->fac[fi].e[hd][hf * 32 + i * 8 + 2 * (lane & 3)]);
#pragma unroll 1
      for (int lh = 0; lh < 2; ++lh) {
        float a[16], b[16];
        tmem_ld_16x256_x4(tq + ((uint32_t)(lh * 16) << 16) + TM_YI + hf * 32, a);
        tmem_ld_16x256_x4(tq + ((uint32_t)(lh * 16) << 16) + TM_YM + par * 64 + hf * 32, b);
        const uint32_t at = smem_u32(stage) + xoff + ((col0 ^ (lh * 2)) << 4);
        uint32_t x[2][4];
        ldsm_x4_trans(x[0], at);
        ldsm_x4_trans(x[1], at + 2048);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // block i / 2 of 8 tokens, lanes 0-7 or 8-15 of the 16
          float u = bf_lo(x[i >> 2][i & 3]), w = bf_hi(x[i >> 2][i & 3]);
          fma2(a[2 * i], a[2 * i + 1], e[i >> 1].x, e[i >> 1].y, b[2 * i], b[2 * i + 1]);
          fma2(u, w, dskip, dskip, a[2 * i], a[2 * i + 1]);
          x[i >> 2][i & 3] = pack_bf16x2(u, w);
        }
        stsm_x4_trans(at, x[0][0], x[0][1], x[0][2], x[0][3]);
        stsm_x4_trans(at + 2048, x[1][0], x[1][1], x[1][2], x[1][3]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&c->bar[T_EPI + par]);
        mbar_arrive(&c->bar[T_FAC_FREE + fi]);
      }
      if (m < kL && real) {
        // a partial chunk's box would cover the next sequence's rows: the warp's own, 16 bytes a lane
#pragma unroll 1
        for (int i = lane >> 2; i < 32; i += 8) {
          const int row = hf * 32 + i, cell = (quad & 1) * 4 + (lane & 3);
          if (row < m && KDA_CHECK(t0 + row < p.T))
            *reinterpret_cast<uint4*>(p.y + ((t0 + row) * p.H + it.h0) * p.V + half * 64 + cell * 8) =
                *reinterpret_cast<const uint4*>(stage + OFF_X + half * 8192 + sw128_off(row, cell));
        }
      }
      fence_async_smem();
      warp_arrive(&c->bar[T_EMPTY + st]);  // a full chunk's tile is stored by the loader
    }
    // the state after the sequence
    if (!all_lanes(tc_wait(T_SU, (j - 1) & 1))) return;
    tc_fence_after();
    {
#pragma unroll 1
      for (int i0 = 0; i0 < KH; i0 += 16) {
        float s[16];
        tmem_ld16(tq + TM_S + hf * KH + i0, s);
        tmem_ld_wait();
        if (dst) {
#pragma unroll
          for (int i = 0; i < 16; ++i) dst[(i0 + i) * p.V] = from_f32<ST>(s[i]);
        }
      }
      tc_fence_before();
    }
  }
}

// ---- the pass that forms states only -------------------------------------------------------------
// What a part adds to the state, sum_s exp(g_{s+1} + .. + g_end) d_s b_s x_s^T, from its last chunk to
// its first: the sum of the log-decays after a chunk is then known when the chunk comes, so that x'
// can take the decay to the part's end and S is not decayed on the way. No chain is left from chunk to
// chunk but the accumulator, and no exponent is positive. Both groups make x' (a chunk each, in turn),
// warps 17 and 16 scan a head each, two buffers hold x' and two S^T. (In the order of time, with S
// decayed every chunk, the pass took as long as the one that makes the outputs.) Chunks are all full: a
// sequence's last part is not in the list.
constexpr int S_XFREE = T_MX, S_DONE = T_G, S_FREE = T_EPI;  // x' is read, S complete, S read: by parity
__device__ __forceinline__ uint32_t states_xp(uint32_t par) { return par ? TM_SB : TM_XP; }
__device__ __forceinline__ uint32_t states_s(uint32_t par) { return par ? TM_YM : TM_S; }

__device__ void run_suffixes(const ScanParams& p, Ctl* c, int hd) {
  const int lane = threadIdx.x & 31, rep = p.H / p.G;
  uint32_t j = 0;
  for (uint32_t k = 0;; ++k) {
    const Item it = tc_item_warp(p, c, k);
    if (it.done) return;
    const int h = it.h0 + hd;
    const bool real = hd == 0 || (it.h0 % rep) + 1 < rep;
    const float rate2 = real ? ssm_rate(p.a_log[h], 1.4426950408889634f) : 0.f;
    const float bias = real && p.dt_bias ? p.dt_bias[h] : 0.f;
    const __nv_bfloat16* at = p.dt + (it.bos + (int64_t)(it.nchunks - 1) * kL + 2 * lane) * p.dt_pitch + h;
    int left = real ? it.nchunks : 0;
    auto read = [&](float (&n)[2]) {  // two scans ahead; -inf: no step
      n[0] = left > 0 ? to_f32(at[0]) : -INFINITY;
      n[1] = left > 0 ? to_f32(at[p.dt_pitch]) : -INFINITY;
      at -= kL * p.dt_pitch;
      --left;
    };
    float cur[2], nxt[2], later = 0.f;  // later: log2-decay of the part after the chunk
    read(cur);
    read(nxt);
#pragma unroll 1
    for (int i = 0; i < it.nchunks; ++i, ++j) {
      const uint32_t fi = j % kFacs;
      float d[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        d[u] = softplus_fast(cur[u] + bias);
        cur[u] = nxt[u];
      }
      read(nxt);
      const float g0 = rate2 * d[0], g1 = rate2 * d[1];
      float dn = g0 + g1;  // sum over the half's 16 lanes from here on
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) {
        const float b = __shfl_down_sync(0xffffffffu, dn, o, 16);
        if ((lane & 15) + o < 16) dn += b;
      }
      float after = __shfl_down_sync(0xffffffffu, dn, 1, 16);
      if ((lane & 15) == 15) after = 0.f;
      const float first = __shfl_sync(0xffffffffu, dn, 0), second = __shfl_sync(0xffffffffu, dn, 16);
      const float then = lane < 16 ? second + later : later;
      const float2 w = make_float2(d[0] * ex2(after + g1 + then), d[1] * ex2(after + then));
      later += first + second;
      if (j >= (uint32_t)kFacs && !all_lanes(tc_wait(T_FAC_FREE + fi, (j / kFacs - 1) & 1))) return;
      *reinterpret_cast<float2*>(&c->fac[fi].e[hd][2 * lane]) = w;
      warp_arrive(&c->bar[T_FAC + fi]);
    }
    if (real && lane == 0) p.decay[it.part * p.H + h] = ex2(later);
  }
}

template <int K, int PARTS>
__device__ void run_sums(uint8_t* sm, Ctl* c, uint32_t tbase) {
  if (!elect_one()) return;
  const uint32_t sbase = smem_u32(sm), id_s = idesc_bf16(128, K, 0, 1);
  uint32_t j = 0;
  bool ok = true;
  for (uint32_t k = 0; ok; ++k) {
    const int slot = k % kItems, sp = k & 1;
    ok = tc_wait(T_ITEM_FULL + slot, (k / kItems) & 1);
    if (!ok) break;
    const int nchunks = c->ring[slot].nchunks, done = c->ring[slot].done;
    mbar_arrive(&c->bar[T_ITEM_EMPTY + slot]);
    if (done) break;
    ok = k < 2 || tc_wait(S_FREE + sp, ((k >> 1) - 1) & 1);
    for (int i = 0; i < nchunks && ok; ++i, ++j) {
      const uint32_t st = j % kStages, par = j & 1;
      ok = tc_wait2({T_FULL + (int)st, (j / kStages) & 1}, {T_XP + (int)par, (j >> 1) & 1});
      if (!ok) break;
      tc_fence_after();
      const Desc b = desc128(sbase + OFF_ST + st * kStageBytes + OFF_B, 8192, 1024);
#pragma unroll
      for (uint32_t part = 0; part < PARTS; ++part)
        issue_ts(tbase + states_s(sp), tbase + states_xp(par) + part * 32, b, 2048, id_s, part > 0 || i > 0);
      mma_commit(&c->bar[S_XFREE + par]);
      mma_commit(&c->bar[T_EMPTY + st]);
    }
    if (ok) mma_commit(&c->bar[S_DONE + sp]);
  }
  mma_commit(&c->bar[T_DRAIN]);
  mbar_wait(&c->bar[T_DRAIN], 0);  // the full limit, aborted or not
}

template <int K, int PARTS>
__device__ void run_weighted(const ScanParams& p, uint8_t* sm, Ctl* c, uint32_t tbase) {
  constexpr int KQ = K / 4;  // k columns of S^T a warp reads
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = warp & 3, th = (warp >> 2) & 1;
  const uint32_t group = warp >> 3, par = group;
  // as in the M group
  const uint32_t xoff = OFF_X + (quad >> 1) * 8192 + th * 4096 + ((lane >> 4) << 10) + (lane & 7) * 128;
  const uint32_t col0 = ((quad & 1) * 4 + ((lane >> 3) & 1)) ^ (lane & 7);
  const uint32_t tq = tbase + ((uint32_t)(quad * 32) << 16), txp = tq + states_xp(par) + th * 16;
  const int v = quad * 32 + lane, hd = p.V == 64 ? v >> 6 : 0, vh = p.V == 64 ? v & 63 : v;
  const int rep = p.H / p.G;
  const int64_t whole = (int64_t)p.H * K * p.V;
  uint32_t j = 0;
  for (uint32_t k = 0;; ++k) {
    const Item it = tc_item_warp(p, c, k);
    if (it.done) return;
    for (int i = 0; i < it.nchunks; ++i, ++j) {
      if ((j & 1) != group) continue;
      const uint32_t st = j % kStages, fi = j % kFacs;
      if (!all_lanes(tc_wait2({T_FULL + (int)st, (j / kStages) & 1}, {T_FAC + (int)fi, (j / kFacs) & 1}))) return;
      float2 w[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        w[u] = *reinterpret_cast<const float2*>(&c->fac[fi].e[hd][th * 32 + u * 8 + 2 * (lane & 3)]);
      uint32_t raw[4][4], parts[PARTS][8];
      load_x(raw, smem_u32(sm) + OFF_ST + st * kStageBytes + xoff, col0);
      split_half<PARTS>(raw[0], raw[1], w, parts);
      warp_arrive(&c->bar[T_FAC_FREE + fi]);
      if (j >= 2 && !all_lanes(tc_wait(S_XFREE + (int)par, ((j >> 1) - 1) & 1))) return;
      tc_fence_after();
      put_half<PARTS>(txp, parts);
      split_half<PARTS>(raw[2], raw[3], w, parts);
      put_half<PARTS>(txp + (16u << 16), parts);
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(&c->bar[T_XP + par]);
    }
    // what the part adds, into the slot of the part after it
    const int sp = k & 1;
    if (!all_lanes(tc_wait(S_DONE + sp, (k >> 1) & 1))) return;
    tc_fence_after();
    const bool real = p.V == 128 || hd == 0 || (it.h0 % rep) + 1 < rep;
    float* dst = p.scratch + (it.part + 1) * whole + ((int64_t)(it.h0 + hd) * K + (warp >> 2) * KQ) * p.V + vh;
#pragma unroll 1
    for (int i0 = 0; i0 < KQ; i0 += 16) {
      float s[16];
      tmem_ld16(tq + states_s(sp) + (warp >> 2) * KQ + i0, s);
      tmem_ld_wait();
      if (real) {
#pragma unroll
        for (int i = 0; i < 16; ++i) dst[(int64_t)(i0 + i) * p.V] = s[i];
      }
    }
    tc_fence_before();
    warp_arrive(&c->bar[S_FREE + sp]);
  }
}

// ---- kernels ---------------------------------------------------------------------------------------
// Barriers and TMEM; false: the CTA leaves.
template <bool kState>
__device__ __forceinline__ bool tc_begin(const ScanParams& p, Ctl* c) {
  if (kState) grid_dep_launch_dependents();
  if (smem_u32(ssm_smem) & 1023u) {  // the swizzled tiles need it; the window starts so without static smem
    grid_dep_wait();
    if (threadIdx.x == 0) raise_status(p.status, KDA_DEVICE_PIPE_TIMEOUT);
    return false;
  }
  if (threadIdx.x == 0) {
    const uint32_t scans = kState && p.V == 64 ? 2 : 1;  // warps
    for (int b = 0; b < T_COUNT; ++b) {
      uint32_t count = 1;  // a loader's, a scan's or a commit's arrival
      if (b >= T_EMPTY && b < T_EMPTY + kStages) count = kState ? 1 : 9;        // a commit's, one an R warp
      if (b >= T_FAC && b < T_FAC + kFacs) count = scans;
      if (b >= T_FAC_FREE && b < T_FAC_FREE + kFacs) count = kState ? 8 : 16;   // one a warp of a group, of both
      if (b >= T_M && b <= T_S) count = 8;                                      // one a warp of a group
      if (kState && b >= S_FREE && b < S_FREE + 2) count = 16;
      // both groups' warps, issuers, scans
      if (b >= T_ITEM_EMPTY && b < T_ITEM_EMPTY + kItems) count = 16 + (kState ? 1 : 2) + scans;
      mbar_init(&c->bar[b], count);
    }
    c->abort = 0;
    c->wait_limit_ns = p.wait_limit_ns;
    c->status = p.status;
    c->poll = p.wait_limit_ns < kSleepHintNs ? 1 : 0;
    fence_mbar_init();
    prefetch_tensormap(&p.tm_x);
    prefetch_tensormap(&p.tm_b);
    if (!kState) {
      prefetch_tensormap(&p.tm_c);
      prefetch_tensormap(&p.tm_y);
    }
  }
  if (threadIdx.x >> 5 == 16) tmem_alloc(&c->tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_wait();
  return true;
}
__device__ __forceinline__ void tc_end(const ScanParams& p, uint32_t tbase) {
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x >> 5 == 16) tmem_dealloc(tbase, 512);
  if (threadIdx.x == 0) KDA_DEBUG_FOLD(p.status);
}

template <typename ST, int K>
__global__ void __launch_bounds__(kTcThreads, 1) ssm_scan_tc_kernel(const __grid_constant__ ScanParams p) {
  constexpr int PARTS = sizeof(ST) == 4 ? 3 : 2;
  uint8_t* sm = ssm_smem;
  Ctl* c = ctl();
  const int warp = threadIdx.x >> 5;
  if (!tc_begin<false>(p, c)) return;
  const uint32_t tbase = c->tmem_base;
  // (The order in which the five programs lie in the kernel, the M group's code next to the R group's and the
  // short ones last, is worth 1 to 3 %: 32768 tokens of 32 heads 241 us with the R group's second.)
  if (warp >= 8 && warp < 16) run_rgroup<ST, K>(p, sm, c, tbase);
  else if (warp < 8) run_mgroup<PARTS>(p, sm, c, tbase);
  else if (warp == 17) run_scan(p, c);
  else if (warp == 16) run_state<K, PARTS>(sm, c, tbase);
  else if (warp == 19) run_output<K>(p, sm, c, tbase);
  else run_loader<K, false>(p, sm, c);
  tc_end(p, tbase);
}

template <int K, int PARTS>
__global__ void __launch_bounds__(kTcThreads, 1) ssm_states_tc_kernel(const __grid_constant__ ScanParams p) {
  uint8_t* sm = ssm_smem;
  Ctl* c = ctl();
  const int warp = threadIdx.x >> 5;
  if (!tc_begin<true>(p, c)) return;
  const uint32_t tbase = c->tmem_base;
  if (*p.entries == 0) {  // no sequence was cut
  } else if (warp < 16) {
    run_weighted<K, PARTS>(p, sm, c, tbase);
  } else if (warp == 16) {
    if (p.V == 64) run_suffixes(p, c, 1);
  } else if (warp == 17) run_suffixes(p, c, 0);
  else if (warp == 18) run_loader<K, true>(p, sm, c);
  else run_sums<K, PARTS>(sm, c, tbase);
  tc_end(p, tbase);
}

// ---- host ----------------------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 tc_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess || q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// [T, cols] bf16 rows `pitch` elements apart, boxes of 64 tokens x 64 columns.
bool tc_map(CUtensorMap* m, const void* base, int64_t T, int64_t cols, int64_t pitch) {
  auto enc = tc_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)(T > 0 ? T : 1)};
  cuuint64_t strides[1] = {(cuuint64_t)pitch * 2};
  cuuint32_t box[2] = {64u, (cuuint32_t)kL};
  cuuint32_t es[2] = {1u, 1u};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_tc(void (*kern)(ScanParams), const ScanParams& p, int grid, cudaStream_t st) {
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kTcSmem);
  if (err != cudaSuccess) return err;
  return launch_pass(kern, dim3((unsigned)grid), kTcThreads, kTcSmem, p.list != nullptr, st, p);
}

int items_a_sequence(const kda_desc_t& d) {
  const int rep = d.num_v_heads / d.num_k_heads;
  return d.num_k_heads * (d.head_v_dim == 64 ? (rep + 1) / 2 : rep);
}

template <typename ST, int K>
cudaError_t launch_all(ScanParams& p, const SsmArgs& a, cudaStream_t st) {
  const SsmPlan plan = ssm_plan(a, p.pairs, gpu_sms(), kMinPart);
  p.status = &reinterpret_cast<PlanHdr*>(a.ws)->status;
  const int grid = (int)std::min<int64_t>(gpu_sms(), (int64_t)p.N * p.pairs);
  if (!plan.lists) {  // the sequences in their order; the header starts at zero
    p.next_item = &reinterpret_cast<PlanHdr*>(a.ws)->next_full;
    cudaError_t err = cudaMemsetAsync(a.ws, 0, sizeof(WsHeader), st);
    return err == cudaSuccess ? launch_tc(ssm_scan_tc_kernel<ST, K>, p, grid, st) : err;
  }
  cudaError_t err = launch_ssm_plan(plan, a, st);
  if (err != cudaSuccess) return err;
  p.decay = plan.decay;
  p.scratch = plan.scratch;
  if (plan.cap > 0) {
    p.list = plan.state;
    p.entries = &plan.hdr->n_state;
    p.next_item = &plan.hdr->next_state;
    err = launch_tc(ssm_states_tc_kernel<K, sizeof(ST) == 4 ? 3 : 2>, p, gpu_sms(), st);
    if (err == cudaSuccess) err = launch_ssm_combine(plan, a, st);
    if (err != cudaSuccess) return err;
  }
  p.list = plan.full;
  p.entries = &plan.hdr->n_full;
  p.next_item = &plan.hdr->next_full;
  return launch_tc(ssm_scan_tc_kernel<ST, K>, p, plan.cap > 0 ? gpu_sms() : grid, st);
}

}  // namespace

bool ssm_tc_supported(const kda_desc_t& d) {
  return d.qkv_dtype == KDA_BF16 && (d.flags & KDA_FLAG_CUDA_CORE_PATH) == 0u &&
         d.total_tokens > 0 && d.total_tokens < (int64_t)1 << 31;
}

size_t ssm_tc_workspace(const kda_desc_t& d) {
  return ssm_plan_workspace(d, items_a_sequence(d), gpu_sms(), kMinPart);
}

cudaError_t launch_ssm_tc(const SsmArgs& a, cudaStream_t st) {
  const kda_desc_t& d = a.d;
  const int H = d.num_v_heads, G = d.num_k_heads, K = d.head_k_dim, V = d.head_v_dim;
  ScanParams p;
  memset(&p, 0, sizeof(p));
  const int64_t T = d.total_tokens;
  if (!tc_map(&p.tm_x, a.in.x, T, (int64_t)H * V, a.in.x_pitch) ||
      !tc_map(&p.tm_b, a.in.b, T, (int64_t)G * K, a.in.b_pitch) ||
      !tc_map(&p.tm_c, a.in.c, T, (int64_t)G * K, a.in.c_pitch) ||
      !tc_map(&p.tm_y, a.y, T, (int64_t)H * V, (int64_t)H * V))
    return cudaErrorInvalidValue;
  p.dt = static_cast<const __nv_bfloat16*>(a.in.dt);
  p.dt_pitch = a.in.dt_pitch;
  p.a_log = a.in.a_log;
  p.dt_bias = a.in.dt_bias;
  p.d = a.in.d;
  p.cu = a.cu;
  p.idx = a.idx;
  p.state_in = a.state_in;
  p.state_out = a.state_out;
  p.y = static_cast<__nv_bfloat16*>(a.y);
  p.wait_limit_ns = pipeline_wait_limit_ns();
  p.N = d.num_seqs;
  p.H = H;
  p.G = G;
  p.V = V;
  p.T = T;
  p.num_slots = d.num_slots;
  p.slot_stride = a.slot_stride;
  p.pairs = items_a_sequence(d);
  if (d.state_dtype == KDA_BF16)
    return K == 128 ? launch_all<__nv_bfloat16, 128>(p, a, st) : launch_all<__nv_bfloat16, 64>(p, a, st);
  return K == 128 ? launch_all<float, 128>(p, a, st) : launch_all<float, 64>(p, a, st);
}

}  // namespace kda
