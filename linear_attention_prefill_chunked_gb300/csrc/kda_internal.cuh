// kda_internal.cuh -- shared device/host helpers of the KDA CUDA library.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda.h"

namespace kda {

// Workspace header: the device status word and scheduler counters live in the
// first 256 bytes; per-path scratch follows at kWsPayload.
struct WsHeader {
  uint32_t status;        // KDA_DEVICE_* bits
  uint32_t next_item;     // dynamic work counter of the persistent prefill
  uint32_t num_entries;   // work-list entries written by the planning kernel
  uint32_t num_splits;    // sequences the planning kernel cut in two
  uint32_t reserved[60];
};
static_assert(sizeof(WsHeader) == 256, "workspace header is 256 bytes");
constexpr size_t kWsPayload = 256;

__device__ __forceinline__ void raise_status(uint32_t* status, uint32_t bit) {
  atomicOr(status, bit);
}

// Bounds checks of computed indices in the debug build (compiled with -DKDA_DEBUG): a failed
// check records itself in a per-file device flag and the access it guards is skipped (never a
// trap); each kernel folds the flag into KDA_DEVICE_DEBUG_BOUNDS of its status word before it
// returns.  In the normal build KDA_CHECK(c) is the constant true and costs nothing.
#ifdef KDA_DEBUG
#define KDA_DEBUG_FLAG_DEFINE() static __device__ unsigned int g_kda_bounds = 0
#define KDA_CHECK(c) ((c) ? true : (atomicOr(&g_kda_bounds, 1u), false))
#define KDA_DEBUG_FOLD(status) \
  do { if (*(volatile unsigned int*)&g_kda_bounds) atomicOr((status), KDA_DEVICE_DEBUG_BOUNDS); } while (0)
#else
#define KDA_DEBUG_FLAG_DEFINE() static_assert(true, "")
#define KDA_CHECK(c) (true || (c))  // never evaluated; keeps the operands referenced
#define KDA_DEBUG_FOLD(status) do { } while (0)
#endif

// ---- element conversions ----------------------------------------------------
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);  // round to nearest even
}

// Resolved per-sequence state slot: index -1 -> sentinel (num_slots - 1);
// returns -1 for an index outside [-1, num_slots).
__device__ __forceinline__ int64_t resolve_slot(const int32_t* idx, int n, int64_t num_slots) {
  const int32_t s = idx[n];
  if (s < -1 || (int64_t)s >= num_slots) return -1;
  return s < 0 ? num_slots - 1 : (int64_t)s;
}

// Sequence bounds with validation against [0, T]; returns false if invalid.
__device__ __forceinline__ bool seq_bounds(const int32_t* cu, int n, int64_t T, int64_t* bos,
                                           int64_t* eos) {
  const int64_t a = cu[n], b = cu[n + 1];
  if (a < 0 || b < a || b > T) return false;
  *bos = a;
  *eos = b;
  return true;
}

}  // namespace kda

// Internal launchers (C++ linkage, defined in the .cu files).
namespace kda {
// In-kernel gate activation.  When `a` is set the log-decay is not read from g but
// computed per (token, v-head, channel) as
//   g = max(-exp(A_log[h]) * softplus(a + dt_bias[h][c]), lb)
// (the gate form of the KDA / GDN tests in the sglang PR 27488 and PR 30169 digests).
struct GateAct {
  const void* a;         // [T, Hv, K], qkv dtype; null: g is given
  const float* A_log;    // [Hv]
  const float* dt_bias;  // [Hv, K] or null
  float lb;              // lower bound of g; -inf: none
};
// softplus(x) = log(1 + e^x), evaluated without overflow
__device__ __forceinline__ float softplus_f32(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }

struct PrefillArgs {
  kda_desc_t d;
  float scale;
  int64_t slot_stride;
  const void *q, *k, *v;
  const float *g, *beta;
  GateAct act;               // act.a null: g is given
  int gate_k;                // gate values per (token, v-head): K, or 1 (scalar gate)
  bool l2norm;               // normalise q and k rows in the kernel
  bool state_vk;             // states stored [V][K] per head (KDA_FLAG_STATE_VK)
  const int32_t* cu;
  const void* state_in;      // pool, dense h0 or null
  const int32_t* idx;        // null in dense mode
  void* state_out;           // pool (== state_in), dense ht, or null
  void* o;
  uint32_t* status;
  uint8_t* ws;               // workspace base
  size_t ws_bytes;
};
// Bound of the tensor-core prefill's pipeline waits for launches from now on
// (kda_set_pipeline_wait_limit; 2 s by default).
uint64_t pipeline_wait_limit_ns();
cudaError_t launch_prefill_simt(const PrefillArgs& a, cudaStream_t st);
cudaError_t launch_prefill_tc(const PrefillArgs& a, cudaStream_t st);
size_t prefill_tc_workspace(const kda_desc_t& d);      // beyond the header, with splitting
size_t prefill_tc_min_workspace(const kda_desc_t& d);  // beyond the header, no splitting
bool prefill_tc_supported(const kda_desc_t& d);

struct DecodeArgs {
  kda_desc_t d;
  float scale;
  int64_t slot_stride;
  const void *q, *k, *v;
  const float *g, *beta;
  int gate_k;                // K, or 1 (scalar gate)
  bool l2norm;               // normalise q and k rows in the kernel
  bool state_vk;             // states stored [V][K] per head (KDA_FLAG_STATE_VK)
  void* pool;
  const int32_t* idx;
  void* o;
  uint32_t* status;
  // draft steps (kda_decode_draft); plain decode: cu null, cache null, update_pool true
  const int32_t* cu;
  void* cache;
  int64_t cache_pitch;
  int max_steps;
  bool update_pool;
};
cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t st);
}  // namespace kda

// Operators of the layers around the recurrence (kda_conv.cu, kda_ssm.cu, kda_draft.cu).
namespace kda {

// Launches a kernel that may set itself up while the one before it on the stream still runs; it waits for that
// (grid_dep_wait) before it reads or writes anything that kernel touches.
template <typename... P, typename... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, dim3 block, size_t bytes, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// SMs of the current device (152, for sizes asked for where there is none).
int gpu_sms();

// Their status word is written by one block, which looks every sequence and slot over before
// anything else of its work, so that a call needs no clear of the word in front of the kernel
// (one stream operation less a call).  The debug build, where any block may add
// KDA_DEVICE_DEBUG_BOUNDS, clears it on the host and adds to it instead.
__device__ __forceinline__ void set_status(uint32_t* status, uint32_t bits) {
#ifdef KDA_DEBUG
  if (bits) atomicOr(status, bits);
#else
  *status = bits;
#endif
}

// The whole block checks cu (null: none; runs longer than max_len are bad) and the slot indices
// (null: slot n, when num_slots > 0) of n < N and writes the status word.  Ends with a barrier.
__device__ __forceinline__ void check_all(uint32_t* status, const int32_t* cu, const int32_t* idx,
                                          int N, int64_t T, int64_t max_len, int64_t num_slots) {
  uint32_t bits = 0;
  for (int n = threadIdx.x; n < N; n += blockDim.x) {
    int64_t a, b;
    if (cu && (!seq_bounds(cu, n, T, &a, &b) || b - a > max_len)) bits |= KDA_DEVICE_BAD_SEQLENS;
    if (idx ? resolve_slot(idx, n, num_slots) < 0 : (num_slots > 0 && n >= num_slots))
      bits |= KDA_DEVICE_BAD_SLOT;
  }
  const int s = __syncthreads_or((int)(bits & KDA_DEVICE_BAD_SEQLENS));
  const int i = __syncthreads_or((int)(bits & KDA_DEVICE_BAD_SLOT));
  if (threadIdx.x == 0)
    set_status(status, (s ? KDA_DEVICE_BAD_SEQLENS : 0u) | (i ? KDA_DEVICE_BAD_SLOT : 0u));
}

// The whole block (of R threads) writes the sequence of rows t0 .. t0 + R - 1 to s_seq: -1 where none that is
// valid holds a row, the last one where lengths run backwards.  Ends with a barrier.
template <int R>
__device__ __forceinline__ void sequences_of(int* s_seq, const int32_t* cu, const int32_t* idx, int64_t num_slots,
                                             int N, int64_t T, int64_t t0) {
  const int tid = threadIdx.x;
  s_seq[tid] = -1;
  __syncthreads();
  for (int base = 0; base < N; base += R) {
    const int n = base + tid;
    int64_t a = 0, b = 0;
    bool hit = n < N && seq_bounds(cu, n, T, &a, &b) && a < t0 + R && b > t0 && a < b;
    if (hit && idx) hit = resolve_slot(idx, n, num_slots) >= 0;
    unsigned m = __ballot_sync(0xffffffffu, hit);
    while (m) {  // a warp writes each of its hits together: a long sequence fills all rows
      const int src = __ffs(m) - 1;
      m &= m - 1;
      const int64_t sa = __shfl_sync(0xffffffffu, a, src), sb = __shfl_sync(0xffffffffu, b, src);
      const int sn = __shfl_sync(0xffffffffu, n, src);
      const int lo = (int)(sa > t0 ? sa - t0 : 0), hi = (int)(sb < t0 + R ? sb - t0 : R);
      for (int i = lo + (tid & 31); i < hi; i += 32) atomicMax(&s_seq[i], sn);
    }
  }
  __syncthreads();
}

// Rows of `row` elements of the sequences without tokens: to <- from (zeros if null); with `zero_bad` those of
// invalid sequences become 0.  A warp of the grid's (32 a block, the last block's first: others have their rows'
// sequences to see to) takes 256 elements of 32 sequences at a time, of every eighth of them where the grid has
// warps enough (2741 x 1003 fp32 in 37 sequences, 7 of them empty: the convolution's backward pass 25 us, 29 where
// a warp takes all 32 and the first blocks come first).
constexpr int kRowChunk = 256, kRowParts = 8;
template <typename T>
__device__ __forceinline__ void rows_without_tokens(const int32_t* cu, int N, int64_t total, const T* from, T* to,
                                                    int64_t row, bool zero_bad) {
  const int lane = threadIdx.x & 31;
  const int64_t chunks = (row + kRowChunk - 1) / kRowChunk, pairs = ((int64_t)N + 31) / 32 * chunks;
  const int parts = pairs * kRowParts <= gridDim.x * 32ll ? kRowParts : 1;
  for (int64_t w = (gridDim.x - 1 - blockIdx.x) * 32ll + (threadIdx.x >> 5); w < pairs * parts; w += gridDim.x * 32ll) {
    const int64_t group = w / parts / chunks * 32;
    const unsigned mine = parts == 1 ? 0xffffffffu : 0x01010101u << (w % parts);
    const int n = (int)group + lane;
    int64_t a = 0, b = 1;
    const bool ok = n < N && seq_bounds(cu, n, total, &a, &b);
    const unsigned empty = __ballot_sync(0xffffffffu, ok && a == b);
    unsigned todo = (empty | __ballot_sync(0xffffffffu, n < N && !ok && zero_bad)) & mine;
    while (todo) {
      const int i = __ffs(todo) - 1;
      todo &= todo - 1;
      const bool copy = ((empty >> i) & 1) && from;
      const int64_t at = (group + i) * row, c0 = w / parts % chunks * kRowChunk + lane;
      T v[kRowChunk / 32];
#pragma unroll
      for (int j = 0; j < kRowChunk / 32; ++j)
        v[j] = copy && c0 + j * 32 < row ? from[at + c0 + j * 32] : from_f32<T>(0.f);
#pragma unroll
      for (int j = 0; j < kRowChunk / 32; ++j)
        if (c0 + j * 32 < row) to[at + c0 + j * 32] = v[j];
    }
  }
}
// Blocks of 32 warps for it, beside the others of a grid of `most`.
inline int64_t row_blocks(int64_t N, int64_t row, int64_t most) {
  const int64_t pairs = (N + 31) / 32 * ((row + kRowChunk - 1) / kRowChunk), parts = (pairs * kRowParts + 31) / 32;
  return parts <= most ? parts : (pairs + 31) / 32;
}

// Two fp32 operations as one packed instruction, each rounded to nearest.
__device__ __forceinline__ void mul2(float& a, float& b, float x, float y) {
  unsigned long long ab, xy;
  asm("mov.b64 %0, {%1, %2};" : "=l"(ab) : "f"(a), "f"(b));
  asm("mov.b64 %0, {%1, %2};" : "=l"(xy) : "f"(x), "f"(y));
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(ab) : "l"(xy));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(ab));
}
__device__ __forceinline__ void sub2(float& a, float& b, float x, float y) {
  unsigned long long ab, xy;
  asm("mov.b64 %0, {%1, %2};" : "=l"(ab) : "f"(a), "f"(b));
  asm("mov.b64 %0, {%1, %2};" : "=l"(xy) : "f"(x), "f"(y));
  asm("sub.rn.f32x2 %0, %0, %1;" : "+l"(ab) : "l"(xy));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(ab));
}
__device__ __forceinline__ void add2(float& a, float& b, float x, float y) {
  unsigned long long ab, xy;
  asm("mov.b64 %0, {%1, %2};" : "=l"(ab) : "f"(a), "f"(b));
  asm("mov.b64 %0, {%1, %2};" : "=l"(xy) : "f"(x), "f"(y));
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(ab) : "l"(xy));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(ab));
}
// (a, b) <- (a, b) + (x, y) * (u, v)
__device__ __forceinline__ void acc2(float& a, float& b, float x, float y, float u, float v) {
  unsigned long long ab, xy, uv;
  asm("mov.b64 %0, {%1, %2};" : "=l"(ab) : "f"(a), "f"(b));
  asm("mov.b64 %0, {%1, %2};" : "=l"(xy) : "f"(x), "f"(y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(uv) : "f"(u), "f"(v));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(ab) : "l"(xy), "l"(uv));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(ab));
}
// (a, b) <- (a, b) * (x, y) + (u, v)
__device__ __forceinline__ void fma2(float& a, float& b, float x, float y, float u, float v) {
  unsigned long long ab, xy, uv;
  asm("mov.b64 %0, {%1, %2};" : "=l"(ab) : "f"(a), "f"(b));
  asm("mov.b64 %0, {%1, %2};" : "=l"(xy) : "f"(x), "f"(y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(uv) : "f"(u), "f"(v));
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(ab) : "l"(xy), "l"(uv));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(ab));
}

struct ConvArgs {
  kda_conv_desc_t d;
  const void *x, *w, *bias;
  const int32_t* cu;       // null: one token a row
  const void* state_in;    // pool or dense initial states or null
  const int32_t* idx;      // null: dense, or slot n in the token form
  void* state_out;         // pool, dense final states or null
  int64_t slot_stride;
  void* y;
  uint32_t* status;
  void* cache;             // token form: states after each step, or null
  int64_t cache_pitch;
  int max_steps;
  bool update_pool;
};
cudaError_t launch_conv(const ConvArgs& a, cudaStream_t st);
cudaError_t launch_conv_decode(const ConvArgs& a, cudaStream_t st);

struct ConvBackArgs {
  kda_conv_desc_t d;
  const void* dy;
  int64_t dy_pitch;
  const void *x, *w, *bias;
  const int32_t* cu;
  const void *state, *dfinal;  // [N, W-1, Ch] or null
  void *dx, *dstate;           // dstate may be null
  float *dw, *db;              // db may be null
  uint8_t* ws;
};
size_t conv_back_workspace(const kda_conv_desc_t& d);  // the whole workspace, header included
cudaError_t launch_conv_back(const ConvBackArgs& a, cudaStream_t st);

// Four elements as fp32, aligned to four.
__device__ __forceinline__ void load4(const float* p, float (&r)[4]) {
  const float4 x = *reinterpret_cast<const float4*>(p);
  r[0] = x.x; r[1] = x.y; r[2] = x.z; r[3] = x.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&r)[4]) {
  const uint2 x = *reinterpret_cast<const uint2*>(p);
  r[0] = __uint_as_float(x.x << 16); r[1] = __uint_as_float(x.x & 0xffff0000u);
  r[2] = __uint_as_float(x.y << 16); r[3] = __uint_as_float(x.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(float* p, const float (&r)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(r[0], r[1], r[2], r[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&r)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(r[0], r[1]), b = __floats2bfloat162_rn(r[2], r[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                            *reinterpret_cast<const uint32_t*>(&b));
}

struct SsmArgs {
  kda_desc_t d;
  kda_ssm_inputs_t in;
  const int32_t* cu;
  const void* state_in;
  const int32_t* idx;
  void* state_out;
  int64_t slot_stride;
  void* y;
  uint32_t* status;
  uint8_t* ws;
  size_t ws_bytes;
  void* cache;
  int64_t cache_pitch;
  int max_steps;
  bool update_pool;
};
cudaError_t launch_ssm_decode(const SsmArgs& a, cudaStream_t st);
cudaError_t launch_ssm_simt(const SsmArgs& a, cudaStream_t st);
bool ssm_tc_supported(const kda_desc_t& d);
size_t ssm_tc_workspace(const kda_desc_t& d);  // the whole workspace, header included
size_t ssm_simt_workspace(const kda_desc_t& d);
cudaError_t launch_ssm_tc(const SsmArgs& a, cudaStream_t st);
// Log-decay a unit of step of a head, -exp(a_log) (times `unit`: its logarithm's base). Kept finite: from
// a_log = 89 on any step above 1e-36 forgets everything all the same, and a step of zero nothing.
__device__ __forceinline__ float ssm_rate(float a_log, float unit = 1.f) {
  const float r = -expf(a_log) * unit;
  return r < -3.402823466e38f ? -3.402823466e38f : r;  // NaN stays
}
// Step size of one (token, head): softplus(dt + bias).
__device__ __forceinline__ float ssm_step(float dt, float bias) { return softplus_f32(dt + bias); }

struct GatedArgs {
  kda_gated_desc_t d;
  const void *x, *r, *i;      // i null: no input gate
  const float* a_log;
  const int32_t* cu;          // null: one token a row
  const float* state_in;      // pool, dense initial states or null
  const int32_t* idx;         // null: dense, or slot n in the token form
  float* state_out;           // pool, dense final states or null
  int64_t slot_stride;
  void* y;
  float* carries;             // written by the forward pass, read by the backward pass
  uint8_t* ws;
  // token form
  float* cache;
  int64_t cache_pitch;
  int max_steps;
  bool update_pool;
  // backward pass
  const void* dy;
  int64_t dy_pitch;
  const float* dfinal;
  void *dx, *dr, *di;
  float *da_log, *dstate;
};
size_t gated_scan_workspace(const kda_gated_desc_t& d);  // the whole workspace, header included
size_t gated_back_workspace(const kda_gated_desc_t& d);
bool gated_fits(const kda_gated_desc_t& d);
cudaError_t launch_gated_scan(const GatedArgs& a, cudaStream_t st);
cudaError_t launch_gated_back(const GatedArgs& a, cudaStream_t st);
cudaError_t launch_gated_token(const GatedArgs& a, cudaStream_t st);

struct SampleArgs {
  kda_sample_desc_t d;
  const void* logits;
  const float* noise;                       // tokens only
  const float *temperature, *top_p, *min_p; // [num_rows], or null: the descriptor's
  const int32_t* top_k;
  int32_t* token;                           // one of token and probs is null
  float* probs;
  uint32_t* status;
};
bool sample_fits(const kda_sample_desc_t& d);
cudaError_t launch_sample(const SampleArgs& a, cudaStream_t st);

cudaError_t launch_verify(int N, int64_t T, int vocab, const int32_t* tokens, const float* p,
                          const float* q, const float* u, const float* noise, const int32_t* cu,
                          int32_t* kept, int32_t* next, uint32_t* status, uint32_t flags, cudaStream_t st);
cudaError_t launch_commit(int N, int elem_bytes, int64_t row, const void* cache, int64_t pitch,
                          int max_steps, const int32_t* kept, void* pool, int64_t num_slots,
                          int64_t slot_stride, const int32_t* idx, uint32_t* status,
                          cudaStream_t st);
}  // namespace kda
