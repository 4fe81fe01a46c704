// kda_ssm.cu -- selective state space scan on CUDA cores: one token (or a few drafted ones) a
// row, and packed prompts token by token (fp32 inputs and the cross-check of the tensor-core scan).
//
//   d = softplus(dt + dt_bias);  S <- exp(-exp(a_log) d) S + d b x^T;  y = S^T c + D x
//
// per head, S [K, V] in fp32 registers.
#include "kda_internal.cuh"

namespace kda {
namespace {

KDA_DEBUG_FLAG_DEFINE();

// Four consecutive state elements as fp32.
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

// ---- one token, or a few drafted ones, a row ---------------------------------------------
// Bound by HBM: each state is streamed in and out once (with drafts: in once, out once a step).
// Grid (rows, heads): rows and heads on axes of their own, rows on grid.x.  A block of 256 threads
// holds a head's K x V state in registers, V/4 threads a row of 16-byte accesses, the row groups
// splitting K; all state loads are issued before anything is computed.  y's sum over K goes through
// shared memory.
constexpr int kDecThreads = 256;

template <typename QT, typename ST, int K, int V>
__global__ void __launch_bounds__(kDecThreads, 2)
ssm_decode_kernel(kda_ssm_inputs_t in, ST* pool, const int32_t* __restrict__ idx,
                  const int32_t* __restrict__ cu, QT* __restrict__ y,
                  uint32_t* __restrict__ status, int N, int64_t T, int H, int G,
                  int64_t num_slots, int64_t slot_stride, ST* __restrict__ cache,
                  int64_t cache_pitch, int max_steps, bool update_pool) {
  constexpr int TPR = V / 4;               // threads a state row
  constexpr int RG = kDecThreads / TPR;    // row groups
  constexpr int RPT = K / RG;              // rows a thread
  __shared__ float s_bc[2][2][K];          // d b and c of the token, by parity
  __shared__ float s_red[2][RG][V];

  const int n = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  const int rg = tid / TPR, col = (tid % TPR) * 4;
  if (n == 0 && h == 0) check_all(status, cu, idx, N, T, max_steps, num_slots);
  int64_t bos = n, eos = n + 1;
  if (cu && (!seq_bounds(cu, n, T, &bos, &eos) || eos - bos > max_steps)) return;
  const int64_t slot = idx ? resolve_slot(idx, n, num_slots) : (n < num_slots ? n : -1);
  if (slot < 0 || bos == eos) return;

  ST* S = pool + slot * slot_stride + (size_t)h * K * V + col;
  float s[RPT][4];
#pragma unroll
  for (int j = 0; j < RPT; ++j) load4(S + (size_t)(rg + j * RG) * V, s[j]);

  const float rate = -expf(in.a_log[h]);
  const float bias = in.dt_bias ? in.dt_bias[h] : 0.f;
  const float dskip = in.d ? in.d[h] : 0.f;
  const int g = h / (H / G);
  for (int64_t t = bos; t < eos; ++t) {
    const int par = (int)(t - bos) & 1;
    const float step =
        ssm_step(to_f32(static_cast<const QT*>(in.dt)[t * in.dt_pitch + h]), bias);
    const float keep = expf(rate * step);
    if (tid < K)
      s_bc[par][0][tid] = step * to_f32(static_cast<const QT*>(in.b)[t * in.b_pitch + g * K + tid]);
    else if (tid < 2 * K)
      s_bc[par][1][tid - K] =
          to_f32(static_cast<const QT*>(in.c)[t * in.c_pitch + g * K + tid - K]);
    float xv[4];
    load4(static_cast<const QT*>(in.x) + t * in.x_pitch + h * V + col, xv);
    __syncthreads();
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < RPT; ++j) {
      const float b = s_bc[par][0][rg + j * RG], c = s_bc[par][1][rg + j * RG];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[j][i] = fmaf(b, xv[i], keep * s[j][i]);
        acc[i] = fmaf(c, s[j][i], acc[i]);
      }
    }
    if (cache) {
      ST* co = cache + n * cache_pitch + (t - bos) * ((int64_t)H * K * V) + (size_t)h * K * V + col;
#pragma unroll
      for (int j = 0; j < RPT; ++j) store4(co + (size_t)(rg + j * RG) * V, s[j]);
    }
    *reinterpret_cast<float4*>(&s_red[par][rg][col]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    __syncthreads();
    if (tid < V && KDA_CHECK(t >= 0 && t < T)) {
      float r = 0.f;
#pragma unroll
      for (int i = 0; i < RG; ++i) r += s_red[par][i][tid];
      const float x = to_f32(static_cast<const QT*>(in.x)[t * in.x_pitch + h * V + tid]);
      y[((size_t)t * H + h) * V + tid] = from_f32<QT>(fmaf(dskip, x, r));
    }
  }
  if (update_pool) {
#pragma unroll
    for (int j = 0; j < RPT; ++j) store4(S + (size_t)(rg + j * RG) * V, s[j]);
  }
  KDA_DEBUG_FOLD(status);
}

// ---- prompts, token by token ---------------------------------------------------------------
// A block takes one sequence, one head and VT columns of its state: a thread holds K/8 rows of one
// column, eight lanes share a column and add their parts of y by shuffles.  Tokens are staged in
// shared memory kStage at a time.  fp32 FMAs bound it; time runs along one thread's registers.
constexpr int kStage = 32, kVT = 32, kScanThreads = 256;

template <typename QT, typename ST, int K>
__global__ void __launch_bounds__(kScanThreads)
ssm_scan_simt_kernel(kda_ssm_inputs_t in, const ST* state_in, const int32_t* __restrict__ idx,
                     ST* state_out, const int32_t* __restrict__ cu, QT* __restrict__ y,
                     uint32_t* __restrict__ status, int N, int64_t T, int H, int G, int V,
                     int64_t num_slots, int64_t slot_stride) {
  constexpr int RPT = K / 8;
  __shared__ __align__(16) float s_b[kStage][K], s_c[kStage][K];
  __shared__ float s_x[kStage][kVT], s_y[kStage][kVT], s_step[kStage], s_keep[kStage];

  const int n = blockIdx.x, h = blockIdx.y, v0 = blockIdx.z * kVT, tid = threadIdx.x;
  if (n == 0 && h == 0 && v0 == 0)
    check_all(status, cu, idx, N, T, T, idx ? num_slots : 0);
  int64_t bos, eos;
  if (!seq_bounds(cu, n, T, &bos, &eos)) return;
  const int64_t slot = idx ? resolve_slot(idx, n, num_slots) : n;
  if (slot < 0) return;

  // lane l of a warp: column l / 8 of the warp's four, rows [(l % 8) * 4, + 4) of each 32 rows
  const int warp = tid >> 5, lane = tid & 31;
  const int vc = warp * 4 + lane / 8, r0 = (lane % 8) * 4;
  const size_t at = slot * slot_stride + (size_t)h * K * V + v0 + vc;
  float s[RPT];
#pragma unroll
  for (int j = 0; j < RPT; ++j) {
    const int k = (j / 4) * 32 + r0 + j % 4;
    s[j] = state_in ? to_f32(state_in[at + (size_t)k * V]) : 0.f;
  }
  const float rate = -expf(in.a_log[h]);
  const float bias = in.dt_bias ? in.dt_bias[h] : 0.f;
  const float dskip = in.d ? in.d[h] : 0.f;
  const int g = h / (H / G);
  for (int64_t t0 = bos; t0 < eos; t0 += kStage) {
    const int m = eos - t0 < kStage ? (int)(eos - t0) : kStage;
    __syncthreads();  // the readers of the stage before are done
    for (int i = tid; i < m * K; i += kScanThreads) {
      const int t = i / K, k = i % K;
      s_b[t][k] = to_f32(static_cast<const QT*>(in.b)[(t0 + t) * in.b_pitch + g * K + k]);
      s_c[t][k] = to_f32(static_cast<const QT*>(in.c)[(t0 + t) * in.c_pitch + g * K + k]);
    }
    for (int i = tid; i < m * kVT; i += kScanThreads)
      s_x[i / kVT][i % kVT] = to_f32(
          static_cast<const QT*>(in.x)[(t0 + i / kVT) * in.x_pitch + h * V + v0 + i % kVT]);
    if (tid < m) {
      const float step =
          ssm_step(to_f32(static_cast<const QT*>(in.dt)[(t0 + tid) * in.dt_pitch + h]), bias);
      s_step[tid] = step;
      s_keep[tid] = expf(rate * step);
    }
    __syncthreads();
    for (int t = 0; t < m; ++t) {
      const float x = s_x[t][vc], dx = s_step[t] * x, keep = s_keep[t];
      float acc = 0.f;
#pragma unroll
      for (int j4 = 0; j4 < RPT / 4; ++j4) {
        const float4 b = *reinterpret_cast<const float4*>(&s_b[t][j4 * 32 + r0]);
        const float4 c = *reinterpret_cast<const float4*>(&s_c[t][j4 * 32 + r0]);
        float* q = s + j4 * 4;
        q[0] = fmaf(b.x, dx, keep * q[0]); acc = fmaf(c.x, q[0], acc);
        q[1] = fmaf(b.y, dx, keep * q[1]); acc = fmaf(c.y, q[1], acc);
        q[2] = fmaf(b.z, dx, keep * q[2]); acc = fmaf(c.z, q[2], acc);
        q[3] = fmaf(b.w, dx, keep * q[3]); acc = fmaf(c.w, q[3], acc);
      }
      acc += __shfl_xor_sync(0xffffffffu, acc, 1);
      acc += __shfl_xor_sync(0xffffffffu, acc, 2);
      acc += __shfl_xor_sync(0xffffffffu, acc, 4);
      if (lane % 8 == 0) s_y[t][vc] = fmaf(dskip, x, acc);
    }
    __syncthreads();
    for (int i = tid; i < m * kVT; i += kScanThreads) {
      const int64_t t = t0 + i / kVT;
      if (KDA_CHECK(t >= 0 && t < T))
        y[((size_t)t * H + h) * V + v0 + i % kVT] = from_f32<QT>(s_y[i / kVT][i % kVT]);
    }
  }
  if (state_out) {
#pragma unroll
    for (int j = 0; j < RPT; ++j) {
      const int k = (j / 4) * 32 + r0 + j % 4;
      state_out[at + (size_t)k * V] = from_f32<ST>(s[j]);
    }
  }
  KDA_DEBUG_FOLD(status);
}

template <typename QT, typename ST, int K, int V>
cudaError_t decode_kv(const SsmArgs& a, cudaStream_t st) {
  dim3 grid((unsigned)a.d.num_seqs, (unsigned)a.d.num_v_heads);
  ssm_decode_kernel<QT, ST, K, V><<<grid, kDecThreads, 0, st>>>(
      a.in, (ST*)a.state_out, a.idx, a.cu, (QT*)a.y, a.status, a.d.num_seqs, a.d.total_tokens,
      a.d.num_v_heads, a.d.num_k_heads, a.d.num_slots, a.slot_stride, (ST*)a.cache, a.cache_pitch,
      a.max_steps, a.update_pool);
  return cudaGetLastError();
}

template <typename QT, typename ST>
cudaError_t decode_types(const SsmArgs& a, cudaStream_t st) {
  if (a.d.head_k_dim == 128)
    return a.d.head_v_dim == 128 ? decode_kv<QT, ST, 128, 128>(a, st) : decode_kv<QT, ST, 128, 64>(a, st);
  return a.d.head_v_dim == 128 ? decode_kv<QT, ST, 64, 128>(a, st) : decode_kv<QT, ST, 64, 64>(a, st);
}

template <typename QT, typename ST, int K>
cudaError_t scan_k(const SsmArgs& a, cudaStream_t st) {
  dim3 grid((unsigned)a.d.num_seqs, (unsigned)a.d.num_v_heads, (unsigned)(a.d.head_v_dim / kVT));
  ssm_scan_simt_kernel<QT, ST, K><<<grid, kScanThreads, 0, st>>>(
      a.in, (const ST*)a.state_in, a.idx, (ST*)a.state_out, a.cu, (QT*)a.y, a.status, a.d.num_seqs,
      a.d.total_tokens, a.d.num_v_heads, a.d.num_k_heads, a.d.head_v_dim, a.d.num_slots,
      a.slot_stride);
  return cudaGetLastError();
}

template <typename QT, typename ST>
cudaError_t scan_types(const SsmArgs& a, cudaStream_t st) {
  return a.d.head_k_dim == 128 ? scan_k<QT, ST, 128>(a, st) : scan_k<QT, ST, 64>(a, st);
}

}  // namespace

cudaError_t launch_ssm_decode(const SsmArgs& a, cudaStream_t st) {
  const bool qb = a.d.qkv_dtype == KDA_BF16, sb = a.d.state_dtype == KDA_BF16;
  if (qb) return sb ? decode_types<__nv_bfloat16, __nv_bfloat16>(a, st) : decode_types<__nv_bfloat16, float>(a, st);
  return sb ? decode_types<float, __nv_bfloat16>(a, st) : decode_types<float, float>(a, st);
}

cudaError_t launch_ssm_simt(const SsmArgs& a, cudaStream_t st) {
  const bool qb = a.d.qkv_dtype == KDA_BF16, sb = a.d.state_dtype == KDA_BF16;
  if (qb) return sb ? scan_types<__nv_bfloat16, __nv_bfloat16>(a, st) : scan_types<__nv_bfloat16, float>(a, st);
  return sb ? scan_types<float, __nv_bfloat16>(a, st) : scan_types<float, float>(a, st);
}

}  // namespace kda
