// kda_ssm.cu -- selective state space scan on CUDA cores: one token (or a few drafted ones) a
// row, and packed prompts token by token (fp32 inputs and the cross-check of the tensor-core scan).
//
//   d = softplus(dt + dt_bias);  S <- exp(-exp(a_log) d) S + d b x^T;  y = S^T c + D x
//
// per head, S [K, V] in fp32 registers.
#include "kda_internal.cuh"
#include "kda_ssm_plan.cuh"

namespace kda {
namespace {

KDA_DEBUG_FLAG_DEFINE();

// ---- one token, or a few drafted ones, a row ---------------------------------------------
// Bound by HBM: each state is streamed in and out once (with drafts: in once, out once a step).
// Grid (rows, heads): rows and heads on axes of their own, rows on grid.x.  A block of 256 threads
// holds a head's K x V state in registers, V/4 threads a row of 16-byte accesses, the row groups
// splitting K; all state loads are issued before anything is computed.  y's sum over K goes through
// shared memory.  1024 rows of 32 heads of 128 x 128 in fp32, 4.3 GB, take 636 us: a copy's rate.
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

  const float rate = ssm_rate(in.a_log[h]);
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
// A block takes one sequence (or part of one), one head and VT columns of its state: a thread holds 4
// rows of 4 columns, K/4 lanes all rows of a column. Tokens are staged in shared memory kStage at a
// time, the next ones on their way in registers. The lanes' parts of y are added for eight tokens and
// four columns at once, every step of the tree halving the sums a lane still carries.
// Bound by instructions and their latency, ~45 a token and warp: 115 ns a token where a block has its SM
// alone (fp32, K = 128); with 16 rows of one column a thread, whose reads of b and c alone take 256 cycles
// of shared memory, it was 265 ns. Time runs along a block, so long sequences are cut as
// the tensor-core scan's are: a pass that forms states only (kState), the combine, all parts at once.
constexpr int kStage = 32, kScanThreads = 256, kEight = 8;
constexpr int kSimtMinPart = 8;  // chunks

struct SimtLists {
  const Entry* list;        // null: a sequence each
  const uint32_t* entries;
  float *scratch, *decay;
};

template <typename QT, typename ST, int K, bool kState>
__global__ void __launch_bounds__(kScanThreads)
ssm_scan_simt_kernel(kda_ssm_inputs_t in, const ST* state_in, const int32_t* __restrict__ idx,
                     ST* state_out, const int32_t* __restrict__ cu, QT* __restrict__ y,
                     uint32_t* __restrict__ status, int N, int64_t T, int H, int G, int V,
                     int64_t num_slots, int64_t slot_stride, SimtLists lists) {
  constexpr int KL = K / 4;                 // lanes of a column
  constexpr int VT = 32 / KL * 4 * 8;       // columns a block: 32 (K = 128) or 64
  constexpr int NB = kStage * K / 4 / kScanThreads, NX = kStage * VT / 4 / kScanThreads;
  __shared__ __align__(16) float s_b[kStage][K], s_c[kState ? 1 : kStage][K];
  __shared__ __align__(16) float s_x[kStage][VT], s_y[kState ? 1 : kStage][VT];
  __shared__ float2 s_step[kStage];         // step and decay of a token

  const int tid = threadIdx.x, tiles = V / VT;
  if (kState) tc::grid_dep_launch_dependents();
  tc::grid_dep_wait();
  const int e = (int)(blockIdx.x / (unsigned)(H * tiles)), q = (int)(blockIdx.x % (unsigned)(H * tiles));
  const int h = q / tiles, v0 = q % tiles * VT;
  Entry en{e, 0, 0, -1, 1, {0, 0, 0}};
  if (lists.list) {
    if (e >= (int)*lists.entries) return;
    en = lists.list[e];
  } else if (blockIdx.x == 0) {
    check_all(status, cu, idx, N, T, T, idx ? num_slots : 0);
  }
  int64_t bos, eos;
  if (!seq_bounds(cu, en.n, T, &bos, &eos)) return;
  const int64_t slot = idx ? resolve_slot(idx, en.n, num_slots) : en.n;
  if (slot < 0) return;
  if (lists.list) {
    bos += (int64_t)en.chunk0 * kSsmChunk;
    const int64_t end = bos + (int64_t)en.nchunks * kSsmChunk;
    if (end < eos) eos = end;
  }

  const int warp = tid >> 5, lane = tid & 31, l = lane % KL;
  const int r0 = l * 4, c0 = (warp * (32 / KL) + lane / KL) * 4;  // the thread's rows and columns
  const size_t in_state = (size_t)h * K * V + (size_t)r0 * V + v0 + c0, at = slot * slot_stride + in_state;
  // a part starts from its slot of the scratch; what it adds goes into the next one's (kState)
  float* part = en.part >= 0 ? lists.scratch + (size_t)en.part * H * K * V + in_state : nullptr;
  float s[4][4];  // [row][column]
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (part && !kState) load4(part + (size_t)r * V, s[r]);
    else if (state_in && !kState) load4(state_in + at + (size_t)r * V, s[r]);
    else s[r][0] = s[r][1] = s[r][2] = s[r][3] = 0.f;
  }
  const float rate = ssm_rate(in.a_log[h]);
  const float bias = in.dt_bias ? in.dt_bias[h] : 0.f;
  const float dskip = in.d ? in.d[h] : 0.f;
  const QT* pb = static_cast<const QT*>(in.b) + h / (H / G) * K;
  const QT* pc = static_cast<const QT*>(in.c) + h / (H / G) * K;
  const QT* px = static_cast<const QT*>(in.x) + h * V + v0;
  const QT* pd = static_cast<const QT*>(in.dt) + h;

  float nb[NB][4], nc[NB][4], nx[NX][4], nd = 0.f;
  // tokens past the end: of no step, of a decay of one, zero otherwise
  auto fetch = [&](int64_t t0) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int j = tid + i * kScanThreads, k = j % (K / 4) * 4;
      const int64_t t = t0 + j / (K / 4);
      nb[i][0] = nb[i][1] = nb[i][2] = nb[i][3] = 0.f;
      nc[i][0] = nc[i][1] = nc[i][2] = nc[i][3] = 0.f;
      if (t < eos) {
        load4(pb + t * in.b_pitch + k, nb[i]);
        if (!kState) load4(pc + t * in.c_pitch + k, nc[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int j = tid + i * kScanThreads;
      const int64_t t = t0 + j / (VT / 4);
      nx[i][0] = nx[i][1] = nx[i][2] = nx[i][3] = 0.f;
      if (t < eos) load4(px + t * in.x_pitch + j % (VT / 4) * 4, nx[i]);
    }
    if (tid < kStage && t0 + tid < eos) nd = to_f32(pd[(t0 + tid) * in.dt_pitch]);
  };
  if (bos < eos) fetch(bos);
  float total = 1.f;
  for (int64_t t0 = bos; t0 < eos; t0 += kStage) {
    const int m = eos - t0 < kStage ? (int)(eos - t0) : kStage;
    __syncthreads();  // the readers of the stage before are done
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int j = tid + i * kScanThreads;
      store4(&s_b[0][0] + j * 4, nb[i]);
      if (!kState) store4(&s_c[0][0] + j * 4, nc[i]);
    }
#pragma unroll
    for (int i = 0; i < NX; ++i) store4(&s_x[0][0] + (tid + i * kScanThreads) * 4, nx[i]);
    if (tid < kStage) {
      const float step = tid < m ? ssm_step(nd, bias) : 0.f;
      s_step[tid] = make_float2(step, tid < m ? expf(rate * step) : 1.f);
    }
    __syncthreads();
    if (t0 + kStage < eos) fetch(t0 + kStage);
#pragma unroll 1
    for (int tb = 0; tb < m; tb += kEight) {
      float acc[kEight * 4];
#pragma unroll
      for (int u = 0; u < kEight; ++u) {
        const float2 st = s_step[tb + u];
        float dx[4], b[4], c[4];
        load4(&s_x[tb + u][c0], dx);
        load4(&s_b[tb + u][r0], b);
        if (!kState) load4(&s_c[tb + u][r0], c);
        mul2(dx[0], dx[1], st.x, st.x);
        mul2(dx[2], dx[3], st.x, st.x);
        float* a = acc + u * 4;
        a[0] = a[1] = a[2] = a[3] = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          mul2(s[r][0], s[r][1], st.y, st.y);
          mul2(s[r][2], s[r][3], st.y, st.y);
          acc2(s[r][0], s[r][1], dx[0], dx[1], b[r], b[r]);
          acc2(s[r][2], s[r][3], dx[2], dx[3], b[r], b[r]);
          if (!kState) {
            acc2(a[0], a[1], s[r][0], s[r][1], c[r], c[r]);
            acc2(a[2], a[3], s[r][2], s[r][3], c[r], c[r]);
          }
        }
        if (kState) total *= st.y;
      }
      if (!kState) {
        // sums over a column's lanes: a lane keeps the half of its values that its lane bit names
#pragma unroll
        for (int i = 0; i < (KL == 32 ? 5 : 4); ++i) {
          const int o = (KL / 2) >> i, n = (kEight * 2) >> i;
#pragma unroll
          for (int u = 0; u < n; ++u) {
            const float mine = l & o ? acc[u + n] : acc[u], other = l & o ? acc[u] : acc[u + n];
            acc[u] = mine + __shfl_xor_sync(0xffffffffu, other, o);
          }
        }
        // value l n + u: token / 4, column % 4
#pragma unroll
        for (int u = 0; u < kEight * 4 / KL; ++u) {
          const int i = l * (kEight * 4 / KL) + u, t = tb + i / 4, v = c0 + i % 4;
          s_y[t][v] = fmaf(dskip, s_x[t][v], acc[u]);
        }
      }
    }
    if (kState) continue;
    __syncthreads();
    for (int i = tid; i < m * (VT / 4); i += kScanThreads) {
      const int64_t t = t0 + i / (VT / 4);
      float r[4];
      load4(&s_y[i / (VT / 4)][i % (VT / 4) * 4], r);
      if (KDA_CHECK(t >= 0 && t < T)) store4(y + ((size_t)t * H + h) * V + v0 + i % (VT / 4) * 4, r);
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (kState) store4(part + (size_t)H * K * V + (size_t)r * V, s[r]);
    else if (state_out && en.last) store4(state_out + at + (size_t)r * V, s[r]);
  }
  if (kState && tid == 0 && v0 == 0) lists.decay[en.part * H + h] = total;
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

int simt_items(const kda_desc_t& d) { return d.num_v_heads * (d.head_v_dim / (d.head_k_dim == 128 ? 32 : 64)); }
// Blocks an SM. Two have hardly more throughput than one (106 ns a token against 115), and the order in
// which a grid's blocks reach the SMs pairs some while other SMs stay empty: 1024 tokens of 64 heads, 128
// blocks of a longer grid, took 219 us against 120 us. So a block has its SM alone, by the shared memory
// it asks for (8192 tokens of those heads: 940 us, in pairs 1247), unless there are several rounds of them
// (32 sequences, 4096 tokens: 396 us in pairs, 488 alone).
int simt_per_sm(const kda_desc_t& d) { return (int64_t)d.num_seqs * simt_items(d) >= 4ll * gpu_sms() ? 2 : 1; }
int simt_workers(const kda_desc_t& d) { return simt_per_sm(d) * gpu_sms(); }
constexpr int kAloneSmem = 120 * 1024;  // more than half of an SM's


template <typename QT, typename ST, int K, bool kState>
cudaError_t scan_pass(const SsmArgs& a, int64_t entries, const SimtLists& lists, cudaStream_t st) {
  const int64_t blocks = entries * simt_items(a.d);  // entries outermost: those not there leave last
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  auto kern = ssm_scan_simt_kernel<QT, ST, K, kState>;
  const int smem = simt_per_sm(a.d) == 1 ? kAloneSmem : 0;
  if (smem) {
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
  }
  return launch_pass(kern, dim3((unsigned)blocks), kScanThreads, smem, lists.list != nullptr, st, a.in,
                     (const ST*)a.state_in, a.idx, (ST*)a.state_out, a.cu, (QT*)a.y, a.status, a.d.num_seqs,
                     a.d.total_tokens, a.d.num_v_heads, a.d.num_k_heads, a.d.head_v_dim, a.d.num_slots,
                     a.slot_stride, lists);
}

template <typename QT, typename ST, int K>
cudaError_t scan_k(const SsmArgs& a, cudaStream_t st) {
  const SsmPlan p = ssm_plan(a, simt_items(a.d), simt_workers(a.d), kSimtMinPart);
  if (p.cap == 0)
    return scan_pass<QT, ST, K, false>(a, a.d.num_seqs, SimtLists{nullptr, nullptr, nullptr, nullptr}, st);
  cudaError_t err = launch_ssm_plan(p, a, st);
  if (err == cudaSuccess)
    err = scan_pass<QT, ST, K, true>(a, p.cap, SimtLists{p.state, &p.hdr->n_state, p.scratch, p.decay}, st);
  if (err == cudaSuccess) err = launch_ssm_combine(p, a, st);
  if (err != cudaSuccess) return err;
  return scan_pass<QT, ST, K, false>(a, (int64_t)a.d.num_seqs + p.cap,
                                     SimtLists{p.full, &p.hdr->n_full, p.scratch, p.decay}, st);
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

size_t ssm_simt_workspace(const kda_desc_t& d) {
  return ssm_plan_workspace(d, simt_items(d), simt_workers(d), kSimtMinPart);
}

cudaError_t launch_ssm_simt(const SsmArgs& a, cudaStream_t st) {
  const bool qb = a.d.qkv_dtype == KDA_BF16, sb = a.d.state_dtype == KDA_BF16;
  if (qb) return sb ? scan_types<__nv_bfloat16, __nv_bfloat16>(a, st) : scan_types<__nv_bfloat16, float>(a, st);
  return sb ? scan_types<float, __nv_bfloat16>(a, st) : scan_types<float, float>(a, st);
}

}  // namespace kda
