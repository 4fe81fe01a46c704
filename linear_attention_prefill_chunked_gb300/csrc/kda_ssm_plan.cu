// kda_ssm_plan.cu -- the planning kernel of the state space scan, and the kernel that adds up the states
// along the parts of a cut sequence.
#include "kda_ssm_plan.cuh"

#include <algorithm>

namespace kda {
namespace {

// ---- planning: the work lists ---------------------------------------------------------------------
// One block, in front of the scan on its stream; it writes the whole header, so that nothing has to be
// cleared before. Entries are sorted by chunk count, most first (a counting sort), as items are claimed
// in the list's order: an item claimed last is a short one.
//
// Cuts. A worker's share is L = chunks x items a sequence / workers. A sequence of many more than
// S = max(1.2 L, min_part) chunks would outlast the others: one of more than 1.5 S + 4 is cut into parts
// of at most S. A pass that forms states only (0.45 of a chunk's time on the tensor cores, 0.6 on CUDA
// cores) takes all parts but the last, each from a zero state; a kernel adds up S_end = decay S_start +
// S_local along the parts; then all parts run at once, each from its own start. One sequence of 64 heads
// takes 115 us for 8192 tokens (of 276 uncut), 50 us for 2048 (74); 1024 tokens stay whole (40, cut 51).
// S and so the parts' number follow from the lengths, the heads and the GPU alone: parts of more
// than S / 2 chunks, at most 2 / 1.2 CTAs' worth of items, for which the scratch has room.
constexpr int kPlanThreads = 1024, kKeys = 1024;

__global__ void __launch_bounds__(kPlanThreads)
ssm_plan_kernel(const int32_t* __restrict__ cu, const int32_t* __restrict__ idx, int N, int64_t T,
                int64_t num_slots, int items, int workers, int cap, int min_part, PlanHdr* hdr, Entry* full,
                Entry* state, Split* splits) {
  __shared__ uint32_t s_at[2][kKeys];  // entries of a chunk count, then where they go: full, state list
  __shared__ uint32_t s_scan[2][kPlanThreads / 32];
  __shared__ unsigned long long s_chunks;
  __shared__ uint32_t s_parts, s_splits;
  const int tid = threadIdx.x;
  tc::grid_dep_launch_dependents();
  check_all(&hdr->status, cu, idx, N, T, T, idx ? num_slots : 0);
  if (tid == 0) {
    s_chunks = 0;
    s_parts = s_splits = 0;
  }
  s_at[0][tid] = s_at[1][tid] = 0;
  __syncthreads();
  auto chunks_of = [&](int n) -> int64_t {  // -1: not run
    int64_t a, b;
    if (!seq_bounds(cu, n, T, &a, &b) || (idx && resolve_slot(idx, n, num_slots) < 0)) return -1;
    return (b - a + kSsmChunk - 1) / kSsmChunk;
  };
  unsigned long long mine = 0;
  for (int n = tid; n < N; n += kPlanThreads) {
    const int64_t c = chunks_of(n);
    if (c > 0) mine += (unsigned long long)c;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if ((tid & 31) == 0) atomicAdd(&s_chunks, mine);
  __syncthreads();
  // S = ceil(1.2 L) in whole numbers
  const unsigned long long work = s_chunks * (unsigned)items;
  int64_t S = (int64_t)((work * 6 + 5ull * workers - 1) / (5ull * workers));
  if (S < min_part) S = min_part;
  const int64_t most = cap == 0 ? INT64_MAX : S + S / 2 + 4;  // chunks of a sequence that stays whole
  auto key = [](int64_t len) { return (int)(len < kKeys - 1 ? len : kKeys - 1); };
  for (int n = tid; n < N; n += kPlanThreads) {
    const int64_t c = chunks_of(n);
    if (c < 0) continue;
    const int64_t m = c > most ? (c + S - 1) / S : 1, len = (c + m - 1) / m;
    const int64_t whole = m > 1 ? c / len : 1, tail = m > 1 ? c - whole * len : 0;  // full parts, the rest
    atomicAdd(&s_at[0][key(len)], (uint32_t)whole);
    if (tail > 0) atomicAdd(&s_at[0][key(tail)], 1u);
    if (m > 1) atomicAdd(&s_at[1][key(len)], (uint32_t)(tail > 0 ? whole : whole - 1));
  }
  __syncthreads();
  // where each count's entries begin: an exclusive scan from the largest count down
#pragma unroll 1
  for (int l = 0; l < 2; ++l) {
    const int k = kKeys - 1 - tid;
    const uint32_t v = s_at[l][k];
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if ((tid & 31) >= o) x += y;
    }
    if ((tid & 31) == 31) s_scan[l][tid >> 5] = x;
    __syncthreads();
    uint32_t before = 0, all = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w < (tid >> 5)) before += s_scan[l][w];
      all += s_scan[l][w];
    }
    s_at[l][k] = before + x - v;
    if (tid == 0) (l == 0 ? hdr->n_full : hdr->n_state) = all;
    __syncthreads();
  }
  for (int n = tid; n < N; n += kPlanThreads) {
    const int64_t c = chunks_of(n);
    if (c < 0) continue;
    const int64_t m = c > most ? (c + S - 1) / S : 1, len = (c + m - 1) / m;
    if (m == 1) {
      full[atomicAdd(&s_at[0][key(len)], 1u)] = Entry{n, 0, (int)c, -1, 1, {0, 0, 0}};
      continue;
    }
    const int parts = (int)((c + len - 1) / len);
    const int p0 = (int)atomicAdd(&s_parts, (uint32_t)parts);
    splits[atomicAdd(&s_splits, 1u)] = Split{p0, parts, idx ? resolve_slot(idx, n, num_slots) : n};
    for (int i = 0; i < parts; ++i) {
      const int64_t left = c - i * len;
      const Entry e{n, (int)(i * len), (int)(left < len ? left : len), p0 + i, i == parts - 1, {0, 0, 0}};
      full[atomicAdd(&s_at[0][key(e.nchunks)], 1u)] = e;
      if (i < parts - 1) state[atomicAdd(&s_at[1][key(len)], 1u)] = e;
    }
  }
  __syncthreads();
  if (tid == 0) {
    hdr->next_state = hdr->next_full = 0;
    hdr->n_splits = s_splits;
  }
}

// The state before each part of the cut sequences, four elements a thread: the initial one, then
// S_end = decay S_start + what the part adds. The next part's are read before they are wanted.
template <typename ST>
__global__ void __launch_bounds__(256)
ssm_combine_kernel(const PlanHdr* __restrict__ hdr, const Split* __restrict__ splits, float* scratch,
                   const float* __restrict__ decay, const ST* __restrict__ state_in, int64_t slot_stride, int H,
                   int KV) {
  tc::grid_dep_launch_dependents();
  tc::grid_dep_wait();
  const int64_t whole = (int64_t)H * KV;
  const int64_t at = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 4;
  if (at >= whole) return;
  const int h = (int)(at / KV);
  for (uint32_t i = blockIdx.y; i < hdr->n_splits; i += gridDim.y) {
    const Split sp = splits[i];
    float s[4] = {0.f, 0.f, 0.f, 0.f}, l[4], n[4];
    if (state_in) load4(state_in + sp.slot * slot_stride + at, s);
    float* part = scratch + sp.part0 * whole + at;
    load4(part + whole, n);
    for (int q = 0; q + 1 < sp.parts; ++q, part += whole) {
#pragma unroll
      for (int u = 0; u < 4; ++u) l[u] = n[u];
      if (q + 2 < sp.parts) load4(part + 2 * whole, n);
      const float d = decay[(sp.part0 + q) * H + h];
      store4(part, s);
#pragma unroll
      for (int u = 0; u < 4; ++u) s[u] = fmaf(d, s[u], l[u]);
    }
    store4(part, s);
  }
}

}  // namespace

int gpu_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) == cudaSuccess &&
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && n > 0)
    return n;
  (void)cudaGetLastError();
  return 152;
}

namespace {
// Offsets behind the header: the list of sequences, then what cuts need.
struct Layout {
  int cap;
  size_t full, lists_end, state, splits, decay, scratch, end;
};
Layout layout(const kda_desc_t& d, int items, int workers) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  Layout l;
  l.cap = 2 * workers / items + 2;  // 2 / 1.2 workers' worth of items, rounded up
  size_t at = kWsPayload;
  l.full = at;
  at += up(sizeof(Entry) * ((size_t)d.num_seqs + l.cap));
  l.lists_end = at;
  l.state = at;
  at += up(sizeof(Entry) * (size_t)l.cap);
  l.splits = at;
  at += up(sizeof(Split) * (size_t)l.cap);
  l.decay = at;
  at += up(sizeof(float) * (size_t)l.cap * d.num_v_heads);
  l.scratch = at;
  at += sizeof(float) * (size_t)l.cap * d.num_v_heads * d.head_k_dim * d.head_v_dim;
  l.end = at;
  return l;
}
}  // namespace

// Where no sequence can be long enough to be cut, none is long enough for its place in the order to
// matter: the sequences are taken as they come, in one launch.
static bool may_cut(const kda_desc_t& d, int min_part) {
  return d.total_tokens > (int64_t)(min_part + min_part / 2 + 4) * kSsmChunk;
}

size_t ssm_plan_workspace(const kda_desc_t& d, int items, int workers, int min_part) {
  return may_cut(d, min_part) ? layout(d, items, workers).end : kWsPayload;
}

SsmPlan ssm_plan(const SsmArgs& a, int items, int workers, int min_part) {
  const Layout l = layout(a.d, items, workers);
  SsmPlan p;
  p.lists = a.ws_bytes >= l.lists_end && may_cut(a.d, min_part);
  p.cap = p.lists && a.ws_bytes >= l.end ? l.cap : 0;
  p.items = items;
  p.workers = workers;
  p.min_part = min_part;
  p.hdr = reinterpret_cast<PlanHdr*>(a.ws);
  p.full = reinterpret_cast<Entry*>(a.ws + l.full);
  p.state = reinterpret_cast<Entry*>(a.ws + l.state);
  p.splits = reinterpret_cast<Split*>(a.ws + l.splits);
  p.decay = reinterpret_cast<float*>(a.ws + l.decay);
  p.scratch = reinterpret_cast<float*>(a.ws + l.scratch);
  return p;
}

cudaError_t launch_ssm_plan(const SsmPlan& p, const SsmArgs& a, cudaStream_t st) {
  ssm_plan_kernel<<<1, kPlanThreads, 0, st>>>(a.cu, a.idx, a.d.num_seqs, a.d.total_tokens, a.d.num_slots,
                                              p.items, p.workers, p.cap, p.min_part, p.hdr, p.full, p.state,
                                              p.splits);
  return cudaGetLastError();
}

cudaError_t launch_ssm_combine(const SsmPlan& p, const SsmArgs& a, cudaStream_t st) {
  const int kv = a.d.head_k_dim * a.d.head_v_dim;
  const int64_t whole = (int64_t)a.d.num_v_heads * kv;
  const dim3 grid((unsigned)((whole / 4 + 255) / 256), (unsigned)std::min(p.cap / 2, 16));
  if (a.d.state_dtype == KDA_BF16)
    return launch_pass(ssm_combine_kernel<__nv_bfloat16>, grid, 256, 0, true, st, p.hdr, p.splits, p.scratch,
                       p.decay, (const __nv_bfloat16*)a.state_in, a.slot_stride, a.d.num_v_heads, kv);
  return launch_pass(ssm_combine_kernel<float>, grid, 256, 0, true, st, p.hdr, p.splits, p.scratch, p.decay,
                     (const float*)a.state_in, a.slot_stride, a.d.num_v_heads, kv);
}

}  // namespace kda
