// kda_layer_api.cu -- the extern "C" boundary of the operators around the recurrence: argument
// checks and dispatch of the short convolution, the state space scan, verification and commit.
#include "kda_internal.cuh"

namespace {

bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }
bool ws_ok(const void* ws) { return ws && (uintptr_t)ws % 256 == 0; }
uint32_t* status_of(void* ws) { return &reinterpret_cast<kda::WsHeader*>(ws)->status; }

// A clear status word for a call without work (and for every call of the debug build, whose
// kernels add to the word).
kda_status_t clear_status(void* ws, cudaStream_t st) {
  return cudaMemsetAsync(ws, 0, sizeof(kda::WsHeader), st) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

// Launches through `f` after an error left by earlier, unrelated work is cleared, so that the
// result reports this call's own launches.
template <typename F> kda_status_t launched(void* ws, cudaStream_t st, F f) {
  (void)cudaGetLastError();
#ifdef KDA_DEBUG
  if (clear_status(ws, st) != KDA_OK) return KDA_ERR_CUDA;
#else
  (void)ws;
  (void)st;
#endif
  return f() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

bool conv_ok(const kda_conv_desc_t* d) {
  return d && d->num_seqs >= 0 && d->total_tokens >= 0 && d->channels > 0 && d->width >= 2 &&
         d->width <= 4 && (d->dtype == KDA_BF16 || d->dtype == KDA_F32) &&
         (d->silu == 0 || d->silu == 1) && d->x_pitch >= d->channels;
}
// grid.y holds the channel blocks; 32 channels a block at least
bool conv_fits(const kda_conv_desc_t* d) { return d->channels <= 65535 * 32; }

bool elem_aligned(const void* p, kda_dtype_t t) { return (uintptr_t)p % (t == KDA_BF16 ? 2 : 4) == 0; }

bool ssm_ok(const kda_desc_t* d) {
  return d && d->num_seqs >= 0 && d->total_tokens >= 0 && d->num_k_heads > 0 &&
         d->num_v_heads > 0 && d->num_v_heads % d->num_k_heads == 0 &&
         (d->flags & ~KDA_FLAG_CUDA_CORE_PATH) == 0 &&
         (d->qkv_dtype == KDA_BF16 || d->qkv_dtype == KDA_F32) &&
         (d->state_dtype == KDA_BF16 || d->state_dtype == KDA_F32);
}
bool ssm_supported(const kda_desc_t* d) {
  return (d->head_k_dim == 64 || d->head_k_dim == 128) &&
         (d->head_v_dim == 64 || d->head_v_dim == 128) && d->num_v_heads <= 65535;
}
int64_t ssm_state_elems(const kda_desc_t* d) {
  return (int64_t)d->num_v_heads * d->head_k_dim * d->head_v_dim;
}
bool ssm_inputs_ok(const kda_desc_t* d, const kda_ssm_inputs_t* in) {
  const int64_t hv = (int64_t)d->num_v_heads * d->head_v_dim;
  const int64_t gk = (int64_t)d->num_k_heads * d->head_k_dim;
  const int64_t e16 = d->qkv_dtype == KDA_BF16 ? 8 : 4;  // elements of 16 bytes
  if (!in || !in->a_log) return false;
  if (d->total_tokens > 0 && (!in->x || !in->dt || !in->b || !in->c)) return false;
  if (in->x_pitch < hv || in->b_pitch < gk || in->c_pitch < gk || in->dt_pitch < d->num_v_heads)
    return false;
  if (in->x_pitch % e16 || in->b_pitch % e16 || in->c_pitch % e16) return false;
  return aligned16(in->x) && aligned16(in->b) && aligned16(in->c) &&
         elem_aligned(in->dt, d->qkv_dtype);
}

bool gated_ok(const kda_gated_desc_t* d) {
  return d && d->num_seqs >= 0 && d->total_tokens >= 0 && d->total_tokens <= 0x7fffffffll && d->channels > 0 &&
         (d->dtype == KDA_BF16 || d->dtype == KDA_F32);
}
bool gated_inputs_ok(const kda_gated_desc_t* d, const void* x, const void* r, const void* i, const float* a_log) {
  if (!a_log || !elem_aligned(a_log, KDA_F32) || (d->total_tokens > 0 && (!x || !r))) return false;
  return elem_aligned(x, d->dtype) && elem_aligned(r, d->dtype) && elem_aligned(i, d->dtype) &&
         d->x_pitch >= d->channels && d->r_pitch >= d->channels && (!i || d->i_pitch >= d->channels);
}

bool sample_ok(const kda_sample_desc_t* d, const float* temperature, const int32_t* top_k, const float* top_p,
               const float* min_p) {
  if (!d || d->num_rows < 0 || d->vocab <= 0 || d->logits_pitch < d->vocab ||
      !(d->dtype == KDA_BF16 || d->dtype == KDA_F32))
    return false;
  if (!temperature && !(d->temperature >= 0.f)) return false;
  if ((!top_p && d->top_p != d->top_p) || (!min_p && d->min_p != d->min_p)) return false;
  const void* ptrs[] = {temperature, top_k, top_p, min_p};
  for (const void* p : ptrs)
    if ((uintptr_t)p % 4 != 0) return false;
  return true;
}

}  // namespace

extern "C" {

kda_status_t kda_causal_conv(const kda_conv_desc_t* d, const void* x, const void* weight,
                             const void* bias, const int32_t* cu_seqlens, void* state,
                             const int32_t* state_indices, void* final_state, void* y,
                             void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!conv_ok(d) || !weight || !cu_seqlens || !ws_ok(workspace)) return KDA_ERR_INVALID_ARGUMENT;
  if (!conv_fits(d)) return KDA_ERR_UNSUPPORTED;
  if (d->total_tokens > 0 && (!x || !y)) return KDA_ERR_INVALID_ARGUMENT;
  const int64_t row = (int64_t)(d->width - 1) * d->channels;
  const bool pool = state_indices != nullptr;
  const int64_t stride = pool && d->slot_stride_elems != 0 ? d->slot_stride_elems : row;
  if (pool && (!state || d->num_slots <= 0 || stride < row ||
               (final_state != nullptr && final_state != state)))
    return KDA_ERR_INVALID_ARGUMENT;
  {
    const void* ptrs[] = {x, weight, bias, state, final_state, y};
    for (const void* p : ptrs)
      if (!elem_aligned(p, d->dtype)) return KDA_ERR_INVALID_ARGUMENT;
  }
  if (workspace_bytes < KDA_STATUS_WORKSPACE_BYTES) return KDA_ERR_WORKSPACE_TOO_SMALL;
  if (d->num_seqs == 0) return clear_status(workspace, stream);
  kda::ConvArgs a{};
  a.d = *d;
  a.x = x; a.w = weight; a.bias = bias; a.cu = cu_seqlens;
  a.state_in = state;
  a.idx = state_indices;
  a.state_out = pool ? state : final_state;
  a.slot_stride = stride;
  a.y = y;
  a.status = status_of(workspace);
  return launched(workspace, stream, [&] { return kda::launch_conv(a, stream); });
}

kda_status_t kda_causal_conv_decode(const kda_conv_desc_t* d, const void* x, const void* weight,
                                    const void* bias, const int32_t* cu_seqlens, void* state_pool,
                                    const int32_t* state_indices, void* step_cache,
                                    int64_t cache_pitch_elems, int32_t max_steps, int update_pool,
                                    void* y, void* workspace, size_t workspace_bytes,
                                    cudaStream_t stream) {
  if (!conv_ok(d) || !weight || !ws_ok(workspace)) return KDA_ERR_INVALID_ARGUMENT;
  if (!conv_fits(d)) return KDA_ERR_UNSUPPORTED;
  if (d->total_tokens > 0 && (!x || !y)) return KDA_ERR_INVALID_ARGUMENT;
  if (!cu_seqlens && d->total_tokens != d->num_seqs) return KDA_ERR_INVALID_ARGUMENT;
  const int64_t row = (int64_t)(d->width - 1) * d->channels;
  const int64_t stride = d->slot_stride_elems != 0 ? d->slot_stride_elems : row;
  if ((d->num_seqs > 0 && !state_pool) || d->num_slots <= 0 || stride < row || max_steps < 1)
    return KDA_ERR_INVALID_ARGUMENT;
  if (step_cache && cache_pitch_elems < (int64_t)max_steps * row) return KDA_ERR_INVALID_ARGUMENT;
  {
    const void* ptrs[] = {x, weight, bias, state_pool, step_cache, y};
    for (const void* p : ptrs)
      if (!elem_aligned(p, d->dtype)) return KDA_ERR_INVALID_ARGUMENT;
  }
  if (workspace_bytes < KDA_STATUS_WORKSPACE_BYTES) return KDA_ERR_WORKSPACE_TOO_SMALL;
  if (d->num_seqs == 0) return clear_status(workspace, stream);
  kda::ConvArgs a{};
  a.d = *d;
  a.x = x; a.w = weight; a.bias = bias; a.cu = cu_seqlens;
  a.state_in = state_pool;
  a.idx = state_indices;
  a.state_out = state_pool;
  a.slot_stride = stride;
  a.y = y;
  a.status = status_of(workspace);
  a.cache = step_cache;
  a.cache_pitch = cache_pitch_elems;
  a.max_steps = cu_seqlens ? max_steps : 1;
  a.update_pool = update_pool != 0;
  return launched(workspace, stream, [&] { return kda::launch_conv_decode(a, stream); });
}

size_t kda_causal_conv_backward_workspace_size(const kda_conv_desc_t* d) {
  return conv_ok(d) && conv_fits(d) ? kda::conv_back_workspace(*d) : 0;
}

kda_status_t kda_causal_conv_backward(const kda_conv_desc_t* d, const void* dy, int64_t dy_pitch, const void* x,
                                      const void* weight, const void* bias, const int32_t* cu_seqlens,
                                      const void* state, const void* dfinal, void* dx, float* dweight,
                                      float* dbias, void* dstate, void* workspace, size_t workspace_bytes,
                                      cudaStream_t stream) {
  if (!conv_ok(d) || !weight || !cu_seqlens || !ws_ok(workspace) || !dweight || dy_pitch < d->channels)
    return KDA_ERR_INVALID_ARGUMENT;
  if (!conv_fits(d)) return KDA_ERR_UNSUPPORTED;
  if (d->total_tokens > 0 && (!x || !dy || !dx)) return KDA_ERR_INVALID_ARGUMENT;
  {
    const void* ptrs[] = {dy, x, weight, bias, state, dfinal, dx, dstate};
    for (const void* p : ptrs)
      if (!elem_aligned(p, d->dtype)) return KDA_ERR_INVALID_ARGUMENT;
  }
  if (!elem_aligned(dweight, KDA_F32) || !elem_aligned(dbias, KDA_F32)) return KDA_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < kda::conv_back_workspace(*d)) return KDA_ERR_WORKSPACE_TOO_SMALL;
  kda::ConvBackArgs a{};
  a.d = *d;
  a.dy = dy;
  a.dy_pitch = dy_pitch;
  a.x = x; a.w = weight; a.bias = bias; a.cu = cu_seqlens;
  a.state = state;
  a.dfinal = dfinal;
  a.dx = dx;
  a.dstate = dstate;
  a.dw = dweight;
  a.db = dbias;
  a.ws = static_cast<uint8_t*>(workspace);
  return launched(workspace, stream, [&] { return kda::launch_conv_back(a, stream); });
}

size_t kda_ssm_scan_workspace_size(const kda_desc_t* d) {
  if (!ssm_ok(d) || !ssm_supported(d)) return 0;
  return kda::ssm_tc_supported(*d) ? kda::ssm_tc_workspace(*d) : kda::ssm_simt_workspace(*d);
}

kda_status_t kda_ssm_scan(const kda_desc_t* d, const kda_ssm_inputs_t* in,
                          const int32_t* cu_seqlens, void* state, const int32_t* state_indices,
                          void* final_state, void* y, void* workspace, size_t workspace_bytes,
                          cudaStream_t stream) {
  if (!ssm_ok(d)) return KDA_ERR_INVALID_ARGUMENT;
  if (!ssm_supported(d)) return KDA_ERR_UNSUPPORTED;
  if (!ssm_inputs_ok(d, in) || !cu_seqlens || !ws_ok(workspace)) return KDA_ERR_INVALID_ARGUMENT;
  if (d->total_tokens > 0 && !y) return KDA_ERR_INVALID_ARGUMENT;
  const int64_t row = ssm_state_elems(d);
  const bool pool = state_indices != nullptr;
  const int64_t stride = pool && d->slot_stride_elems != 0 ? d->slot_stride_elems : row;
  if (pool && (!state || d->num_slots <= 0 || stride < row || stride % 8 != 0 ||
               (final_state != nullptr && final_state != state)))
    return KDA_ERR_INVALID_ARGUMENT;
  if (!aligned16(state) || !aligned16(final_state) || !aligned16(y)) return KDA_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < KDA_STATUS_WORKSPACE_BYTES) return KDA_ERR_WORKSPACE_TOO_SMALL;
  if (d->num_seqs == 0) return clear_status(workspace, stream);
  kda::SsmArgs a{};
  a.d = *d;
  a.in = *in;
  a.cu = cu_seqlens;
  a.state_in = state;
  a.idx = state_indices;
  a.state_out = pool ? state : final_state;
  a.slot_stride = stride;
  a.y = y;
  a.status = status_of(workspace);
  a.ws = static_cast<uint8_t*>(workspace);
  a.ws_bytes = workspace_bytes;
  return launched(workspace, stream, [&] {
    return kda::ssm_tc_supported(*d) ? kda::launch_ssm_tc(a, stream) : kda::launch_ssm_simt(a, stream);
  });
}

kda_status_t kda_ssm_decode(const kda_desc_t* d, const kda_ssm_inputs_t* in,
                            const int32_t* cu_seqlens, void* state_pool,
                            const int32_t* state_indices, void* step_cache,
                            int64_t cache_pitch_elems, int32_t max_steps, int update_pool, void* y,
                            void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!ssm_ok(d)) return KDA_ERR_INVALID_ARGUMENT;
  if (!ssm_supported(d)) return KDA_ERR_UNSUPPORTED;
  if (!ssm_inputs_ok(d, in) || !ws_ok(workspace)) return KDA_ERR_INVALID_ARGUMENT;
  if (d->total_tokens > 0 && !y) return KDA_ERR_INVALID_ARGUMENT;
  if (!cu_seqlens && d->total_tokens != d->num_seqs) return KDA_ERR_INVALID_ARGUMENT;
  const int64_t row = ssm_state_elems(d);
  const int64_t stride = d->slot_stride_elems != 0 ? d->slot_stride_elems : row;
  if ((d->num_seqs > 0 && !state_pool) || d->num_slots <= 0 || stride < row || stride % 8 != 0 ||
      max_steps < 1)
    return KDA_ERR_INVALID_ARGUMENT;
  if (step_cache && (cache_pitch_elems < (int64_t)max_steps * row || cache_pitch_elems % 8 != 0))
    return KDA_ERR_INVALID_ARGUMENT;
  if (!aligned16(state_pool) || !aligned16(step_cache) || !aligned16(y))
    return KDA_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < KDA_STATUS_WORKSPACE_BYTES) return KDA_ERR_WORKSPACE_TOO_SMALL;
  if (d->num_seqs == 0) return clear_status(workspace, stream);
  kda::SsmArgs a{};
  a.d = *d;
  a.in = *in;
  a.cu = cu_seqlens;
  a.state_in = state_pool;
  a.idx = state_indices;
  a.state_out = state_pool;
  a.slot_stride = stride;
  a.y = y;
  a.status = status_of(workspace);
  a.cache = step_cache;
  a.cache_pitch = cache_pitch_elems;
  a.max_steps = cu_seqlens ? max_steps : 1;
  a.update_pool = update_pool != 0;
  return launched(workspace, stream, [&] { return kda::launch_ssm_decode(a, stream); });
}

size_t kda_gated_scan_workspace_size(const kda_gated_desc_t* d) {
  return gated_ok(d) && kda::gated_fits(*d) ? kda::gated_scan_workspace(*d) : 0;
}

size_t kda_gated_scan_backward_workspace_size(const kda_gated_desc_t* d) {
  return gated_ok(d) && kda::gated_fits(*d) ? kda::gated_back_workspace(*d) : 0;
}

kda_status_t kda_gated_scan(const kda_gated_desc_t* d, const void* x, const void* r, const void* i,
                            const float* a_log, const int32_t* cu_seqlens, float* state,
                            const int32_t* state_indices, float* final_state, void* y, float* carries,
                            void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!gated_ok(d) || !gated_inputs_ok(d, x, r, i, a_log) || !cu_seqlens || !ws_ok(workspace))
    return KDA_ERR_INVALID_ARGUMENT;
  if (!kda::gated_fits(*d)) return KDA_ERR_UNSUPPORTED;
  if (d->total_tokens > 0 && !y) return KDA_ERR_INVALID_ARGUMENT;
  const bool pool = state_indices != nullptr;
  const int64_t stride = pool && d->slot_stride_elems != 0 ? d->slot_stride_elems : d->channels;
  if (pool && (!state || d->num_slots <= 0 || stride < d->channels ||
               (final_state != nullptr && final_state != state)))
    return KDA_ERR_INVALID_ARGUMENT;
  if (!elem_aligned(y, d->dtype) || !elem_aligned(state, KDA_F32) || !elem_aligned(final_state, KDA_F32) ||
      !elem_aligned(carries, KDA_F32))
    return KDA_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < kda::gated_scan_workspace(*d)) return KDA_ERR_WORKSPACE_TOO_SMALL;
  if (d->num_seqs == 0) return clear_status(workspace, stream);
  kda::GatedArgs a{};
  a.d = *d;
  a.x = x; a.r = r; a.i = i; a.a_log = a_log;
  a.cu = cu_seqlens;
  a.state_in = state;
  a.idx = state_indices;
  a.state_out = pool ? state : final_state;
  a.slot_stride = stride;
  a.y = y;
  a.carries = carries;
  a.ws = static_cast<uint8_t*>(workspace);
  return launched(workspace, stream, [&] { return kda::launch_gated_scan(a, stream); });
}

kda_status_t kda_gated_scan_backward(const kda_gated_desc_t* d, const void* dy, int64_t dy_pitch, const void* x,
                                     const void* r, const void* i, const float* a_log,
                                     const int32_t* cu_seqlens, const float* carries, const float* state,
                                     const float* dfinal, void* dx, void* dr, void* di, float* da_log,
                                     float* dstate, void* workspace, size_t workspace_bytes,
                                     cudaStream_t stream) {
  if (!gated_ok(d) || !gated_inputs_ok(d, x, r, i, a_log) || !cu_seqlens || !ws_ok(workspace) || !da_log ||
      dy_pitch < d->channels)
    return KDA_ERR_INVALID_ARGUMENT;
  if (!kda::gated_fits(*d)) return KDA_ERR_UNSUPPORTED;
  if (d->total_tokens > 0 && (!dy || !carries || !dx || !dr || !di != !i)) return KDA_ERR_INVALID_ARGUMENT;
  {
    const void* rows[] = {dy, dx, dr, di};
    for (const void* p : rows)
      if (!elem_aligned(p, d->dtype)) return KDA_ERR_INVALID_ARGUMENT;
    const void* floats[] = {carries, state, dfinal, da_log, dstate};
    for (const void* p : floats)
      if (!elem_aligned(p, KDA_F32)) return KDA_ERR_INVALID_ARGUMENT;
  }
  if (workspace_bytes < kda::gated_back_workspace(*d)) return KDA_ERR_WORKSPACE_TOO_SMALL;
  kda::GatedArgs a{};
  a.d = *d;
  a.x = x; a.r = r; a.i = i; a.a_log = a_log;
  a.cu = cu_seqlens;
  a.state_in = state;
  a.slot_stride = d->channels;
  a.carries = const_cast<float*>(carries);
  a.dy = dy;
  a.dy_pitch = dy_pitch;
  a.dfinal = dfinal;
  a.dx = dx; a.dr = dr; a.di = di;
  a.da_log = da_log;
  a.dstate = dstate;
  a.ws = static_cast<uint8_t*>(workspace);
  return launched(workspace, stream, [&] { return kda::launch_gated_back(a, stream); });
}

kda_status_t kda_gated_decode(const kda_gated_desc_t* d, const void* x, const void* r, const void* i,
                              const float* a_log, const int32_t* cu_seqlens, float* state_pool,
                              const int32_t* state_indices, float* step_cache, int64_t cache_pitch_elems,
                              int32_t max_steps, int update_pool, void* y, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream) {
  if (!gated_ok(d) || !gated_inputs_ok(d, x, r, i, a_log) || !ws_ok(workspace)) return KDA_ERR_INVALID_ARGUMENT;
  if (d->channels > 65535 * 128) return KDA_ERR_UNSUPPORTED;  // grid.y holds 128 channels a block at least
  if (d->total_tokens > 0 && !y) return KDA_ERR_INVALID_ARGUMENT;
  if (!cu_seqlens && d->total_tokens != d->num_seqs) return KDA_ERR_INVALID_ARGUMENT;
  const int64_t stride = d->slot_stride_elems != 0 ? d->slot_stride_elems : d->channels;
  if ((d->num_seqs > 0 && !state_pool) || d->num_slots <= 0 || stride < d->channels || max_steps < 1)
    return KDA_ERR_INVALID_ARGUMENT;
  if (step_cache && cache_pitch_elems / max_steps < d->channels) return KDA_ERR_INVALID_ARGUMENT;
  if (!elem_aligned(y, d->dtype) || !elem_aligned(state_pool, KDA_F32) || !elem_aligned(step_cache, KDA_F32))
    return KDA_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < KDA_STATUS_WORKSPACE_BYTES) return KDA_ERR_WORKSPACE_TOO_SMALL;
  if (d->num_seqs == 0) return clear_status(workspace, stream);
  kda::GatedArgs a{};
  a.d = *d;
  a.x = x; a.r = r; a.i = i; a.a_log = a_log;
  a.cu = cu_seqlens;
  a.state_in = a.state_out = state_pool;
  a.idx = state_indices;
  a.slot_stride = stride;
  a.y = y;
  a.ws = static_cast<uint8_t*>(workspace);
  a.cache = step_cache;
  a.cache_pitch = cache_pitch_elems;
  a.max_steps = cu_seqlens ? max_steps : 1;
  a.update_pool = update_pool != 0;
  return launched(workspace, stream, [&] { return kda::launch_gated_token(a, stream); });
}

kda_status_t kda_sample(const kda_sample_desc_t* d, const void* logits, const float* noise,
                        const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                        int32_t* token, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!sample_ok(d, temperature, top_k, top_p, min_p) || !ws_ok(workspace)) return KDA_ERR_INVALID_ARGUMENT;
  if (!kda::sample_fits(*d)) return KDA_ERR_UNSUPPORTED;
  if (d->num_rows > 0 && (!logits || !noise || !token)) return KDA_ERR_INVALID_ARGUMENT;
  if (!elem_aligned(logits, d->dtype) || !elem_aligned(noise, KDA_F32) || !elem_aligned(token, KDA_F32) ||
      d->noise_pitch < d->vocab)
    return KDA_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < KDA_STATUS_WORKSPACE_BYTES) return KDA_ERR_WORKSPACE_TOO_SMALL;
  if (d->num_rows == 0) return clear_status(workspace, stream);
  kda::SampleArgs a{*d, logits, noise, temperature, top_p, min_p, top_k, token, nullptr, status_of(workspace)};
  return launched(workspace, stream, [&] { return kda::launch_sample(a, stream); });
}

kda_status_t kda_sample_probs(const kda_sample_desc_t* d, const void* logits, const float* temperature,
                              const int32_t* top_k, const float* top_p, const float* min_p, float* probs,
                              void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!sample_ok(d, temperature, top_k, top_p, min_p) || !ws_ok(workspace)) return KDA_ERR_INVALID_ARGUMENT;
  if (!kda::sample_fits(*d)) return KDA_ERR_UNSUPPORTED;
  if (d->num_rows > 0 && (!logits || !probs)) return KDA_ERR_INVALID_ARGUMENT;
  if (!elem_aligned(logits, d->dtype) || !elem_aligned(probs, KDA_F32)) return KDA_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < KDA_STATUS_WORKSPACE_BYTES) return KDA_ERR_WORKSPACE_TOO_SMALL;
  if (d->num_rows == 0) return clear_status(workspace, stream);
  kda::SampleArgs a{*d, logits, nullptr, temperature, top_p, min_p, top_k, nullptr, probs, status_of(workspace)};
  return launched(workspace, stream, [&] { return kda::launch_sample(a, stream); });
}

kda_status_t kda_verify_draft(int32_t num_seqs, int64_t total_tokens, int32_t vocab,
                              const int32_t* tokens, const float* target_probs,
                              const float* draft_probs, const float* accept_u, const float* noise,
                              const int32_t* cu_seqlens, int32_t* num_accepted,
                              int32_t* next_token, void* workspace, size_t workspace_bytes,
                              cudaStream_t stream) {
  return kda_verify_draft_marked(num_seqs, total_tokens, vocab, tokens, target_probs, draft_probs, accept_u,
                                 noise, cu_seqlens, num_accepted, next_token, 0u, workspace, workspace_bytes,
                                 stream);
}

kda_status_t kda_verify_draft_marked(int32_t num_seqs, int64_t total_tokens, int32_t vocab,
                                     const int32_t* tokens, const float* target_probs,
                                     const float* draft_probs, const float* accept_u, const float* noise,
                                     const int32_t* cu_seqlens, int32_t* num_accepted,
                                     int32_t* next_token, uint32_t flags, void* workspace,
                                     size_t workspace_bytes, cudaStream_t stream) {
  if (num_seqs < 0 || total_tokens < 0 || vocab <= 0 || !cu_seqlens || !ws_ok(workspace) ||
      (flags & ~(KDA_VERIFY_MARK_COUNT | KDA_VERIFY_MARK_TOKEN)) != 0)
    return KDA_ERR_INVALID_ARGUMENT;
  if (num_seqs > (1 << 27)) return KDA_ERR_UNSUPPORTED;
  if (num_seqs > 0 && (!num_accepted || !next_token)) return KDA_ERR_INVALID_ARGUMENT;
  if (total_tokens > 0 && (!tokens || !target_probs || !accept_u || !noise))
    return KDA_ERR_INVALID_ARGUMENT;
  {
    const void* ptrs[] = {tokens, target_probs, draft_probs, accept_u, noise, num_accepted, next_token};
    for (const void* p : ptrs)
      if ((uintptr_t)p % 4 != 0) return KDA_ERR_INVALID_ARGUMENT;
  }
  if (workspace_bytes < KDA_STATUS_WORKSPACE_BYTES) return KDA_ERR_WORKSPACE_TOO_SMALL;
  if (num_seqs == 0) return clear_status(workspace, stream);
  return launched(workspace, stream, [&] {
    return kda::launch_verify(num_seqs, total_tokens, vocab, tokens, target_probs, draft_probs,
                              accept_u, noise, cu_seqlens, num_accepted, next_token,
                              status_of(workspace), flags, stream);
  });
}

kda_status_t kda_commit_draft(int32_t num_seqs, kda_dtype_t dtype, int64_t row_elems,
                              const void* step_cache, int64_t cache_pitch_elems, int32_t max_steps,
                              const int32_t* num_accepted, void* pool, int64_t num_slots,
                              int64_t slot_stride_elems, const int32_t* state_indices,
                              void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (num_seqs < 0 || row_elems <= 0 || max_steps < 1 || num_slots <= 0 || !ws_ok(workspace) ||
      !(dtype == KDA_BF16 || dtype == KDA_F32))
    return KDA_ERR_INVALID_ARGUMENT;
  const int64_t stride = slot_stride_elems != 0 ? slot_stride_elems : row_elems;
  if (stride < row_elems || cache_pitch_elems / max_steps < row_elems) return KDA_ERR_INVALID_ARGUMENT;
  if (num_seqs > 0 && (!step_cache || !num_accepted || !pool)) return KDA_ERR_INVALID_ARGUMENT;
  if (!elem_aligned(step_cache, dtype) || !elem_aligned(pool, dtype)) return KDA_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < KDA_STATUS_WORKSPACE_BYTES) return KDA_ERR_WORKSPACE_TOO_SMALL;
  if (num_seqs == 0) return clear_status(workspace, stream);
  return launched(workspace, stream, [&] {
    return kda::launch_commit(num_seqs, dtype == KDA_BF16 ? 2 : 4, row_elems, step_cache,
                              cache_pitch_elems, max_steps, num_accepted, pool, num_slots, stride,
                              state_indices, status_of(workspace), stream);
  });
}

}  // extern "C"
