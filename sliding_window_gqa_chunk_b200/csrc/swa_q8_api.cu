// swa_q8_api.cu - the extern "C" entry points of the 8-bit rolling cache and of
// the rotary positions (declared in swa.h): argument checks, workspace layout
// and dispatch.  Every check that the host can make is made before the first
// launch; nothing here allocates.
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cmath>

#include "swa.h"
#include "swa_internal.h"

namespace {

// NVTX range around the entry point (see swa_api.cu).
struct CallRange {
  explicit CallRange(const char* name) { nvtxRangePushA(name); }
  ~CallRange() { nvtxRangePop(); }
};

// Slot arithmetic of the q8 kernels is in 32 bits with room for a few blocks.
constexpr int kMaxWindow = 1 << 30;

int check_q8_dims(const swa_dims* dims) {
  const int rc = swa::api_check_dims(dims);
  if (rc) return rc;
  if (dims->window > kMaxWindow)
    return swa::api_fail(SWA_ERR_UNSUPPORTED, "window %d above 2^30 for an 8-bit cache", dims->window);
  return SWA_OK;
}

int check_cache(const swa_q8_cache* c, swa::Q8Ring* ring) {
  if (c == nullptr) return swa::api_fail(SWA_ERR_INVALID_ARG, "cache is NULL");
  int rc = swa::api_check_ptrs("cache k, v, k_tail, v_tail", {c->k, c->v, c->k_tail, c->v_tail});
  if (rc) return rc;
  if ((rc = swa::api_check_ptrs4("cache k_scale, v_scale", {c->k_scale, c->v_scale}))) return rc;
  if (c->format != SWA_Q8_E4M3 && c->format != SWA_Q8_INT8)
    return swa::api_fail(SWA_ERR_INVALID_ARG, "cache format %d unknown", c->format);
  ring->k8 = static_cast<uint8_t*>(c->k);
  ring->v8 = static_cast<uint8_t*>(c->v);
  ring->k_scale = c->k_scale;
  ring->v_scale = c->v_scale;
  ring->k_tail = static_cast<__nv_bfloat16*>(c->k_tail);
  ring->v_tail = static_cast<__nv_bfloat16*>(c->v_tail);
  ring->format = c->format;
  return SWA_OK;
}

int check_max_tokens(const swa_dims* dims, int32_t max_tokens) {
  if (max_tokens < 1 || max_tokens > dims->window)
    return swa::api_fail(SWA_ERR_INVALID_ARG, "max_tokens %d not in [1, window=%d]", max_tokens, dims->window);
  return SWA_OK;
}

int cuda_fail(cudaError_t e, const char* what) {
  return swa::api_fail(SWA_ERR_CUDA, "%s launch: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

// Layout of the prefill workspace: the prefill kernel's own part first (it
// stays zero between calls), then the ring in bf16, keys before values.
size_t ring_offset(const swa_dims* dims, int32_t max_tokens) {
  return (swa_prefill_workspace_size(dims, max_tokens) + 1023) / 1024 * 1024;
}
size_t ring_bytes(const swa_dims* dims) {   // of the keys or of the values
  return (size_t)dims->batch * dims->n_kv_heads * dims->window * dims->head_dim * sizeof(__nv_bfloat16);
}

swa::Q8DecodeSplit split_of(const swa_dims* dims, int groups, bool chunk) {
  return swa::q8_decode_split(dims->batch, dims->n_kv_heads, dims->window, dims->head_dim, groups, chunk,
                              dims->n_q_heads / dims->n_kv_heads > 8);
}

// Fills in what decode steps and short chunks share, and launches.
int launch_over_ring(swa::Q8DecodeParams& p, const swa_dims* dims, const swa_q8_cache* cache, void* out, const void* q,
                     const void* k, const void* v, const int32_t* pos, const swa::Q8DecodeSplit& shape_split, void* stream,
                     const char* what) {
  const swa::Q8DecodeSplit sp =
      swa::q8_fit_clusters(shape_split, (long long)dims->batch * dims->n_kv_heads * p.groups, dims->window);
  p.out = out;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_new = static_cast<const __nv_bfloat16*>(k);
  p.v_new = static_cast<const __nv_bfloat16*>(v);
  p.pos = pos;
  p.batch = dims->batch;
  p.n_q_heads = dims->n_q_heads;
  p.n_kv_heads = dims->n_kv_heads;
  p.head_dim = dims->head_dim;
  p.window = dims->window;
  p.n_splits = sp.n_splits;
  p.slots_per_split = sp.slots_per_split;
  p.trace = swa::api_trace();
  p.variant = sp.variant;
  p.cluster = sp.cluster;
  p.scale_log2 = dims->scale * 1.4426950408889634f;
  p.out_f32 = dims->out_dtype == SWA_DTYPE_F32;
  int rc = swa::api_status_word(&p.status);
  if (rc) return rc;
  swa::Q8DecodeMaps maps;
  const long long pairs = (long long)dims->batch * dims->n_kv_heads;
  if ((rc = swa::api_encode_bytes(&maps.k, cache->k, dims->head_dim, dims->window, pairs, swa::kQ8Block, "cache k"))) return rc;
  if ((rc = swa::api_encode_bytes(&maps.v, cache->v, dims->head_dim, dims->window, pairs, swa::kQ8Block, "cache v"))) return rc;
  const cudaError_t e = swa::launch_q8_decode(p, maps, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, what);
  return swa::api_ok();
}

}  // namespace

extern "C" {

int swa_q8_append(const swa_dims* dims, const swa_q8_cache* cache, const void* k, const void* v, int32_t max_tokens,
                  const int32_t* start_pos, const int32_t* n_tokens, void* stream) {
  CallRange range_("swa_q8_append");
  int rc = check_q8_dims(dims);
  if (rc) return rc;
  swa::Q8AppendParams p;
  if ((rc = check_cache(cache, &p.ring))) return rc;
  if ((rc = swa::api_check_ptrs("k, v", {k, v}))) return rc;
  if ((rc = swa::api_check_ptrs4("start_pos, n_tokens", {start_pos, n_tokens}))) return rc;
  if ((rc = check_max_tokens(dims, max_tokens))) return rc;
  if ((rc = swa::api_status_word(&p.status))) return rc;
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.start_pos = start_pos;
  p.n_tokens = n_tokens;
  p.batch = dims->batch;
  p.n_kv_heads = dims->n_kv_heads;
  p.head_dim = dims->head_dim;
  p.window = dims->window;
  p.max_tokens = max_tokens;
  const cudaError_t e = swa::launch_q8_append(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "swa_q8_append");
  return swa::api_ok();
}

size_t swa_q8_prefill_workspace_size(const swa_dims* dims, int32_t max_tokens) {
  if (check_q8_dims(dims) != SWA_OK || check_max_tokens(dims, max_tokens) != SWA_OK) return 0;
  return ring_offset(dims, max_tokens) + 2 * ring_bytes(dims);
}

int swa_q8_prefill_chunk(const swa_dims* dims, void* out, const void* q, const void* k, const void* v,
                         int32_t max_tokens, const swa_q8_cache* cache, const int32_t* start_pos,
                         const int32_t* n_tokens, void* workspace, size_t workspace_bytes, void* stream) {
  CallRange range_("swa_q8_prefill_chunk");
  int rc = check_q8_dims(dims);
  if (rc) return rc;
  swa::Q8ExpandParams p;
  if ((rc = check_cache(cache, &p.ring))) return rc;
  if ((rc = swa::api_check_ptrs("out, q, k, v, workspace", {out, q, k, v, workspace}))) return rc;
  if ((rc = swa::api_check_ptrs4("start_pos, n_tokens", {start_pos, n_tokens}))) return rc;
  if ((rc = check_max_tokens(dims, max_tokens))) return rc;
  const size_t need = swa_q8_prefill_workspace_size(dims, max_tokens);
  if (workspace_bytes < need)
    return swa::api_fail(SWA_ERR_WORKSPACE_TOO_SMALL, "q8 prefill workspace of %zu bytes, %zu needed",
                         workspace_bytes, need);
  const int groups = swa::q8_chunk_groups(max_tokens, dims->n_q_heads / dims->n_kv_heads,
                                          (long long)dims->batch * dims->n_kv_heads, dims->window);
  if (groups > 0 && (long long)dims->n_kv_heads * groups <= 65535) {   // CTAs along the grid's second axis
    // few columns: straight over the ring's bytes
    swa::Q8DecodeParams d;
    d.ring = p.ring;
    d.ws_o = d.ws_ml = nullptr;
    d.n_tokens = n_tokens;
    d.max_tokens = max_tokens;
    d.groups = groups;
    const swa::Q8DecodeSplit sp = split_of(dims, d.groups, true);
    return launch_over_ring(d, dims, cache, out, q, k, v, start_pos, sp, stream, "swa_q8_prefill_chunk");
  }
  // the prefill's own limit, before the ring is expanded: a refused call enqueues nothing
  const int hpc = swa::prefill_heads_per_cta(dims->n_q_heads, dims->n_kv_heads);
  const long long n_units =
      (long long)dims->batch * (dims->n_q_heads / hpc) * (((long long)max_tokens + 127) / 128);
  if (n_units > (1LL << 29))
    return swa::api_fail(SWA_ERR_UNSUPPORTED, "%lld query tiles x head pairs in one call (limit 2^29)", n_units);
  const size_t at = ring_offset(dims, max_tokens);
  p.k_out = reinterpret_cast<__nv_bfloat16*>(static_cast<char*>(workspace) + at);
  p.v_out = reinterpret_cast<__nv_bfloat16*>(static_cast<char*>(workspace) + at + ring_bytes(dims));
  p.start_pos = start_pos;
  p.n_tokens = n_tokens;
  p.batch = dims->batch;
  p.n_kv_heads = dims->n_kv_heads;
  p.head_dim = dims->head_dim;
  p.window = dims->window;
  p.max_tokens = max_tokens;
  const cudaError_t e = swa::launch_q8_expand(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "swa_q8_prefill_chunk");
  return swa_prefill_chunk(dims, out, q, k, v, max_tokens, p.k_out, p.v_out, start_pos, n_tokens, workspace, at,
                           stream);
}

size_t swa_q8_decode_workspace_size(const swa_dims* dims) {
  if (check_q8_dims(dims) != SWA_OK) return 0;
  const swa::Q8DecodeSplit sp = split_of(dims, 1, false);
  if (sp.n_splits == 1 || sp.cluster) return 16;  // nothing needed; a non-zero size keeps callers simple
  return (size_t)dims->batch * dims->n_q_heads * sp.n_splits * (dims->head_dim + 4) * sizeof(float);
}

int swa_q8_decode(const swa_dims* dims, void* out, const void* q, const void* k_new, const void* v_new,
                  const swa_q8_cache* cache, const int32_t* pos, void* workspace, size_t workspace_bytes,
                  void* stream) {
  CallRange range_("swa_q8_decode");
  int rc = check_q8_dims(dims);
  if (rc) return rc;
  swa::Q8DecodeParams p;
  if ((rc = check_cache(cache, &p.ring))) return rc;
  if ((rc = swa::api_check_ptrs("out, q, k_new, v_new, workspace", {out, q, k_new, v_new, workspace}))) return rc;
  if ((rc = swa::api_check_ptrs4("pos", {pos}))) return rc;
  const size_t need = swa_q8_decode_workspace_size(dims);
  if (workspace_bytes < need)
    return swa::api_fail(SWA_ERR_WORKSPACE_TOO_SMALL, "q8 decode workspace of %zu bytes, %zu needed",
                         workspace_bytes, need);
  const swa::Q8DecodeSplit sp = split_of(dims, 1, false);
  p.ws_o = static_cast<float*>(workspace);
  p.ws_ml = p.ws_o + (size_t)dims->batch * dims->n_q_heads * sp.n_splits * dims->head_dim;
  p.n_tokens = nullptr;
  p.max_tokens = 1;
  p.groups = 1;
  return launch_over_ring(p, dims, cache, out, q, k_new, v_new, pos, sp, stream, "swa_q8_decode");
}

int swa_rope(const swa_dims* dims, const swa_rope_spec* spec, void* q_out, void* k_out, const void* q, const void* k,
             int64_t q_stride, int64_t k_stride, int32_t max_tokens, const int32_t* start_pos,
             const int32_t* n_tokens, int32_t transpose, void* stream) {
  CallRange range_("swa_rope");
  int rc = swa::api_check_dims(dims);
  if (rc) return rc;
  if (spec == nullptr) return swa::api_fail(SWA_ERR_INVALID_ARG, "spec is NULL");
  if ((rc = swa::api_check_ptrs("q_out, q", {q_out, q}))) return rc;
  if ((k == nullptr) != (k_out == nullptr))
    return swa::api_fail(SWA_ERR_INVALID_ARG, "one of k, k_out is NULL and the other is not");
  if (k != nullptr && (rc = swa::api_check_ptrs("k_out, k", {k_out, k}))) return rc;
  if ((rc = swa::api_check_ptrs4("inv_freq, start_pos", {spec->inv_freq, start_pos}))) return rc;
  if (n_tokens != nullptr && (rc = swa::api_check_ptrs4("n_tokens", {n_tokens}))) return rc;
  const int d = dims->head_dim, r = spec->rotary_dim;
  if (r < 16 || r > d || r % 16 != 0)
    return swa::api_fail(SWA_ERR_UNSUPPORTED, "rotary_dim %d is not a multiple of 16 in [16, head_dim=%d]", r, d);
  if (!(spec->factor > 0.f) || !std::isfinite(spec->factor))
    return swa::api_fail(SWA_ERR_INVALID_ARG, "factor must be finite and > 0");
  if ((spec->interleaved | transpose) & ~1)
    return swa::api_fail(SWA_ERR_INVALID_ARG, "interleaved %d / transpose %d is neither 0 nor 1", spec->interleaved,
                         transpose);
  if (max_tokens < 1 || (long long)dims->batch * max_tokens >= (1LL << 31))
    return swa::api_fail(SWA_ERR_INVALID_ARG, "max_tokens %d with batch %d: need 1 <= max_tokens, B * max_tokens < 2^31",
                         max_tokens, dims->batch);
  const int64_t q_row = (int64_t)dims->n_q_heads * d, k_row = (int64_t)dims->n_kv_heads * d;
  if (q_stride < q_row || q_stride % 8 != 0 || (k != nullptr && (k_stride < k_row || k_stride % 8 != 0)))
    return swa::api_fail(SWA_ERR_INVALID_ARG, "row strides (%lld, %lld) must be multiples of 8 and at least (%lld, %lld)",
                         (long long)q_stride, (long long)k_stride, (long long)q_row, (long long)k_row);
  if ((q == q_out && q_stride != q_row) || (k != nullptr && k == k_out && k_stride != k_row))
    return swa::api_fail(SWA_ERR_INVALID_ARG, "in place only for dense rows");
  swa::RopeParams p;
  if ((rc = swa::api_status_word(&p.status))) return rc;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.inv_freq = spec->inv_freq;
  p.start_pos = start_pos;
  p.n_tokens = n_tokens;
  p.batch = dims->batch;
  p.n_q_heads = dims->n_q_heads;
  p.n_kv_heads = k != nullptr ? dims->n_kv_heads : 0;
  p.head_dim = d;
  p.max_tokens = max_tokens;
  p.rotary_dim = r;
  p.interleaved = spec->interleaved;
  p.q_in_place = q == q_out;
  p.k_in_place = k == k_out;
  p.factor = spec->factor;
  p.sin_sign = transpose ? -1.f : 1.f;
  const cudaError_t e = swa::launch_rope(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "swa_rope");
  return swa::api_ok();
}

}  // extern "C"
