// swa_internal.h - launch parameter blocks shared between the C-ABI layer
// (swa_api.cu) and the kernel files.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <initializer_list>

namespace swa {

struct AppendParams {
  __nv_bfloat16* k_cache;       // [B][Hkv][W][d]
  __nv_bfloat16* v_cache;
  const __nv_bfloat16* k;       // [B][max_tokens][Hkv][d]
  const __nv_bfloat16* v;
  const int32_t* start_pos;     // device [B]
  const int32_t* n_tokens;      // device [B]
  int* status;                  // device status word
  int batch, n_kv_heads, head_dim, window, max_tokens;
};

struct DecodeParams {
  void* out;                    // [B][Hq][d] bf16 or f32
  const __nv_bfloat16* q;       // [B][Hq][d]
  const __nv_bfloat16* k_new;   // [B][Hkv][d]
  const __nv_bfloat16* v_new;
  const __nv_bfloat16* k_cache; // [B][Hkv][W][d] (read path)
  const __nv_bfloat16* v_cache;
  __nv_bfloat16* k_cache_w;     // same buffers (write of slot pos mod W)
  __nv_bfloat16* v_cache_w;
  const int32_t* pos;           // device [B]
  float* ws_o;                  // [B][Hq][n_splits][d] partial O (n_splits > 1)
  float* ws_ml;                 // [B][Hq][n_splits][2] partial (max, sum), log2 domain
  int* status;
  int batch, n_q_heads, n_kv_heads, head_dim, window;
  int n_splits, slots_per_split;
  int warps;                    // warps per CTA
  int cluster;                  // 1: the n_splits CTAs of a (sequence, kv head) form a
                                // thread-block cluster and merge through distributed
                                // shared memory (no workspace, no combine kernel)
  int stream;                   // 1: a producer warp streams the slots into shared
                                // memory with bulk copies (few (sequence, kv head) pairs)
  float scale_log2;             // scale * log2(e)
  int out_f32;
};

// Largest thread-block cluster of decode split CTAs (the portable cluster size).
constexpr int kDecodeMaxClusterSplits = 8;

// Split of the W slots of one (sequence, kv head) across CTAs; depends only
// on the shape so that the workspace size is a function of the dims.
struct DecodeSplit {
  int n_splits;
  int slots_per_split;
  int warps;
  int cluster;
  int stream;
  int ws_splits;   // splits the workspace is sized for (fp32 partials per split)
};
DecodeSplit decode_split(int batch, int n_q_heads, int n_kv_heads, int window, int head_dim);

// Thread-block clusters of `cs` stream-variant decode CTAs (head dimension
// head_dim) that the current device holds at once, or -1 when it cannot be
// asked (no device).
int decode_resident_clusters(int head_dim, int cs);

struct PrefillParams {
  void* out;                    // [B][max_tokens][Hq][d] bf16 or f32
  const int32_t* start_pos;     // device [B]
  const int32_t* n_tokens;      // device [B]
  int* status;
  int batch, n_q_heads, n_kv_heads, head_dim, window, max_tokens;
  int heads_per_cta;            // 1 or 2 query heads of one kv group per CTA
  int n_q_tiles;                // ceil(max_tokens / 128)
  int n_whole;                  // work items that are whole units (query tile x head pair x sequence)
  int n_pieces;                 // pieces per split unit (units n_whole.. are split)
  int n_items;                  // total work items
  int persistent;               // 1: CTAs take items from the workspace counter
  float scale_log2;
  int out_f32;
  int out_v8;                   // 1: out is 32-byte aligned (the epilogue stores 32 bytes per instruction)
  int out_tma;                  // 1: whole output tiles go out through shared memory and a TMA
                                // store (bf16 output, d = 128; maps.out is encoded)
  void* workspace;              // caller scratch (NULL: no key-range splits)
  int* trace;                   // progress words in host-mapped memory (trace builds only)
};

// Query heads of one kv group that share a prefill CTA (and its K/V tiles).
inline int prefill_heads_per_cta(int n_q_heads, int n_kv_heads) {
  return ((n_q_heads / n_kv_heads) % 2 == 0) ? 2 : 1;
}
// Bytes of the prefill workspace for `hpc` heads per CTA and head_dim `d`.
size_t prefill_workspace_bytes(int hpc, int d);

// TMA descriptors of the prefill, built on the host per call.
struct PrefillMaps {
  CUtensorMap q;        // q [B][T][Hq][d]       box {d_box, 1, 128, 1}
  CUtensorMap k;        // k [B][T][Hkv][d]
  CUtensorMap v;
  CUtensorMap kc;       // k_cache [B*Hkv][W][d] box {d_box, 128, 1}
  CUtensorMap vc;
  CUtensorMap out;      // out [B][T][Hq][d] bf16, box {d_box, 1, 128, 1} (out_tma only)
};

cudaError_t launch_append(const AppendParams& p, cudaStream_t stream);
cudaError_t launch_decode(const DecodeParams& p, cudaStream_t stream);
// How a prefill launch covers its units: whole units, the split tail, the grid.
struct PrefillSchedule {
  long long n_whole;
  int n_pieces;
  long long n_items;
  int persistent;
  long long grid;
};
PrefillSchedule prefill_schedule(long long n_units, int n_wtiles, int n_sms, bool have_workspace);
int device_sm_count(int device);
cudaError_t launch_prefill(const PrefillParams& p, const PrefillMaps& maps, int grid, cudaStream_t stream);
// TMA box width (elements of d per box row) and swizzle span used by the prefill kernel.
void prefill_map_geometry(int head_dim, int* box_elems, int* swizzle_bytes);

// SMs of a B200, for the launch shapes of the 8-bit cache's steps and of the rotary positions.  A constant: the shape
// of a decode step fixes the size of its workspace, which is a function of the dims and not of the current device.
constexpr int kSms = 148;

// The 8-bit rolling cache (swa_q8_cache of swa.h): blocks of kQ8Block slots.
constexpr int kQ8Block = 64;

struct Q8Ring {
  uint8_t* k8;                  // [B][Hkv][W][d]
  uint8_t* v8;
  float* k_scale;               // [B][Hkv][ceil(W / 64)]
  float* v_scale;
  __nv_bfloat16* k_tail;        // [B][Hkv][64][d]
  __nv_bfloat16* v_tail;
  int format;
};

struct Q8AppendParams {
  Q8Ring ring;
  const __nv_bfloat16* k;       // [B][max_tokens][Hkv][d]
  const __nv_bfloat16* v;
  const int32_t* start_pos;     // device [B]
  const int32_t* n_tokens;
  int* status;
  int batch, n_kv_heads, head_dim, window, max_tokens;
};
cudaError_t launch_q8_append(const Q8AppendParams& p, cudaStream_t stream);

struct Q8ExpandParams {
  Q8Ring ring;
  __nv_bfloat16* k_out;         // [B][Hkv][W][d] bf16: what the ring's rows stand for
  __nv_bfloat16* v_out;
  const int32_t* start_pos;
  const int32_t* n_tokens;
  int batch, n_kv_heads, head_dim, window, max_tokens;
};
cudaError_t launch_q8_expand(const Q8ExpandParams& p, cudaStream_t stream);

struct Q8DecodeParams {
  Q8Ring ring;
  void* out;                    // [B][Hq][d] bf16 or f32
  const __nv_bfloat16* q;       // [B][Hq][d]
  const __nv_bfloat16* k_new;   // [B][Hkv][d]
  const __nv_bfloat16* v_new;
  const int32_t* pos;           // device [B]
  float* ws_o;                  // [B][Hq][n_splits][d] partial O (two launches)
  float* ws_ml;                 // [B][Hq][n_splits][4] partial (max, score of the sum, sum, 0)
  int* status;
  const int32_t* n_tokens;      // device [B], or NULL: one token, which is taken in
  int max_tokens, groups;       // rows of a chunk, CTAs that share its columns
  int batch, n_q_heads, n_kv_heads, head_dim, window;
  int n_splits, slots_per_split;
  int* trace;                   // fault switch of checked builds, else NULL
  int variant;                  // of kQ8Variants
  int cluster;                  // 1: the splits of a pair merge in a thread-block cluster
  float scale_log2;             // scale * log2(e)
  int out_f32;
};
// CTAs of the q8 decode kernel: warps, tiles in each warp's ring, CTAs an SM holds.
struct Q8Variant {
  int warps, tiles, per_sm;
};
constexpr Q8Variant kQ8Variants[3] = {{8, 3, 1}, {4, 3, 2}, {4, 2, 3}};
constexpr int kQ8MaxCluster = 8;       // portable cluster size
// Split of the W slots of one (sequence, kv head); a function of the shape.
struct Q8DecodeSplit {
  int n_splits, slots_per_split, variant, cluster;
};
Q8DecodeSplit q8_decode_split(int batch, int n_kv_heads, int window, int head_dim, int groups, bool chunk, bool wide);
// The same with clusters of a size of which the current device holds as many as there are pairs at once.
Q8DecodeSplit q8_fit_clusters(Q8DecodeSplit s, long long units, int window);
// Clusters of `size` CTAs, one an SM, that the current device holds at once (0 if it cannot be told).
int q8_clusters_at_once(int size);
// A chunk of few columns (rows x query heads of a kv head) goes through launch_q8_decode too, with q, k, v
// and out as in the prefill and start positions as pos: the CTAs that share a pair's columns; 0 where the
// ring is written out for the prefill kernel instead.
int q8_chunk_groups(long long rows, int group, long long pairs, int window);
// TMA descriptors of the ring's keys and values: [B * Hkv][W][d] bytes, boxes of
// kQ8Block rows, swizzled by the row's size.
struct Q8DecodeMaps {
  CUtensorMap k, v;
};
cudaError_t launch_q8_decode(const Q8DecodeParams& p, const Q8DecodeMaps& maps, cudaStream_t stream);

struct RopeParams {
  __nv_bfloat16* q_out;         // [B][T][Hq][d]
  __nv_bfloat16* k_out;         // [B][T][Hkv][d] or NULL
  const __nv_bfloat16* q;       // rows q_stride elements apart
  const __nv_bfloat16* k;
  int64_t q_stride, k_stride;
  const float* inv_freq;        // device [rotary_dim / 2]
  const int32_t* start_pos;
  const int32_t* n_tokens;      // or NULL
  int* status;
  int batch, n_q_heads, n_kv_heads, head_dim, max_tokens;
  int rotary_dim, interleaved;
  int q_in_place, k_in_place;   // the elements past rotary_dim need no copy
  float factor, sin_sign;
};
cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream);

// Helpers of the C-ABI layer for entry points defined in other files: set the
// thread-local error message, look up the device status word, and run the
// host-side argument checks of a decode call (everything but the workspace).
int api_fail(int code, const char* fmt, ...);
int api_ok();
int api_status_word(int** out);
// Encodes a descriptor of bytes [n][rows][row_bytes] with boxes of box_rows whole rows.
int api_encode_bytes(CUtensorMap* map, const void* ptr, int row_bytes, int rows, long long n, int box_rows,
                     const char* what);
int api_check_dims(const struct swa_dims* dims);
int* api_trace();   // what swa_debug_set_trace of checked builds was given, else NULL
int api_check_ptrs(const char* names, std::initializer_list<const void*> ptrs);      // 16-byte aligned
int api_check_ptrs4(const char* names, std::initializer_list<const void*> ptrs);     // 4-byte aligned
int api_check_decode(const struct swa_dims* dims, const void* out, const void* q, const void* k_new,
                     const void* v_new, const void* k_cache, const void* v_cache, const int32_t* pos);

}  // namespace swa
