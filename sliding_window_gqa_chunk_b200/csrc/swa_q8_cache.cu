// swa_q8_cache.cu - the 8-bit rolling cache: taking a chunk's keys and values
// in, and writing out in bf16 what the ring holds (for the prefill kernel).
//
// Append.  A chunk of n <= W tokens from position s on fills a block of the
// ring up at most once (the block's last slot comes round once in W
// positions), so one CTA per ring block, kv head and sequence decides alone
// whether the chunk completes its block, takes the rows that came before the
// chunk from the tail, finds the largest magnitude and rounds.  The block of
// position s is the only one that reads the tail; its CTA also writes the new
// tail, after that, so no CTA waits for another.
//
// Expand.  One pass that reads a byte and writes two for each element: 8-bit
// number times scale is exact in bf16 (the scales written here are powers of two
// and no 8-bit number has more than 7 significant bits), rows of the block being filled are copied from the tail.
// The slots that hold no position yet are written as zeros up to the end of
// their 128-slot key tile, which the prefill kernel loads whole.
#include "swa_common.cuh"
#include "swa_internal.h"
#include "swa_q8.cuh"

namespace swa {

namespace {
constexpr int kAppendThreads = 256;
constexpr int kExpandThreads = 256;
constexpr int kKeyTile = 128;   // key tile of the prefill kernel
}  // namespace

template <int D, int FMT>
__global__ void __launch_bounds__(kAppendThreads) swa_q8_append_kernel(const Q8AppendParams p) {
  __shared__ uint32_t red[2];
  wait_prior_grid();
  allow_next_grid();
  const int kvh = blockIdx.y, b = blockIdx.z;
  const int W = p.window;
  const int s = p.start_pos[b];
  const int n = p.n_tokens[b];
  if (s < 0 || n < 0 || n > p.max_tokens) {
    if (threadIdx.x == 0) raise_status(p.status, SWA_ERR_DEVICE_ARG);
    return;
  }
  if (n == 0) return;
  const int n_blocks = (W + kQ8Block - 1) / kQ8Block;
  const int s_slot = (int)((uint32_t)s % (uint32_t)W);
  int j = s_slot / kQ8Block + (int)blockIdx.x;   // gridDim.x <= n_blocks
  if (j >= n_blocks) j -= n_blocks;
  const int first = j * kQ8Block;
  const int size = min(kQ8Block, W - first);
  const size_t unit = (size_t)b * p.n_kv_heads + kvh;
  const size_t row_elems = (size_t)p.n_kv_heads * D;
  const __nv_bfloat16* kc = p.k + (size_t)b * p.max_tokens * row_elems + (size_t)kvh * D;
  const __nv_bfloat16* vc = p.v + (size_t)b * p.max_tokens * row_elems + (size_t)kvh * D;
  __nv_bfloat16* kt = p.ring.k_tail + unit * kQ8Block * D;
  __nv_bfloat16* vt = p.ring.v_tail + unit * kQ8Block * D;

  // chunk row that lands on the block's last slot, the next time round
  int t_full = first + size - 1 - s_slot;
  if (t_full < 0) t_full += W;
  if (t_full < n) {
    const int t0 = t_full - (size - 1);          // chunk row of the block's row 0 (< 0: in the tail)
    auto k_row = [&](int i) { return t0 + i >= 0 ? kc + (size_t)(t0 + i) * row_elems : kt + (size_t)i * D; };
    auto v_row = [&](int i) { return t0 + i >= 0 ? vc + (size_t)(t0 + i) * row_elems : vt + (size_t)i * D; };
    const size_t dst = (unit * W + first) * D;
    q8::round_block<D, FMT, kAppendThreads>(k_row, v_row, size, p.ring.k8 + dst, p.ring.v8 + dst,
                            p.ring.k_scale + unit * n_blocks + j, p.ring.v_scale + unit * n_blocks + j, red);
  }
  if (blockIdx.x != 0) return;

  // the block that the last token leaves unfilled: its rows that the chunk brings
  const int e_slot = (int)(((uint32_t)s + (uint32_t)(n - 1)) % (uint32_t)W);   // below 2^32: n <= W <= 2^30
  const int e_row = e_slot % kQ8Block;
  if (e_slot + 1 == W || e_row + 1 == kQ8Block) return;
  __syncthreads();                               // the tail's old rows have been read
  const int rows = min(n, e_row + 1);
  constexpr int kVecs = D / 8;
  for (int i = threadIdx.x; i < rows * kVecs; i += blockDim.x) {
    const int r = e_row - i / kVecs, t = n - 1 - i / kVecs, c = i % kVecs;
    reinterpret_cast<uint4*>(kt + (size_t)r * D)[c] = reinterpret_cast<const uint4*>(kc + (size_t)t * row_elems)[c];
    reinterpret_cast<uint4*>(vt + (size_t)r * D)[c] = reinterpret_cast<const uint4*>(vc + (size_t)t * row_elems)[c];
  }
}

// 16 8-bit numbers times `scale` -> 16 bf16.
template <int FMT>
__device__ __forceinline__ void expand16(const uint4& x, float scale, uint4& a, uint4& b) {
  const uint32_t in[4] = {x.x, x.y, x.z, x.w};
  uint32_t out[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t lo, hi;
    q8::unpack4<FMT>(in[i], lo, hi);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    out[2 * i] = pack_bf16x2(f.x * scale, f.y * scale);
    out[2 * i + 1] = pack_bf16x2(g.x * scale, g.y * scale);
  }
  a = make_uint4(out[0], out[1], out[2], out[3]);
  b = make_uint4(out[4], out[5], out[6], out[7]);
}

template <int D, int FMT>
__global__ void __launch_bounds__(kExpandThreads) swa_q8_expand_kernel(const Q8ExpandParams p) {
  wait_prior_grid();
  allow_next_grid();
  const int j = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
  const int W = p.window;
  const int n_blocks = (W + kQ8Block - 1) / kQ8Block;
  const int first = j * kQ8Block;
  const int size = min(kQ8Block, W - first);
  const size_t unit = (size_t)b * p.n_kv_heads + kvh;
  const size_t base = (unit * W + first) * D;
  // the block's bytes are asked for together with the sequence's position, not after it
  constexpr int kVecs = D / 16;
  constexpr int kPer = (kQ8Block * kVecs + kExpandThreads - 1) / kExpandThreads;
  uint4 k[kPer], v[kPer];
#pragma unroll
  for (int m = 0; m < kPer; ++m) {
    const int i = threadIdx.x + m * kExpandThreads;
    k[m] = v[m] = make_uint4(0, 0, 0, 0);
    if (i < size * kVecs) {
      k[m] = ldg_stream(p.ring.k8 + base + 16 * (size_t)i);
      v[m] = ldg_stream(p.ring.v8 + base + 16 * (size_t)i);
    }
  }
  const float ks = p.ring.k_scale[unit * n_blocks + j], vs = p.ring.v_scale[unit * n_blocks + j];
  const int s = p.start_pos[b];
  const int n = p.n_tokens[b];
  if (s <= 0 || n <= 0 || n > p.max_tokens) return;   // nothing is read from the ring
  const int held = s < W ? s : W;                     // slots [0, held) hold a position
  if (first >= (held + kKeyTile - 1) / kKeyTile * kKeyTile) return;
  const int s_slot = (int)((uint32_t)s % (uint32_t)W);
  const int open = s_slot / kQ8Block == j ? s_slot - first : 0;   // rows that are in the tail
#pragma unroll
  for (int m = 0; m < kPer; ++m) {
    const int i = threadIdx.x + m * kExpandThreads, r = i / kVecs, c = i % kVecs;
    if (i >= size * kVecs) continue;
    uint4 k0 = make_uint4(0, 0, 0, 0), k1 = k0, v0 = k0, v1 = k0;
    if (r < open) {
      const uint4* kt = reinterpret_cast<const uint4*>(p.ring.k_tail + (unit * kQ8Block + r) * D) + 2 * c;
      const uint4* vt = reinterpret_cast<const uint4*>(p.ring.v_tail + (unit * kQ8Block + r) * D) + 2 * c;
      k0 = kt[0];
      k1 = kt[1];
      v0 = vt[0];
      v1 = vt[1];
    } else if (first + r < held) {
      expand16<FMT>(k[m], ks, k0, k1);
      expand16<FMT>(v[m], vs, v0, v1);
    }
    uint4* ko = reinterpret_cast<uint4*>(p.k_out + base) + 2 * (size_t)i;
    uint4* vo = reinterpret_cast<uint4*>(p.v_out + base) + 2 * (size_t)i;
    ko[0] = k0;
    ko[1] = k1;
    vo[0] = v0;
    vo[1] = v1;
  }
}

namespace {

cudaLaunchConfig_t pdl_config(dim3 grid, int threads, cudaStream_t stream, cudaLaunchAttribute* attr) {
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <int D>
cudaError_t launch_append_d(const Q8AppendParams& p, const cudaLaunchConfig_t& cfg) {
  return p.ring.format == SWA_Q8_E4M3 ? cudaLaunchKernelEx(&cfg, swa_q8_append_kernel<D, SWA_Q8_E4M3>, p)
                                      : cudaLaunchKernelEx(&cfg, swa_q8_append_kernel<D, SWA_Q8_INT8>, p);
}

template <int D>
cudaError_t launch_expand_d(const Q8ExpandParams& p, const cudaLaunchConfig_t& cfg) {
  return p.ring.format == SWA_Q8_E4M3 ? cudaLaunchKernelEx(&cfg, swa_q8_expand_kernel<D, SWA_Q8_E4M3>, p)
                                      : cudaLaunchKernelEx(&cfg, swa_q8_expand_kernel<D, SWA_Q8_INT8>, p);
}

}  // namespace

cudaError_t launch_q8_append(const Q8AppendParams& p, cudaStream_t stream) {
  // T tokens reach ceil((T - 1) / 64) + 1 blocks, and one more where they pass
  // the ring's short last block
  const long long n_blocks = ((long long)p.window + kQ8Block - 1) / kQ8Block;
  long long reach = ((long long)p.max_tokens + kQ8Block - 2) / kQ8Block + 2;
  if (reach > n_blocks) reach = n_blocks;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      pdl_config(dim3((unsigned)reach, (unsigned)p.n_kv_heads, (unsigned)p.batch), kAppendThreads, stream, attr);
  switch (p.head_dim) {
    case 16: return launch_append_d<16>(p, cfg);
    case 64: return launch_append_d<64>(p, cfg);
    case 128: return launch_append_d<128>(p, cfg);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_q8_expand(const Q8ExpandParams& p, cudaStream_t stream) {
  const unsigned n_blocks = (unsigned)(((long long)p.window + kQ8Block - 1) / kQ8Block);
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      pdl_config(dim3(n_blocks, (unsigned)p.n_kv_heads, (unsigned)p.batch), kExpandThreads, stream, attr);
  switch (p.head_dim) {
    case 16: return launch_expand_d<16>(p, cfg);
    case 64: return launch_expand_d<64>(p, cfg);
    case 128: return launch_expand_d<128>(p, cfg);
  }
  return cudaErrorInvalidValue;
}

}  // namespace swa
