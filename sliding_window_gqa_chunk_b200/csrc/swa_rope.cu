// swa_rope.cu - rotary positions: the first r elements of each head's row are
// pairs, and the pair i of the row at position p is turned by p * inv_freq[i].
//
// Pure streaming: every row is read and written once, so the bound is HBM for
// chunks and the launch for a decode step.  The angles of a token are the same
// for all its heads: the CTA computes the cos and sin of its tokens once into
// shared memory, and each thread keeps those of its 8 pairs in registers
// while it goes through its share of the heads, two at a time: 4096 tokens of
// 40 heads of 128 take 17.4 us (4.8 TB/s; 16384 tokens 56.5, 5.9 TB/s), one
// head at a time with 5 CTAs an SM 18.1, three with 3 CTAs 17.9.  A thread's unit is 16
// elements of a head, two 16-byte pieces that hold whole pairs: [8c, 8c + 8)
// and [r/2 + 8c, ...) with halves, [16c, 16c + 16) interleaved; pair 8c + i is
// the i-th of unit c either way.
//
// The angle is p * f in fp64, brought to a fraction of a turn there, and only
// then rounded to fp32: p * f in fp32 would be off by half a radian at
// positions above 2^23.
#include "swa_common.cuh"
#include "swa_internal.h"

namespace swa {

namespace {
constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;      // tokens of a CTA
constexpr int kHeads = 2;           // heads of a thread whose loads are in flight together
constexpr int kCtasPerSm = 4;       // at 64 registers a thread
constexpr int kMaxPairs = 64;       // rotary_dim <= 128

__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Turns the 8 pairs of a unit.  INTER: the pairs lie side by side in (a, b),
// else pair i is element i of a and of b.
template <bool INTER>
__device__ __forceinline__ void turn(uint4& a, uint4& b, const float (&cs)[8], const float (&sn)[8]) {
  uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
  if constexpr (INTER) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float u = lo(x[i]), v = hi(x[i]);
      x[i] = pack_bf16x2(u * cs[i] - v * sn[i], v * cs[i] + u * sn[i]);
      const float w = lo(y[i]), z = hi(y[i]);
      y[i] = pack_bf16x2(w * cs[4 + i] - z * sn[4 + i], z * cs[4 + i] + w * sn[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float u0 = lo(x[i]), u1 = hi(x[i]), v0 = lo(y[i]), v1 = hi(y[i]);
      x[i] = pack_bf16x2(u0 * cs[2 * i] - v0 * sn[2 * i], u1 * cs[2 * i + 1] - v1 * sn[2 * i + 1]);
      y[i] = pack_bf16x2(v0 * cs[2 * i] + u0 * sn[2 * i], v1 * cs[2 * i + 1] + u1 * sn[2 * i + 1]);
    }
  }
  a = make_uint4(x[0], x[1], x[2], x[3]);
  b = make_uint4(y[0], y[1], y[2], y[3]);
}
}  // namespace

// `tokens` tokens (of all B * T, numbered through) per CTA; units * tokens * lanes threads, and those
// that make it whole warps.
template <bool INTER>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) swa_rope_kernel(const RopeParams p, int tokens, int lanes) {
  __shared__ float2 ang[kMaxTokens][kMaxPairs];
  __shared__ int live[kMaxTokens];
  wait_prior_grid();
  allow_next_grid();
  const int T = p.max_tokens, r2 = p.rotary_dim / 2;
  const uint32_t first = blockIdx.x * tokens;
  const uint32_t n_rows = p.batch * T;                // below 2^31; the last CTA's tokens may pass it
  for (int i = threadIdx.x; i < tokens * r2; i += blockDim.x) {
    const uint32_t tok = first + i / r2;
    const int pair = i % r2;
    bool ok = false;
    if (tok < n_rows) {
      const int b = (int)tok / T, t = (int)tok - b * T;
      const int s = p.start_pos[b], n = p.n_tokens != nullptr ? p.n_tokens[b] : T;
      if (s < 0 || n < 0 || n > T) {
        if (t == 0 && pair == 0) raise_status(p.status, SWA_ERR_DEVICE_ARG);
      } else if (t < n) {
        ok = true;
        const double turns = (double)((long long)s + t) * (double)p.inv_freq[pair] * 0.15915494309189535;
        float sn, cs;
        sincospif(2.f * (float)(turns - rint(turns)), &sn, &cs);
        ang[i / r2][pair] = make_float2(cs * p.factor, sn * p.factor * p.sin_sign);
      }
    }
    if (pair == 0) live[i / r2] = ok;
  }
  __syncthreads();

  // thread -> (unit c of a row, token, first head); the heads go in steps
  const int units = p.head_dim / 16;                  // 1, 4 or 8
  const int c = threadIdx.x % units;
  const int tk = threadIdx.x / units % tokens;
  const int lane = threadIdx.x / (units * tokens);
  const bool turned = c < p.rotary_dim / 16;
  if (lane >= lanes || !live[tk] || (!turned && p.q_in_place && p.k_in_place)) return;
  const int tok = (int)first + tk;                    // a live one: below n_rows
  float cs[8], sn[8];
  if (turned) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 a = ang[tk][8 * c + i];
      cs[i] = a.x;
      sn[i] = a.y;
    }
  }
  // first elements of the unit's two pieces
  const int e0 = (!INTER && turned) ? 8 * c : 16 * c;
  const int e1 = (!INTER && turned) ? p.rotary_dim / 2 + 8 * c : 16 * c + 8;
  // where head h of the token's row is: k's heads are counted on from q's
  const int D = p.head_dim, Hq = p.n_q_heads, heads = Hq + p.n_kv_heads;
  const __nv_bfloat16* q = p.q + tok * p.q_stride;
  const __nv_bfloat16* k = p.k + (tok * p.k_stride - Hq * D);
  __nv_bfloat16* q_out = p.q_out + (size_t)tok * Hq * D;
  __nv_bfloat16* k_out = p.k_out + ((int64_t)tok * p.n_kv_heads - Hq) * D;
  for (int h0 = lane; h0 < heads; h0 += kHeads * lanes) {
    uint4 a[kHeads], b[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const int h = h0 + i * lanes;
      if (h >= heads) break;
      const __nv_bfloat16* src = (h < Hq ? q : k) + h * D;
      a[i] = *reinterpret_cast<const uint4*>(src + e0);
      b[i] = *reinterpret_cast<const uint4*>(src + e1);
    }
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const int h = h0 + i * lanes;
      if (h >= heads) break;
      const bool is_q = h < Hq;
      if (!turned && (is_q ? p.q_in_place : p.k_in_place)) continue;
      __nv_bfloat16* dst = (is_q ? q_out : k_out) + h * D;
      if (turned) turn<INTER>(a[i], b[i], cs, sn);
      *reinterpret_cast<uint4*>(dst + e0) = a[i];
      *reinterpret_cast<uint4*>(dst + e1) = b[i];
    }
  }
}

cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream) {
  // As many tokens to a CTA as leave the last wave of CTAs full, but not so many that a token has less than
  // four threads for each unit (below 16 heads, one for every eight), or than 16 (24 and 32: the same
  // up to 10 % slower): 4096 tokens of 40 heads of 128 take one wave of 586 CTAs of 7; 12000 three of CTAs of 7, the last
  // one nearly full, 42.8 us (two and a half waves of CTAs of 8 42.5, two of CTAs of 11 45.6).
  const int units = p.head_dim / 16, heads = p.n_q_heads + p.n_kv_heads;
  const int share = heads < 16 ? (heads + 7) / 8 : 4, cap = kThreads / (units * share);
  const int most = cap < kMaxTokens ? cap : kMaxTokens;
  const long long rows = (long long)p.batch * p.max_tokens, slots = (long long)kSms * kCtasPerSm;
  const long long waves = (rows + slots * most - 1) / (slots * most);
  const int tokens = (int)((rows + slots * waves - 1) / (slots * waves));
  int lanes = kThreads / (units * tokens);
  if (lanes > heads) lanes = heads;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((rows + tokens - 1) / tokens));
  cfg.blockDim = dim3((unsigned)((units * tokens * lanes + 31) / 32 * 32));
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.interleaved ? cudaLaunchKernelEx(&cfg, swa_rope_kernel<true>, p, tokens, lanes)
                       : cudaLaunchKernelEx(&cfg, swa_rope_kernel<false>, p, tokens, lanes);
}

}  // namespace swa
