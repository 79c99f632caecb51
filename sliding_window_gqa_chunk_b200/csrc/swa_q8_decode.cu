// swa_q8_decode.cu - single-token decode over the 8-bit rolling cache.
//
// The step is the bf16 decode's (a query attends over the min(pos + 1, W)
// positions (pos - W, pos]), over half the bytes: every (sequence, kv head)
// streams W slots x d x 1 B of keys and the same of values.  One warp handles
// all G query heads of its kv head, and the dot products run on mma.sync
// m16n8k16 in f16 with fp32 sums, in which every 8-bit number is exact:
//
//   S^T[slot][head] = K[slot][:] . Q[head][:]        (M = 16 slots, N = 8 heads, K = d)
//   O^T[d][head]   += V^T[d][slot] . P^T[slot][head] (M = 16 d, N = 8 heads, K = 16 slots)
//
// tcgen05 has nothing to offer here: at G = 4 the tensor work is a few percent
// of the time that the bytes take, and its operands would have to be written
// back to shared memory in 16 bits.
//
// Scales.  A block's key scale multiplies its scores.  Its value scale 2^v is
// put into the exponent of the softmax: with x the score in log2 units, the
// weight of a slot is w = 2^(x + v - m), where the running m is the maximum of
// x + v rather than of x.  The numbers of a block's values always reach the top
// of their format, so w orders the slots by what they can add to the output
// and is at most 1: rounding w to f16 loses what is below 2^-24 of the largest
// such addition.  The softmax sum is that of 2^(x - m) = w 2^-v, in fp32.
// Q goes to f16 with one power of two for each head (its largest magnitude to
// [2^14, 2^15)): its 8 bits are kept in all elements above 2^-28 of the
// largest.  The rows of the block being filled (at most 64, in bf16) go
// through the same products, 16 rows with a power of two of their own at a time.
//
// Work split: grid (n_splits, Hkv, B); the warps of a CTA take pieces of 16 or
// 32 slots (never across a scale block) in turn, then merge their (m, l, O) in
// shared memory, and the splits of a pair merge through distributed shared
// memory (thread-block cluster) or through the workspace and a second kernel.
// The CTA whose split holds slot pos mod W takes the rows of the tail into its
// sweep, writes the new row there or, if it is its block's last, rounds the
// block into the ring.  That block's old rows are then all out of the window,
// so no CTA reads what is being written.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include "swa_common.cuh"
#include "swa_internal.h"
#include "swa_q8.cuh"
#include "swa_tc.cuh"

namespace swa {

namespace {

constexpr int kSub = 16;            // slots of one mma block
constexpr int kMaxCluster = 8;      // portable cluster size

// Row fragments of a lane: bytes of a key row (D / 4) and of a value row (D / 8).
template <int D>
struct Q8Frag {
  static constexpr int kKWords = D / 16;                    // 4 numbers each = one mma k-step
  static constexpr int kVBytes = D / 8;
  static constexpr int kVWords = kVBytes < 4 ? 1 : kVBytes / 4;
  static constexpr int kMTiles = D / 16;
};

// Tiles in shared memory lie as TMA writes them: rows of D bytes whose 16-byte
// pieces are permuted (128-byte swizzle for d = 128: piece ^ (row & 7), 64-byte
// swizzle for d = 64: piece ^ (row / 2 & 3)), so that the lanes of a load fall on
// different banks.
template <int D>
__device__ __forceinline__ uint32_t piece_at(int row, int piece) {
  if constexpr (D == 128) return row * 128 + ((piece ^ (row & 7)) << 4);
  if constexpr (D == 64) return row * 64 + ((piece ^ (row >> 1 & 3)) << 4);
  return row * 16;
}

// First element of lane-quad t's key word w.  Dot products do not depend on
// the order of d; this one reads whole pieces, and with the swizzle above the
// two rows and four pieces of 8 lanes fall on all 32 banks.
template <int D>
__device__ __forceinline__ int key_elem(int t, int w) {
  if constexpr (D == 16) return 4 * t;
  if constexpr (D == 64) return 16 * t + 4 * w;
  return (2 * t + w / 4) * 16 + (w % 4) * 4;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
  return r;
}

template <int D>
__device__ __forceinline__ void load_key8(uint32_t (&w)[Q8Frag<D>::kKWords], uint32_t tile, int row, int t) {
  if constexpr (D == 16) {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(tile + row * 16 + 4 * t));
  } else {
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      const uint4 x = lds128(tile + piece_at<D>(row, (D / 64) * t + j));
      w[4 * j] = x.x;
      w[4 * j + 1] = x.y;
      w[4 * j + 2] = x.z;
      w[4 * j + 3] = x.w;
    }
  }
}

// Lane-group g's values: elements [g D / 8, (g + 1) D / 8) of a row.
template <int D>
__device__ __forceinline__ void load_val8(uint32_t (&w)[Q8Frag<D>::kVWords], uint32_t tile, int row, int g) {
  if constexpr (D == 16) {
    uint16_t x;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(tile + row * 16 + 2 * g));
    w[0] = x;
  } else if constexpr (D == 64) {
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                 : "=r"(w[0]), "=r"(w[1])
                 : "r"(tile + piece_at<D>(row, g >> 1) + (g & 1) * 8));
  } else {
    const uint4 x = lds128(tile + piece_at<D>(row, g));
    w[0] = x.x;
    w[1] = x.y;
    w[2] = x.z;
    w[3] = x.w;
  }
}

// D += A * B for one 16x8x16 f16 tile, fp32 accumulators (warp-wide).
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two fp32 -> packed f16x2, round to nearest even; `lo` goes to bits 0..15.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// A bf16 pair times a power of two, as an f16 pair.
__device__ __forceinline__ uint32_t bf16_to_f16(uint32_t w, float s) {
  return pack_f16x2(q8::bf16_lo(w) * s, q8::bf16_hi(w) * s);
}
__device__ __forceinline__ uint32_t amax_word(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }
// Exponent that brings a largest magnitude (bf16 bits) to [2^14, 2^15): x 2^-e.
__device__ __forceinline__ int f16_exp(uint32_t amax) {
  if (amax == 0) return 0;
  const int e = (int)(amax >> 7) - 127 - 14;
  return e < -126 ? -126 : (e > 113 ? 113 : e);
}

template <int D>
constexpr int q8_o_stride() { return D + 1; }
template <int D, int NT, int NW>
constexpr int q8_merge_bytes() {
  return (int)sizeof(float) * (NW * 8 * NT * (2 + q8_o_stride<D>()) + 8 * NT * (2 + D));
}
// Shared memory: the warps' rings (the merge reuses them), 2 words, barriers, and
// what it takes to start on a 1024-byte boundary (the swizzle goes by the address).
template <int D, int NT, int NW, int SUB, int R>
constexpr int q8_ring_bytes() {
  constexpr int ring = NW * R * SUB * kSub * D, merge = q8_merge_bytes<D, NT, NW>();
  return ((ring > merge ? ring : merge) + 15) / 16 * 16;
}
template <int D, int NT, int NW, int SUB, int R>
constexpr int q8_smem_bytes() {
  return 1024 + q8_ring_bytes<D, NT, NW, SUB, R>() + 16 + NW * R * 8;
}

__device__ __forceinline__ void store_out(void* out, size_t i, float x, int f32) {
  if (f32) reinterpret_cast<float*>(out)[i] = x;
  else reinterpret_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(x);
}

// Running softmax state of one n-tile (8 heads) of a warp: lane (g, t) holds
// heads 2t and 2t + 1; O rows (mt, g) and (mt, g + 8) are elements
// g D / 8 + 2 mt and the next one.
template <int D>
struct State {
  float m[2], l[2];
  float o[Q8Frag<D>::kMTiles][4];
};

// Scores `x` (log2 units, -inf where masked) of SUB blocks of 16 slots whose
// value scale is 2^v -> weights as B fragments; updates m, l and rescales O.
template <int D, int SUB>
__device__ __forceinline__ void softmax_step(State<D>& st, float (&x)[SUB][4], int v, uint32_t (&pb)[SUB][2]) {
  float mx0 = -CUDART_INF_F, mx1 = -CUDART_INF_F;
#pragma unroll
  for (int u = 0; u < SUB; ++u) {
    mx0 = fmaxf(mx0, fmaxf(x[u][0], x[u][2]));
    mx1 = fmaxf(mx1, fmaxf(x[u][1], x[u][3]));
  }
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
  }
  const float fv = (float)v, inv = q8::exp2_int(-v);
  const float n0 = fmaxf(st.m[0], mx0 + fv), n1 = fmaxf(st.m[1], mx1 + fv);
  const float a0 = fast_exp2(st.m[0] - n0), a1 = fast_exp2(st.m[1] - n1);
  st.m[0] = n0;
  st.m[1] = n1;
  const float c0 = fv - n0, c1 = fv - n1;
  float s0 = 0.f, s1 = 0.f;
#pragma unroll
  for (int u = 0; u < SUB; ++u) {
    const float p0 = fast_exp2(x[u][0] + c0), p1 = fast_exp2(x[u][1] + c1);
    const float p2 = fast_exp2(x[u][2] + c0), p3 = fast_exp2(x[u][3] + c1);
    s0 += p0 + p2;
    s1 += p1 + p3;
    pb[u][0] = movmatrix_trans(pack_f16x2(p0, p1));
    pb[u][1] = movmatrix_trans(pack_f16x2(p2, p3));
  }
  st.l[0] = st.l[0] * a0 + s0 * inv;
  st.l[1] = st.l[1] * a1 + s1 * inv;
  if (__any_sync(0xffffffffu, a0 != 1.f || a1 != 1.f)) {   // a maximum moved
#pragma unroll
    for (int mt = 0; mt < Q8Frag<D>::kMTiles; ++mt) {
      st.o[mt][0] *= a0;
      st.o[mt][1] *= a1;
      st.o[mt][2] *= a0;
      st.o[mt][3] *= a1;
    }
  }
}

}  // namespace

// NT = number of 8-head n-tiles (ceil(G / 8)); NW = warps; SUB = 16-slot
// blocks that a warp takes at a time; R = tiles (keys or values of a piece) in
// a warp's ring.
template <int D, int NT, int NW, int SUB, int R, int FMT>
__global__ void __launch_bounds__(NW * 32)
swa_q8_decode_kernel(const Q8DecodeParams p, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map) {
  using F = Q8Frag<D>;
  constexpr int kPiece = kSub * SUB;
  constexpr int kTile = kPiece * D;
  static_assert(kQ8Block % kPiece == 0, "a piece has one scale");
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem_al = smem_raw + (1024 - (tc::smem_u32(smem_raw) & 1023)) % 1024;
  float* smem = reinterpret_cast<float*>(smem_al);

  const int split = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int G = p.n_q_heads / p.n_kv_heads;
  const int W = p.window;

  // each warp streams its own pieces: tiles K0 V0 K1 V1 ... through a ring of R,
  // one barrier a place, filled by TMA and freed by the warp itself
  const uint32_t ring = tc::smem_u32(smem_al) + warp * R * kTile;
  const uint32_t bars = tc::smem_u32(smem_al) + q8_ring_bytes<D, NT, NW, SUB, R>() + 16 + warp * R * 8;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < R; ++i) tc::mbar_init(bars + 8 * i, 1);
    tc::mbar_fence_init();
    tc::prefetch_map(&k_map);
    tc::prefetch_map(&v_map);
  }
  __syncwarp();

  wait_prior_grid();
  allow_next_grid();
  const long long pos = p.pos[b];
  if (pos < 0) {   // every CTA of the sequence leaves here, whole clusters at a time
    if (threadIdx.x == 0) raise_status(p.status, SWA_ERR_DEVICE_ARG);
    return;
  }
  const int n_valid = (int)(pos + 1 < (long long)W ? pos + 1 : (long long)W);
  const int s_new = (int)(pos % W);
  const int blk0 = s_new / kQ8Block * kQ8Block;      // first slot of the block being filled
  const int row_new = s_new - blk0;
  const int r_begin = split * p.slots_per_split;     // a multiple of 64
  const int r_stop = r_begin + p.slots_per_split;
  const int r_end = r_stop < n_valid ? r_stop : n_valid;
  const bool owner = s_new >= r_begin && s_new < r_stop;

  const size_t unit = (size_t)b * p.n_kv_heads + kvh;
  const int n_blocks = (W + kQ8Block - 1) / kQ8Block;
  const float* ksc = p.ring.k_scale + unit * n_blocks;
  const float* vsc = p.ring.v_scale + unit * n_blocks;
  __nv_bfloat16* kt = p.ring.k_tail + unit * kQ8Block * D;
  __nv_bfloat16* vt = p.ring.v_tail + unit * kQ8Block * D;
  const __nv_bfloat16* kn = p.k_new + unit * D;
  const __nv_bfloat16* vn = p.v_new + unit * D;

  // rows [first_row(x), r_end) of the piece at slot x are held in 8 bits and in the window
  auto first_row = [&](int x) { return (x >= blk0 && x <= s_new) ? s_new + 1 : x; };
  auto next_piece = [&](int x) {
    do x += NW * kPiece;
    while (x < r_end && first_row(x) >= min(x + kPiece, r_end));
    return x;
  };
  // the tile after the last one issued: piece, whether its values, place in the ring
  int is_x = next_piece(r_begin + warp * kPiece - NW * kPiece), is_v = 0, is_at = 0;
  auto issue = [&]() {
    if (is_x >= r_end) return;
    if (lane == 0) {
      tc::mbar_arrive_expect_tx(bars + 8 * is_at, kTile);
      tc::tma_load_3d(ring + is_at * kTile, is_v ? &v_map : &k_map, 0, is_x, (int)unit, bars + 8 * is_at);
    }
    if (is_v) is_x = next_piece(is_x);
    is_v ^= 1;
    is_at = is_at + 1 == R ? 0 : is_at + 1;
  };
  int x0 = is_x;
#pragma unroll
  for (int i = 0; i < R; ++i) issue();
  float ks = 0.f, vs = 1.f;
  if (x0 < r_end) {
    ks = ksc[x0 / kQ8Block];
    vs = vsc[x0 / kQ8Block];
  }

  // Q as the B operand of S^T = K Q^T, f16: lane (g, t) holds head 8 nt + g.
  uint32_t qf[NT][2 * F::kKWords];
  float qs[NT][2];                                   // factor of the scores of heads 2t, 2t + 1
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int hl = nt * 8 + g;
    const bool hv = hl < G;
    const __nv_bfloat16* qrow = p.q + ((size_t)b * p.n_q_heads + (size_t)kvh * G + (hv ? hl : 0)) * D;
    uint32_t m = 0;
#pragma unroll
    for (int w = 0; w < F::kKWords; ++w) {
      const uint2 x = hv ? ldg_stream8(qrow + key_elem<D>(t, w)) : make_uint2(0, 0);
      qf[nt][2 * w] = x.x;
      qf[nt][2 * w + 1] = x.y;
      m = amax_word(amax_word(m, x.x), x.y);
    }
    m = max(m & 0xffffu, m >> 16);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const int e = f16_exp(m);
    const float s = q8::exp2_int(-e);
#pragma unroll
    for (int w = 0; w < 2 * F::kKWords; ++w) qf[nt][w] = bf16_to_f16(qf[nt][w], s);
    const float back = q8::exp2_int(e) * p.scale_log2;
    qs[nt][0] = __shfl_sync(0xffffffffu, back, 8 * t);
    qs[nt][1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
  }

  State<D> st[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    st[nt].m[0] = st[nt].m[1] = -CUDART_INF_F;
    st[nt].l[0] = st[nt].l[1] = 0.f;
#pragma unroll
    for (int mt = 0; mt < F::kMTiles; ++mt) st[nt].o[mt][0] = st[nt].o[mt][1] = st[nt].o[mt][2] = st[nt].o[mt][3] = 0.f;
  }

  if (owner) {
    // rows 0 .. row_new of the block being filled, 16 at a time: rows before
    // row_new from the tail, row_new from k_new / v_new
    for (int y0 = warp * kSub; y0 <= row_new; y0 += NW * kSub) {
      uint32_t kw[2][2 * F::kKWords], vw[4][F::kMTiles];
      uint32_t km = 0, vm = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = y0 + i * 8 + g;
        const __nv_bfloat16* row = r == row_new ? kn : kt + (size_t)r * D;
#pragma unroll
        for (int w = 0; w < F::kKWords; ++w) {
          const uint2 x = r <= row_new ? *reinterpret_cast<const uint2*>(row + key_elem<D>(t, w)) : make_uint2(0, 0);
          kw[i][2 * w] = x.x;
          kw[i][2 * w + 1] = x.y;
          km = amax_word(amax_word(km, x.x), x.y);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = y0 + 2 * t + (i & 1) + (i >> 1) * 8;
        const __nv_bfloat16* row = r == row_new ? vn : vt + (size_t)r * D;
#pragma unroll
        for (int mt = 0; mt < F::kMTiles; ++mt) {
          vw[i][mt] = r <= row_new ? *reinterpret_cast<const uint32_t*>(row + g * (D / 8) + 2 * mt) : 0u;
          vm = amax_word(vm, vw[i][mt]);
        }
      }
      const int ke = f16_exp(__reduce_max_sync(0xffffffffu, max(km & 0xffffu, km >> 16)));
      const int ve = f16_exp(__reduce_max_sync(0xffffffffu, max(vm & 0xffffu, vm >> 16)));
      const float kf = q8::exp2_int(-ke), vf = q8::exp2_int(-ve), ks = q8::exp2_int(ke);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int w = 0; w < 2 * F::kKWords; ++w) kw[i][w] = bf16_to_f16(kw[i][w], kf);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int mt = 0; mt < F::kMTiles; ++mt) vw[i][mt] = bf16_to_f16(vw[i][mt], vf);
      const bool ok0 = y0 + g <= row_new, ok1 = y0 + 8 + g <= row_new;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x[1][4] = {{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int w = 0; w < F::kKWords; ++w)
          mma_f16(x[0], kw[0][2 * w], kw[1][2 * w], kw[0][2 * w + 1], kw[1][2 * w + 1], qf[nt][2 * w],
                  qf[nt][2 * w + 1]);
        // the two powers of two one after the other: their product may leave fp32's range
        x[0][0] = ok0 ? x[0][0] * ks * qs[nt][0] : -CUDART_INF_F;
        x[0][1] = ok0 ? x[0][1] * ks * qs[nt][1] : -CUDART_INF_F;
        x[0][2] = ok1 ? x[0][2] * ks * qs[nt][0] : -CUDART_INF_F;
        x[0][3] = ok1 ? x[0][3] * ks * qs[nt][1] : -CUDART_INF_F;
        uint32_t pb[1][2];
        softmax_step<D, 1>(st[nt], x, ve, pb);
#pragma unroll
        for (int mt = 0; mt < F::kMTiles; ++mt)
          mma_f16(st[nt].o[mt], prmt(vw[0][mt], vw[1][mt], 0x5410), prmt(vw[0][mt], vw[1][mt], 0x7632),
                  prmt(vw[2][mt], vw[3][mt], 0x5410), prmt(vw[2][mt], vw[3][mt], 0x7632), pb[0][0], pb[0][1]);
      }
    }
  }

  bool ok = true;
  int at = 0, phase = 0;                       // place and phase of the next tile to read
  while (x0 < r_end) {
    const int lo = first_row(x0), hi = x0 + kPiece < r_end ? x0 + kPiece : r_end;
    const int x1 = next_piece(x0);
    float ks1 = 0.f, vs1 = 1.f;                // the next piece's scales, a piece ahead
    if (x1 < r_end) {
      ks1 = ksc[x1 / kQ8Block];
      vs1 = vsc[x1 / kQ8Block];
    }
    const int ve = q8::exp_of(vs);

    if (!(ok = __all_sync(0xffffffffu, tc::mbar_wait(bars + 8 * at, phase, p.status)))) break;
    uint32_t tile = ring + at * kTile;
    float x[NT][SUB][4];
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      uint32_t kw[2][F::kKWords];
#pragma unroll
      for (int i = 0; i < 2; ++i) load_key8<D>(kw[i], tile, u * kSub + i * 8 + g, t);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) x[nt][u][0] = x[nt][u][1] = x[nt][u][2] = x[nt][u][3] = 0.f;
#pragma unroll
      for (int w = 0; w < F::kKWords; ++w) {
        uint32_t a0, a1, a2, a3;
        q8::unpack4<FMT>(kw[0][w], a0, a2);
        q8::unpack4<FMT>(kw[1][w], a1, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16(x[nt][u], a0, a1, a2, a3, qf[nt][2 * w], qf[nt][2 * w + 1]);
      }
    }
    __syncwarp();
    issue();                                   // into the place of the keys just read
    if (++at == R) at = 0, phase ^= 1;

    const bool partial = lo > x0 || hi < x0 + kPiece;
    uint32_t pb[NT][SUB][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float f0 = qs[nt][0] * ks, f1 = qs[nt][1] * ks;
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        x[nt][u][0] *= f0;
        x[nt][u][1] *= f1;
        x[nt][u][2] *= f0;
        x[nt][u][3] *= f1;
      }
      if (partial) {
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
          const int r0 = x0 + u * kSub + g, r1 = r0 + 8;
          if (r0 < lo || r0 >= hi) x[nt][u][0] = x[nt][u][1] = -CUDART_INF_F;
          if (r1 < lo || r1 >= hi) x[nt][u][2] = x[nt][u][3] = -CUDART_INF_F;
        }
      }
      softmax_step<D, SUB>(st[nt], x[nt], ve, pb[nt]);
    }

    if (!(ok = __all_sync(0xffffffffu, tc::mbar_wait(bars + 8 * at, phase, p.status)))) break;
    tile = ring + at * kTile;
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      uint32_t vw[4][F::kVWords];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = u * kSub + 2 * t + (i & 1) + (i >> 1) * 8;
        load_val8<D>(vw[i], tile, r, g);
        if (partial && (x0 + r < lo || x0 + r >= hi)) {   // 0 times what the row holds must be 0
#pragma unroll
          for (int w = 0; w < F::kVWords; ++w) vw[i][w] = 0;
        }
      }
#pragma unroll
      for (int mt = 0; mt < F::kMTiles; ++mt) {
        // bytes 2 mt, 2 mt + 1 of rows (2t, 2t + 1) and (2t + 8, 2t + 9), paired by element
        const uint32_t sel = (mt & 1) ? 0x7362 : 0x5140;
        uint32_t a0, a1, a2, a3;
        q8::unpack4<FMT>(prmt(vw[0][mt / 2], vw[1][mt / 2], sel), a0, a1);
        q8::unpack4<FMT>(prmt(vw[2][mt / 2], vw[3][mt / 2], sel), a2, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16(st[nt].o[mt], a0, a1, a2, a3, pb[nt][u][0], pb[nt][u][1]);
      }
    }
    __syncwarp();
    issue();
    if (++at == R) at = 0, phase ^= 1;
    x0 = x1;
    ks = ks1;
    vs = vs1;
  }
  if (!ok) {
    // a wait ran out (raised in the status word): give every copy still in flight its time to land
    for (int i = 0; i < R; ++i) {
      tc::mbar_wait(bars + 8 * at, phase, p.status);
      if (++at == R) at = 0, phase ^= 1;
    }
  }

  // ---- merge the NW warps of the CTA ----
  // smem (the rings, once every warp is done with its own): m[NW][G8], l[NW][G8], O[NW][G8][kOS], then
  // the CTA's m[G8], l[G8], O[G8][D]
  __syncthreads();
  constexpr int G8 = 8 * NT;
  constexpr int kOS = q8_o_stride<D>();
  float* sm_m = smem;
  float* sm_l = sm_m + NW * G8;
  float* sm_o = sm_l + NW * G8;
  float* cta_m = sm_o + (size_t)NW * G8 * kOS;
  float* cta_l = cta_m + G8;
  float* cta_o = cta_l + G8;
  uint32_t* red = reinterpret_cast<uint32_t*>(smem_al + q8_ring_bytes<D, NT, NW, SUB, R>());
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float l0 = st[nt].l[0], l1 = st[nt].l[1];
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, off);
      l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }
    const int h0 = nt * 8 + 2 * t;
    if (g == 0) {
      sm_m[warp * G8 + h0] = st[nt].m[0];
      sm_m[warp * G8 + h0 + 1] = st[nt].m[1];
      sm_l[warp * G8 + h0] = l0;
      sm_l[warp * G8 + h0 + 1] = l1;
    }
    float* oh0 = sm_o + ((size_t)warp * G8 + h0) * kOS + g * (D / 8);
    float* oh1 = oh0 + kOS;
#pragma unroll
    for (int mt = 0; mt < F::kMTiles; ++mt) {
      oh0[2 * mt] = st[nt].o[mt][0];
      oh1[2 * mt] = st[nt].o[mt][1];
      oh0[2 * mt + 1] = st[nt].o[mt][2];
      oh1[2 * mt + 1] = st[nt].o[mt][3];
    }
  }
  __syncthreads();

  const int hq0 = kvh * G;
  for (int idx = threadIdx.x; idx < G * D; idx += NW * 32) {
    const int h = idx / D, dd = idx % D;
    float M = -CUDART_INF_F;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, sm_m[w * G8 + h]);
    float L = 0.f, O = 0.f;
    if (M != -CUDART_INF_F) {
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float sc = fast_exp2(sm_m[w * G8 + h] - M);
        L += sc * sm_l[w * G8 + h];
        O += sc * sm_o[((size_t)w * G8 + h) * kOS + dd];
      }
    }
    const size_t bh = (size_t)b * p.n_q_heads + hq0 + h;
    if (p.n_splits == 1) {
      store_out(p.out, bh * D + dd, O / L, p.out_f32);
    } else if (p.cluster) {
      cta_o[h * D + dd] = O;
      if (dd == 0) {
        cta_m[h] = M;
        cta_l[h] = L;
      }
    } else {
      p.ws_o[(bh * p.n_splits + split) * D + dd] = O;
      if (dd == 0) {
        p.ws_ml[(bh * p.n_splits + split) * 2] = M;
        p.ws_ml[(bh * p.n_splits + split) * 2 + 1] = L;
      }
    }
  }

  if (p.cluster) {
    // each CTA of the pair's cluster merges a share of the G x d outputs
    namespace cg = cooperative_groups;
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    const int R = p.n_splits;
    const int per = (G * D + R - 1) / R, begin = (int)cl.block_rank() * per;
    for (int idx = begin + threadIdx.x; idx < begin + per && idx < G * D; idx += NW * 32) {
      const int h = idx / D;
      float m_r[kMaxCluster], l_r[kMaxCluster], o_r[kMaxCluster];
      float M = -CUDART_INF_F;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        m_r[r] = -CUDART_INF_F;
        l_r[r] = o_r[r] = 0.f;
        if (r < R) {
          m_r[r] = cl.map_shared_rank(cta_m, r)[h];
          l_r[r] = cl.map_shared_rank(cta_l, r)[h];
          o_r[r] = cl.map_shared_rank(cta_o, r)[idx];
        }
      }
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) M = fmaxf(M, m_r[r]);
      float L = 0.f, O = 0.f;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        const float sc = m_r[r] == -CUDART_INF_F ? 0.f : fast_exp2(m_r[r] - M);
        L += sc * l_r[r];
        O += sc * o_r[r];
      }
      store_out(p.out, ((size_t)b * p.n_q_heads + hq0) * D + idx, O / L, p.out_f32);
    }
    cl.sync();  // this CTA's partial stays until every peer has read it
  }

  if (owner) {
    const int size = min(kQ8Block, W - blk0);
    if (row_new + 1 == size) {
      auto k_row = [&](int i) { return i == row_new ? kn : kt + (size_t)i * D; };
      auto v_row = [&](int i) { return i == row_new ? vn : vt + (size_t)i * D; };
      const size_t dst = (unit * W + blk0) * D;
      q8::round_block<D, FMT>(k_row, v_row, size, p.ring.k8 + dst, p.ring.v8 + dst,
                              p.ring.k_scale + unit * n_blocks + blk0 / kQ8Block,
                              p.ring.v_scale + unit * n_blocks + blk0 / kQ8Block, red);
    } else if (warp == 0) {
      for (int i = lane; i < D / 8; i += 32) {
        reinterpret_cast<uint4*>(kt + (size_t)row_new * D)[i] = reinterpret_cast<const uint4*>(kn)[i];
        reinterpret_cast<uint4*>(vt + (size_t)row_new * D)[i] = reinterpret_cast<const uint4*>(vn)[i];
      }
    }
  }
}

// Merge of the per-split partials: grid B * Hq, one thread per element.
template <int D>
__global__ void __launch_bounds__(D < 32 ? 32 : D) swa_q8_decode_combine_kernel(const Q8DecodeParams p) {
  wait_prior_grid();
  allow_next_grid();
  const size_t bh = blockIdx.x;
  const int dd = threadIdx.x;
  if (dd >= D || p.pos[bh / p.n_q_heads] < 0) return;
  const int S = p.n_splits;
  const float* ml = p.ws_ml + bh * S * 2;
  float M = -CUDART_INF_F;
  for (int s = 0; s < S; ++s) M = fmaxf(M, ml[2 * s]);
  float L = 0.f, O = 0.f;
  const float* op = p.ws_o + bh * S * D + dd;
  for (int s = 0; s < S; ++s) {
    const float m = ml[2 * s];
    if (m == -CUDART_INF_F) continue;
    const float sc = fast_exp2(m - M);
    L += sc * ml[2 * s + 1];
    O += sc * op[(size_t)s * D];
  }
  store_out(p.out, bh * D + dd, O / L, p.out_f32);
}

namespace {

constexpr int kMaxDevices = 64;

template <int D, int NT, int NW, int SUB, int R, int FMT>
cudaError_t launch_t(const Q8DecodeParams& p, const Q8DecodeMaps& maps, cudaStream_t stream) {
  constexpr int smem = q8_smem_bytes<D, NT, NW, SUB, R>();
  auto kern = swa_q8_decode_kernel<D, NT, NW, SUB, R, FMT>;
  if (smem > 48 * 1024) {
    // raised once per device (the attribute persists for the process)
    static bool set[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!set[dev]) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      set[dev] = true;
    }
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.n_splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.n_splits, p.n_kv_heads, p.batch);
  cfg.blockDim = dim3(NW * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster ? 2 : 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p, maps.k, maps.v);
  if (e != cudaSuccess || p.n_splits == 1 || p.cluster) return e;
  cudaLaunchConfig_t ccfg = {};
  ccfg.gridDim = dim3((unsigned)((size_t)p.batch * p.n_q_heads));
  ccfg.blockDim = dim3(D < 32 ? 32 : D);
  ccfg.stream = stream;
  ccfg.attrs = attr;
  ccfg.numAttrs = 1;
  return cudaLaunchKernelEx(&ccfg, swa_q8_decode_combine_kernel<D>, p);
}

#ifndef Q8_SUB
#define Q8_SUB 2
#endif
#ifndef Q8_R4
#define Q8_R4 3
#endif
#ifndef Q8_R8
#define Q8_R8 3
#endif
template <int D, int FMT>
cudaError_t launch_f(const Q8DecodeParams& p, const Q8DecodeMaps& maps, cudaStream_t stream) {
  const bool wide = p.n_q_heads / p.n_kv_heads > 8;
  if (p.warps == 8)
    return wide ? launch_t<D, 2, 8, Q8_SUB, Q8_R8, FMT>(p, maps, stream)
                : launch_t<D, 1, 8, Q8_SUB, Q8_R8, FMT>(p, maps, stream);
  return wide ? launch_t<D, 2, 4, Q8_SUB, Q8_R4, FMT>(p, maps, stream)
              : launch_t<D, 1, 4, Q8_SUB, Q8_R4, FMT>(p, maps, stream);
}

template <int D>
cudaError_t launch_d(const Q8DecodeParams& p, const Q8DecodeMaps& maps, cudaStream_t stream) {
  return p.ring.format == SWA_Q8_E4M3 ? launch_f<D, SWA_Q8_E4M3>(p, maps, stream)
                                      : launch_f<D, SWA_Q8_INT8>(p, maps, stream);
}

}  // namespace

Q8DecodeSplit q8_decode_split(int batch, int n_q_heads, int n_kv_heads, int window, int head_dim) {
  (void)n_q_heads;
  (void)head_dim;
  const long long units = (long long)batch * n_kv_heads;
  Q8DecodeSplit s;
  const long long n_blocks = ((long long)window + kQ8Block - 1) / kQ8Block;
  long long splits;
  if (units < 148) {
    splits = 148 / units;
    if (splits > kMaxCluster) splits = kMaxCluster;
    s.warps = 8;
  } else {
    splits = 148 * 4 / units;
    s.warps = 4;
  }
  if (splits < 1) splits = 1;
  if (splits > n_blocks) splits = n_blocks;
  const long long per = (n_blocks + splits - 1) / splits;
  s.slots_per_split = (int)(per * kQ8Block);
  s.n_splits = (int)((n_blocks + per - 1) / per);
  s.cluster = (units < 148 && s.n_splits > 1) ? 1 : 0;
  return s;
}

int q8_decode_box_rows() { return Q8_SUB * kSub; }

cudaError_t launch_q8_decode(const Q8DecodeParams& p, const Q8DecodeMaps& maps, cudaStream_t stream) {
  switch (p.head_dim) {
    case 16: return launch_d<16>(p, maps, stream);
    case 64: return launch_d<64>(p, maps, stream);
    case 128: return launch_d<128>(p, maps, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace swa
