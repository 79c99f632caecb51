// swa_q8_decode.cuh - attention of one token, or of a chunk's few rows, over the 8-bit
// rolling cache.
//
// A decode step attends over the min(pos + 1, W) positions (pos - W, pos], as the
// bf16 one does, over half the bytes: every (sequence, kv head) streams W slots x
// d x 1 B of keys and the same of values.  One warp handles all G query heads of its
// kv head, and the dot products run on mma.sync m16n8k16 in f16 with fp32 sums, in
// which every 8-bit number is exact:
//
//   S^T[slot][head] = K[slot][:] . Q[head][:]        (M = 16 slots, N = 8 heads, K = d)
//   O^T[d][head]   += V^T[d][slot] . P^T[slot][head] (M = 16 d, N = 8 heads, K = 16 slots)
//
// tcgen05 has nothing to offer here: at G = 4 the tensor pipe is busy for a fifth of
// the time that the bytes take, and its operands would have to be written back to
// shared memory in 16 bits.
//
// Scales. A block's key scale multiplies its scores. Its value scale 2^v (v whole for
// scales that the library writes) is put into the exponent of the softmax: with x the
// score in log2 units, the weight of a slot is w = 2^(x + v - m + 15), where the running m
// is the maximum of x + v rather than of x. The numbers of a block's values reach the top
// of their format, so w orders the slots by what they can add to the output and is at most
// 2^15: f16 keeps 11 bits of the weights down to 2^-29 of the largest. The softmax sum is
// that of 2^(x - r), in fp32, against a score r of its own: the first block's largest,
// 2^40 of which may pass before it moves. (m, r and the exponents between them are whole
// multiples of one step, so what rounds m and r cancels up to kMaxTop; larger ones are
// refused: r and m - r kept apart, products as differences from r, gave the same
// outputs for scores of any size, but one sequence 7.2 us and not 7.0, 16 x 4 rows 33.3 and
// 31.5.) It is taken from the weights, w 2^(m - v - 15 - r), but where these have lost it (m above x +
// v by more than 2^55: values of very different sizes), from the scores. A block of zeros
// has a scale of 1 that says nothing of its size: it is told from others of that scale by
// its bytes, and, as zero rows in bf16, takes a scale below all others, which moves no m.
// Q goes to f16 with one power of two for each head (its largest magnitude to [2^14,
// 2^15)): its 8 bits are kept in all elements above 2^-28 of the largest. The rows of the
// block being filled (at most 64, in bf16) and a chunk's own go through the same products,
// 16 rows with a power of two of their own at a time. In a chunk that may be a row that a
// query does not see: where sizes differ by 2^16 the rows go one by one. (16 x 4 rows 31.1
// us for it, 30.6 without; with powers of its own for each row 32.0.)
//
// Bytes.  The bound is HBM: 538 MB for 64 sequences of W = 4096 with 8 kv heads of 128
// take 83 us (6.5 TB/s; a copy reaches 6.56).  Each warp streams its blocks through
// a ring of its own in shared memory, 3 tiles of 64 rows, filled by TMA and freed by the
// warp (a proxy fence of every lane) when the tile is in registers; no warp waits for another before the merge.  8 warps
// an SM keep 192 KB in flight.  Loads into registers with 12 warps an SM took 172 us; rings of
// 12 KB for 16 warps 100 us (the arithmetic of a block is as long as a ring).
//
// Work split: grid (n_splits, Hkv, B); the warps of a CTA take the 64-slot blocks of its split
// in turn and merge their (m, r, l, O) in shared memory, and the splits of a pair merge through
// distributed shared memory (thread-block cluster) or through the workspace and a second
// kernel.  The CTA whose split holds slot pos mod W takes the rows of the tail into its sweep,
// writes the new row there or, if it is its block's last, rounds the block into the ring.  That
// block's old rows are then all out of the window, so no CTA reads what is being written.
#pragma once

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
constexpr int kSubs = kQ8Block / kSub;        // mma blocks of a scale block
constexpr int kMaxCluster = kQ8MaxCluster;
constexpr float kWeightExp = 15.f;  // the largest weight is 2^15
constexpr float kWeightUnit = 1.f / 32768.f;

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

__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a));
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

// Whether rows [lo, hi) of a tile hold nothing but zeros.  (A call, so that the registers it takes are not
// those of the loop it is called from, where blocks of zeros are rare.)
template <int D, int FMT>
__device__ __noinline__ bool all_zero(uint32_t tile, int lo, int hi) {
  uint32_t any = 0;
  for (int i = lo * D + 4 * (int)(threadIdx.x & 31); i < hi * D; i += 4 * 32) {
    const uint32_t x = lds32(tile + i);        // the swizzle moves pieces within a row
    any |= FMT == SWA_Q8_E4M3 ? x & 0x7f7f7f7fu : x;
  }
  return !__any_sync(0xffffffffu, any != 0);
}

// D += A * B for one 16x8x16 f16 tile, fp32 accumulators (warp-wide).
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D = A * B: the first product of a sum.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
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
// Whether magnitudes (bf16 bits) from `least` + 1 (none: ~0) to `most` lie further apart than one power of two serves all of them.
__device__ __forceinline__ bool apart(uint32_t most, uint32_t least) { return (int)(most >> 7) - (int)(least >> 7) > 16; }
// Largest score and value scale (log2) up to which every whole number counts beside it in fp32.
constexpr float kMaxTop = 0x1p24f;
// Exponent of the value scale of zeros: below that of all others by more than scores differ.
constexpr float kZeroExp = -1000.f;

// Exponent that brings a largest magnitude (bf16 bits) to [2^14, 2^15): x 2^-e.
__device__ __forceinline__ int f16_exp(uint32_t amax) {
  if (amax == 0) return 0;
  const int e = (int)(amax >> 7) - 127 - 14;
  return e < -126 ? -126 : (e > 113 ? 113 : e);
}

// Shared memory of the merge: (m, r, l) and O of each warp (in the rings, once every warp is
// done with its own), and what the CTAs of a cluster send to one another.
template <int D, int NT, int NW>
constexpr int q8_merge_bytes() {
  return (int)sizeof(float) * NW * 8 * NT * (4 + D);
}
template <int D, int NT>
constexpr int q8_peer_floats() { return kMaxCluster * 8 * NT * 4 + 8 * NT * D + 4 * kMaxCluster; }
template <int D, int NT, int NW, int R>
constexpr int q8_ring_bytes() {
  constexpr int ring = NW * R * kQ8Block * D, merge = q8_merge_bytes<D, NT, NW>();
  return ((ring > merge ? ring : merge) + 15) / 16 * 16;
}
// All of it: rings, 2 words, barriers, with clusters the peers' part, and what it takes to start on
// a 1024-byte boundary (the swizzle goes by the address).
template <int D, int NT, int NW, int R>
constexpr int q8_smem_bytes(bool clusters) {
  return 1024 + q8_ring_bytes<D, NT, NW, R>() + 16 + NW * R * 8 + (clusters ? 4 * q8_peer_floats<D, NT>() : 0);
}

// A CTA's shared memory may be written by its peers once it has begun: no memory is ordered by this.
__device__ __forceinline__ void cluster_begun_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;"); }
__device__ __forceinline__ void cluster_begun_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

// The address in CTA `rank` of the cluster of what is at `a` here.
__device__ __forceinline__ uint32_t at_rank(uint32_t a, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
// Stores to a peer that count their bytes on its barrier when they have landed.  (Measured against plain stores and a
// cluster barrier: 8 pairs of 64 blocks 0.15 us faster, 2 pairs of 16 query heads 0.8, 74 pairs of two CTAs 0.2 slower.)
__device__ __forceinline__ void send(uint32_t to, const float4& x, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
               "f"(x.x), "f"(x.y), "f"(x.z), "f"(x.w), "r"(bar)
               : "memory");
}

// Four elements of an output: o against m, the largest score and value scale, l against the score r.
// A part is (m, r, l) and its o; one without rows is (-inf, -inf, 0).
struct Four {
  float m, r, l;
  float4 o;
  __device__ __forceinline__ Four() : m(-INFINITY), r(-INFINITY), l(0.f), o(make_float4(0.f, 0.f, 0.f, 0.f)) {}
  __device__ __forceinline__ void against(const float4& part) {
    m = fmaxf(m, part.x);
    r = fmaxf(r, part.y);
  }
  __device__ __forceinline__ void add(const float4& part, const float4& o2) {
    const float s = fast_exp2(part.x - m);
    l += fast_exp2(part.y - r) * part.z;
    o.x += s * o2.x;
    o.y += s * o2.y;
    o.z += s * o2.z;
    o.w += s * o2.w;
  }
  // the i-th four of the output; weights are in units of kWeightUnit, their sum is not.  2^(m - r) in two
  // halves: it may leave fp32's range where the output does not.
  __device__ __forceinline__ void store(void* out, size_t i, int f32) const {
    const float h = fast_exp2(0.5f * (m - r));
    const float x = o.x * kWeightUnit / l * h * h, y = o.y * kWeightUnit / l * h * h;
    const float z = o.z * kWeightUnit / l * h * h, w = o.w * kWeightUnit / l * h * h;
    if (f32) reinterpret_cast<float4*>(out)[i] = make_float4(x, y, z, w);
    else reinterpret_cast<uint2*>(out)[i] = make_uint2(pack_bf16x2(x, y), pack_bf16x2(z, w));
  }
};

// Running softmax state of one n-tile (8 heads) of a warp: lane (g, t) holds
// heads 2t and 2t + 1; O rows (mt, g) and (mt, g + 8) are elements
// g D / 8 + 2 mt and the next one.
template <int D>
struct State {
  float m[2], r[2], l[2];
  float o[Q8Frag<D>::kMTiles][4];
};

// log2 of a block's value scale, exact for the powers of two that the library writes itself.
__device__ __forceinline__ float log2_of(float s) {
  const uint32_t bits = __float_as_uint(s);
  return (float)((int)(bits >> 23) - 127) + __log2f(__uint_as_float((bits & 0x7fffffu) | 0x3f800000u));
}

// Factor of the scores from those of the head and of the keys, both > 0.  Kept
// where a masked -inf stays -inf and a dot product of 0 stays 0.
__device__ __forceinline__ float score_factor(float q, float k) { return fminf(fmaxf(q * k, 1e-37f), 1e37f); }

// Where the sum's terms leave the range in which they are taken from the weights: log2 of the largest
// against the sum's r, and of the factor from a weight to its term.
constexpr float kFar = 40.f;

// Dot products `x` (-inf where masked) of SUB blocks of 16 slots, to be multiplied
// by f0, f1 (> 0, finite; heads 2t, 2t + 1) for scores in log2 units, with the value
// scale 2^v -> weights as B fragments; updates m, r, l and rescales O.
// GUARD: a column may have no unmasked row (else every one has).
template <int D, int SUB, bool GUARD>
__device__ __forceinline__ void softmax_step(State<D>& st, const float (&x)[SUB][4], float f0, float f1, float v,
                                             uint32_t (&pb)[SUB][2]) {
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
  // where nothing has been seen yet, exponents are taken against 0: all of them are of -inf
  auto base = [](float n) { return GUARD && n == -CUDART_INF_F ? 0.f : n; };
  const float y0 = mx0 * f0, y1 = mx1 * f1;
  const float n0 = fmaxf(st.m[0], fmaf(mx0, f0, v)), n1 = fmaxf(st.m[1], fmaf(mx1, f1, v));
  const float a0 = fast_exp2(st.m[0] - base(n0)), a1 = fast_exp2(st.m[1] - base(n1));
  st.m[0] = n0;
  st.m[1] = n1;
  const float c0 = v + kWeightExp - base(n0), c1 = v + kWeightExp - base(n1);
  if (st.r[0] == -CUDART_INF_F) st.r[0] = y0;
  if (st.r[1] == -CUDART_INF_F) st.r[1] = y1;
  // from a weight to its term of the sum
  float e0 = -c0 - base(st.r[0]), e1 = -c1 - base(st.r[1]);
  const bool far = fmaxf(fmaxf(y0 - st.r[0], e0), fmaxf(y1 - st.r[1], e1)) > kFar;
  if (__any_sync(0xffffffffu, a0 != 1.f || a1 != 1.f || far)) {   // a maximum moved
#pragma unroll
    for (int mt = 0; mt < Q8Frag<D>::kMTiles; ++mt) {
      st.o[mt][0] *= a0;
      st.o[mt][1] *= a1;
      st.o[mt][2] *= a0;
      st.o[mt][3] *= a1;
    }
    if (__any_sync(0xffffffffu, far)) {
      const float r0 = fmaxf(st.r[0], y0), r1 = fmaxf(st.r[1], y1);
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        s0 += fast_exp2(fmaf(x[u][0], f0, -base(r0))) + fast_exp2(fmaf(x[u][2], f0, -base(r0)));
        s1 += fast_exp2(fmaf(x[u][1], f1, -base(r1))) + fast_exp2(fmaf(x[u][3], f1, -base(r1)));
      }
      st.l[0] = st.l[0] * fast_exp2(st.r[0] - base(r0)) + s0;
      st.l[1] = st.l[1] * fast_exp2(st.r[1] - base(r1)) + s1;
      st.r[0] = r0;
      st.r[1] = r1;
      e0 = e1 = -CUDART_INF_F;
    }
  }
  float s0 = 0.f, s1 = 0.f;
#pragma unroll
  for (int u = 0; u < SUB; ++u) {
    const float p0 = fast_exp2(fmaf(x[u][0], f0, c0)), p1 = fast_exp2(fmaf(x[u][1], f1, c1));
    const float p2 = fast_exp2(fmaf(x[u][2], f0, c0)), p3 = fast_exp2(fmaf(x[u][3], f1, c1));
    s0 += p0 + p2;
    s1 += p1 + p3;
    pb[u][0] = movmatrix_trans(pack_f16x2(p0, p1));
    pb[u][1] = movmatrix_trans(pack_f16x2(p2, p3));
  }
  st.l[0] += s0 * fast_exp2(e0);
  st.l[1] += s1 * fast_exp2(e1);
}

}  // namespace

// CTAs that an SM holds by their registers.  The CTA that has an SM to itself at d = 128 is not alone at d = 64 if it takes
// 128 registers a thread and not 133: 512 pairs of 64 blocks 47.6 us for 56, 800 pairs 70 for 83 (74 pairs in clusters of
// two 6.1 for 5.9).
template <int D, int NT, int NW, bool CHUNK>
constexpr int q8_ctas(int per) { return D == 64 && NT == 1 && NW == 8 && !CHUNK ? 2 : per; }

// NT = number of 8-column n-tiles; NW = warps; R = tiles (a block's keys or
// values) in a warp's ring; PER = CTAs an SM.
//
// CHUNK: attention of the first rows of a chunk instead of one token that is taken in.  The
// columns of the products are then (row of the chunk, query head) pairs, up to 8 NT of them to
// a CTA; a row at position start + t does not see the ring's slots that it has outlived (those
// 1 .. t places after slot start mod W), and besides the tail's rows it sees the chunk's own up
// to itself.  The cache stays as it is.
template <int D, int NT, int NW, int R, int PER, int FMT, bool CHUNK>
__global__ void __launch_bounds__(NW * 32, q8_ctas<D, NT, NW, CHUNK>(PER))
swa_q8_decode_kernel(const Q8DecodeParams p, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map) {
  using F = Q8Frag<D>;
  constexpr int kTile = kQ8Block * D;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem_al = smem_raw + (1024 - (tc::smem_u32(smem_raw) & 1023)) % 1024;

  const int split = blockIdx.x, b = blockIdx.z;
  const int kvh = CHUNK ? (int)blockIdx.y / p.groups : (int)blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int G = p.n_q_heads / p.n_kv_heads;
  const int W = p.window;

  // each warp streams its own blocks, keys and values of one after those of the other, through a
  // ring of R tiles, one barrier a place, filled by TMA and freed by the warp itself
  const uint32_t ring = tc::smem_u32(smem_al) + warp * R * kTile;
  const uint32_t bars = tc::smem_u32(smem_al) + q8_ring_bytes<D, NT, NW, R>() + 16 + warp * R * 8;
  const uint32_t peers_bar = tc::smem_u32(smem_al) + q8_ring_bytes<D, NT, NW, R>() + 8;   // all that peers send is here
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < R; ++i) tc::mbar_init(bars + 8 * i, 1);
    if (warp == 0) tc::mbar_init(peers_bar, 1);
    tc::mbar_fence_init();
    tc::prefetch_map(&k_map);
    tc::prefetch_map(&v_map);
  }
  __syncwarp();

  wait_prior_grid();
  allow_next_grid();
  asm volatile("fence.proxy.async.global;" ::: "memory");   // earlier kernels' rows, for the copies below
  const size_t unit = (size_t)b * p.n_kv_heads + kvh;
  // the CTA's columns: c0 .. c0 + cols - 1 of the pair's, and where column c's q and output rows are
  const int c0 = CHUNK ? (int)(blockIdx.y % p.groups) * 8 * NT : 0;
  const int cols = CHUNK ? min(8 * NT, p.max_tokens * G - c0) : G;
  auto row_of = [&](int c) -> size_t {
    if constexpr (!CHUNK) return unit * G + c;
    const int tok = (c0 + c) / G;
    return ((size_t)b * p.max_tokens + tok) * p.n_q_heads + (size_t)kvh * G + (c0 + c - tok * G);
  };
  // Q is asked for before the ring's tiles, which would keep it waiting for as long as it takes to
  // fill every ring (about 4 us).  Lane (g, t) holds column 8 nt + g.
  uint32_t qf[NT][2 * F::kKWords];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int c = nt * 8 + g;
    const __nv_bfloat16* qrow = p.q + row_of(c < cols ? c : 0) * D;
#pragma unroll
    for (int w = 0; w < F::kKWords; ++w) {
      const uint2 x = c < cols ? ldg_stream8(qrow + key_elem<D>(t, w)) : make_uint2(0, 0);
      qf[nt][2 * w] = x.x;
      qf[nt][2 * w + 1] = x.y;
    }
  }
  uint4 fresh = make_uint4(0, 0, 0, 0);              // the new row, for the tail
  if (!CHUNK && warp == NW - 1 && lane < 2 * (D / 8))
    fresh = ldg_stream(reinterpret_cast<const uint4*>((lane < D / 8 ? p.k_new : p.v_new) + unit * D) + lane % (D / 8));
  const int pos = p.pos[b];
  const int n_rows = CHUNK ? p.n_tokens[b] : 1;
  if (pos < 0 || n_rows < 0 || (CHUNK && n_rows > p.max_tokens)) {
    // every CTA of the sequence leaves here, whole clusters at a time
    if (threadIdx.x == 0) raise_status(p.status, SWA_ERR_DEVICE_ARG);
    return;
  }
  if (CHUNK && n_rows * G <= c0) return;             // no column of this CTA has a row
  cluster_begun_arrive();                            // waited for before the first store to a peer
  // a cluster's CTAs merge `per` fours of the output each: theirs from every CTA, and every column's (m, r, l)
  int n_cl = 1, rank = 0, per = 0;
  if (p.cluster) {
    n_cl = p.n_splits;
    rank = split;
    per = (cols * (D / 4) + n_cl - 1) / n_cl;
    if (threadIdx.x == 0)
      tc::mbar_arrive_expect_tx(peers_bar, n_cl * 16 * (max(min(per, cols * (D / 4) - rank * per), 0) + cols));
  }
  const int n_valid = pos < W ? pos + 1 : W;
  const int s_new = (int)((uint32_t)pos % (uint32_t)W);   // in 32 bits: a 64-bit remainder is a long subroutine
  const int blk0 = s_new / kQ8Block * kQ8Block;      // first slot of the block being filled
  const int row_new = s_new - blk0;
  const int r_begin = split * p.slots_per_split;     // a multiple of 64
  const int r_stop = r_begin + p.slots_per_split;
  const int r_end = r_stop < n_valid ? r_stop : n_valid;
  const bool owner = s_new >= r_begin && s_new < r_stop;

  const int n_blocks = (W + kQ8Block - 1) / kQ8Block;
  const float* ksc = p.ring.k_scale + unit * n_blocks;
  const float* vsc = p.ring.v_scale + unit * n_blocks;
  __nv_bfloat16* kt = p.ring.k_tail + unit * kQ8Block * D;
  __nv_bfloat16* vt = p.ring.v_tail + unit * kQ8Block * D;
  // the new row, or the chunk's rows, new_stride elements apart
  const __nv_bfloat16* kn = p.k_new + (CHUNK ? ((size_t)b * p.max_tokens * p.n_kv_heads + kvh) : unit) * D;
  const __nv_bfloat16* vn = p.v_new + (CHUNK ? ((size_t)b * p.max_tokens * p.n_kv_heads + kvh) : unit) * D;
  const size_t new_stride = (size_t)p.n_kv_heads * D;

  // The new row goes in: into the tail now (no one reads that row there), or, if it fills its block up,
  // with the tail into the ring when this CTA, the only one to read the tail, is done.
  const bool fills = !CHUNK && owner && s_new + 1 == min(blk0 + kQ8Block, W);
  if (!CHUNK && owner && !fills && warp == NW - 1 && lane < 2 * (D / 8)) {
    const int i = lane % (D / 8);
    reinterpret_cast<uint4*>((lane < D / 8 ? kt : vt) + (size_t)row_new * D)[i] = fresh;
  }

  // The warp's blocks: those of its split in turn.  Rows [first_row(x), r_end) of the block at
  // slot x are held in 8 bits and in the window; the block being filled may have none.
  auto first_row = [&](int x) { return x == blk0 ? s_new + 1 : x; };
  const int skip = s_new + 1 >= min(blk0 + kQ8Block, n_valid) ? blk0 : -1;
  auto next_block = [&](int x) {
    x += NW * kQ8Block;
    return x == skip ? x + NW * kQ8Block : x;
  };
  // Rows in bf16, 16 at a time to the warps of one CTA of the pair: those of the block being filled
  // (the tail's and, if one token is taken in, the new row), then those of the chunk up to the last that
  // the CTA's columns belong to.  They come first in the ring, keys and values in one place (16 rows of
  // bf16 are half as large as a block of bytes).
  const int old_rows = CHUNK ? row_new : row_new + 1;
  const int old_subs = (old_rows + kSub - 1) / kSub;
  const int seen_rows = CHUNK ? min(n_rows, (c0 + cols - 1) / G + 1) : 0;
  const int subs = owner ? old_subs + (seen_rows + kSub - 1) / kSub : 0;
  // the tile after the last one issued: its block, keys or values, its place in the ring
  int is_x = next_block(r_begin + (warp - NW) * kQ8Block), is_at = 0;
  bool is_v = false;
  int x0 = is_x;
  auto issue = [&]() {
    if (is_x >= r_end) return;
#ifdef SWA_TEST_FAULTS
    // checked build: warp 0's first tile of keys (2: in the first split alone) is never asked for, so its wait runs out
    const bool withheld = p.trace != nullptr && *p.trace != 0 && (*p.trace != 2 || split == 0) && warp == 0 && is_at == 0 &&
                          x0 == is_x && !is_v;
#else
    constexpr bool withheld = false;
#endif
    if (lane == 0 && !withheld) {
      tc::mbar_arrive_expect_tx(bars + 8 * is_at, kTile);
      tc::tma_load_3d(ring + is_at * kTile, is_v ? &v_map : &k_map, 0, is_x, (int)unit, bars + 8 * is_at);
    }
    is_at = is_at + 1 == R ? 0 : is_at + 1;
    if (is_v) is_x = next_block(is_x);
    is_v = !is_v;
  };
  int is_e = warp;                                                   // the next 16 rows to issue
  auto issue_rows = [&]() {
    const bool old = !CHUNK || is_e < old_subs;
    const int first = (old ? is_e : is_e - old_subs) * kSub;         // row of the tail or of the chunk
    const int rows = min(kSub, (old ? old_rows : seen_rows) - first);
    const uint32_t row_bytes = 2 * D, bar = bars + 8 * is_at;
    if (lane == 0) tc::mbar_arrive_expect_tx(bar, 2 * rows * row_bytes);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t dst = ring + is_at * kTile + i * (kTile / 2);
      if (old) {
        const int held = CHUNK ? rows : min(rows, row_new - first);  // of them in the tail
        if (lane == 0 && held > 0)
          tc::bulk_load(dst, (i == 0 ? kt : vt) + (size_t)first * D, held * row_bytes, bar);
        if (lane == 0 && held < rows) tc::bulk_load(dst + held * row_bytes, i == 0 ? kn : vn, row_bytes, bar);
      } else if (lane < rows) {
        tc::bulk_load(dst + lane * row_bytes, (i == 0 ? kn : vn) + (first + lane) * new_stride, row_bytes, bar);
      }
    }
    is_at = is_at + 1 == R ? 0 : is_at + 1;
    is_e += NW;
  };
  {
    int used = 0;
    for (; is_e < subs && used < R; ++used) issue_rows();
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (i >= used) issue();
  }
  float ks = 0.f, vs = 1.f;
  if (x0 < r_end) {
    ks = ksc[x0 / kQ8Block];
    vs = vsc[x0 / kQ8Block];
  }

  // Q as the B operand of S^T = K Q^T, f16
  float qs[NT][2];                                   // factor of the scores of columns 2t, 2t + 1
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    uint32_t m = 0;
#pragma unroll
    for (int w = 0; w < 2 * F::kKWords; ++w) m = amax_word(m, qf[nt][w]);
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

  int tok[NT][2];                                    // rows of the chunk that columns 2t, 2t + 1 belong to
  if constexpr (CHUNK) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      tok[nt][0] = (c0 + nt * 8 + 2 * t) / G;
      tok[nt][1] = (c0 + nt * 8 + 2 * t + 1) / G;
    }
  }

  State<D> st[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    st[nt].m[0] = st[nt].m[1] = st[nt].r[0] = st[nt].r[1] = -CUDART_INF_F;
    st[nt].l[0] = st[nt].l[1] = 0.f;
#pragma unroll
    for (int mt = 0; mt < F::kMTiles; ++mt) st[nt].o[mt][0] = st[nt].o[mt][1] = st[nt].o[mt][2] = st[nt].o[mt][3] = 0.f;
  }

  bool ok = true;
  int at = 0, phase = 0;                       // place and phase of the next tile to read
  // waits for the next tile (its address); once a wait has run out there is nothing more to wait for
  auto take = [&]() -> uint32_t {
    if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(bars + 8 * at, phase, p.status));
    return ring + at * kTile;
  };
  // Every lane has read the tile: the next one goes into its place.  The lanes' loads and the copy's writes are
  // of different proxies, which the warp's barrier alone does not order: without the fence of every lane copies
  // overtook loads (batch 100, W = 4096: other outputs in nearly every call).  It costs nothing at batch 64, and
  // 16 x 4 rows 30.0 us for 29.4.
  auto freed = [&]() {
    tc::fence_proxy_async_smem();
    __syncwarp();
  };
  auto done = [&]() {
    freed();
    if (ok) issue();
    if (++at == R) at = 0, phase ^= 1;
  };
  auto done_rows = [&]() {
    freed();
    if (CHUNK && is_e < subs) issue_rows();
    else issue();
    if (++at == R) at = 0, phase ^= 1;
  };
  for (int e = warp; e < subs && ok; e += NW) {
    const bool old = !CHUNK || e < old_subs;
    const int first = (old ? e : e - old_subs) * kSub;
    const int rows = min(kSub, (old ? old_rows : seen_rows) - first);
    const uint32_t tile = take();
    if (!ok) break;
    int from = 0, to = rows;                   // the rows of this pass
    while (true) {
      uint32_t tk[2][2 * F::kKWords], tv[4][F::kMTiles];
      // the largest of a lane's share of the pass, and of its shares of single rows (those with a number) the smallest, less 1
      uint32_t km = 0, vm = 0, kleast = ~0u, vleast = ~0u;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = i * 8 + g;
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < F::kKWords; ++w) {
          uint2 x = lds64(tile + r * (2 * D) + 2 * key_elem<D>(t, w));
          if (r < from || r >= to) x = make_uint2(0, 0);
          tk[i][2 * w] = x.x;
          tk[i][2 * w + 1] = x.y;
          m = amax_word(amax_word(m, x.x), x.y);
        }
        m = max(m & 0xffffu, m >> 16);
        km = max(km, m);
        kleast = min(kleast, m - 1);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 2 * t + (i & 1) + (i >> 1) * 8;
        uint32_t m = 0;
#pragma unroll
        for (int mt = 0; mt < F::kMTiles; ++mt) {
          const uint32_t x = lds32(tile + kTile / 2 + r * (2 * D) + 2 * (g * (D / 8) + 2 * mt));
          tv[i][mt] = r < from || r >= to ? 0u : x;
          m = amax_word(m, tv[i][mt]);
        }
        m = max(m & 0xffffu, m >> 16);
        vm = max(vm, m);
        vleast = min(vleast, m - 1);
      }
      km = __reduce_max_sync(0xffffffffu, km);
      vm = __reduce_max_sync(0xffffffffu, vm);
      if (CHUNK && to - from == rows && rows > 1 && __any_sync(0xffffffffu, apart(km, kleast) || apart(vm, vleast))) {
        to = 1;
        continue;
      }
      if (to == rows) done_rows();             // the last pass
      const int ke = f16_exp(km), ve = f16_exp(vm);
      const float vsize = vm == 0 ? kZeroExp : (float)ve;
      const float kf = q8::exp2_int(-ke), vf = q8::exp2_int(-ve), ks16 = q8::exp2_int(ke);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int w = 0; w < 2 * F::kKWords; ++w) tk[i][w] = bf16_to_f16(tk[i][w], kf);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int mt = 0; mt < F::kMTiles; ++mt) tv[i][mt] = bf16_to_f16(tv[i][mt], vf);
      const bool ok0 = g >= from && g < to, ok1 = 8 + g >= from && 8 + g < to;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x[1][4] = {{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int w = 0; w < F::kKWords; ++w)
          mma_f16(x[0], tk[0][2 * w], tk[1][2 * w], tk[0][2 * w + 1], tk[1][2 * w + 1], qf[nt][2 * w],
                  qf[nt][2 * w + 1]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          bool see0 = ok0, see1 = ok1;
          if constexpr (CHUNK) {
            // a row of the tail, row_new - r places before the chunk, until W tokens have come after it;
            // a row of the chunk from itself on
            const int tc_ = tok[nt][c], r0 = first + g, r1 = r0 + 8;
            see0 = see0 && (old ? tc_ < W - (row_new - r0) : tc_ >= r0);
            see1 = see1 && (old ? tc_ < W - (row_new - r1) : tc_ >= r1);
          }
          if (!see0) x[0][c] = -CUDART_INF_F;
          if (!see1) x[0][2 + c] = -CUDART_INF_F;
        }
        uint32_t pb[1][2];
        softmax_step<D, 1, CHUNK>(st[nt], x, score_factor(qs[nt][0], ks16), score_factor(qs[nt][1], ks16), vsize, pb);
#pragma unroll
        for (int mt = 0; mt < F::kMTiles; ++mt)
          mma_f16(st[nt].o[mt], prmt(tv[0][mt], tv[1][mt], 0x5410), prmt(tv[0][mt], tv[1][mt], 0x7632),
                  prmt(tv[2][mt], tv[3][mt], 0x5410), prmt(tv[2][mt], tv[3][mt], 0x7632), pb[0][0], pb[0][1]);
      }
      if (to == rows) break;
      from = to++;
    }
  }

  while (ok && x0 < r_end) {
    const int lo = first_row(x0), hi = x0 + kQ8Block < r_end ? x0 + kQ8Block : r_end;
    const bool partial = lo > x0 || hi < x0 + kQ8Block;
    const int x1 = next_block(x0);
    float ks1 = 0.f, vs1 = 1.f;                // the next block's scales, a block ahead
    if (x1 < r_end) {
      ks1 = ksc[x1 / kQ8Block];
      vs1 = vsc[x1 / kQ8Block];
    }

    float x[NT][kSubs][4];
    uint32_t tile = take();
    if (!ok) break;
#pragma unroll
    for (int u = 0; u < kSubs; u += 2) {
      // two mma blocks (and the n-tiles) at a time, whose sums are independent chains
      uint32_t kw[2][2][F::kKWords];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) load_key8<D>(kw[s][i], tile, (u + s) * kSub + i * 8 + g, t);
      if (u + 2 == kSubs) done();              // the tile is in registers: its place is free before the arithmetic
#pragma unroll
      for (int w = 0; w < F::kKWords; ++w) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          uint32_t a0, a1, a2, a3;
          q8::unpack4<FMT>(kw[s][0][w], a0, a2);
          q8::unpack4<FMT>(kw[s][1][w], a1, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (w == 0) mma_f16_first(x[nt][u + s], a0, a1, a2, a3, qf[nt][0], qf[nt][1]);
            else mma_f16(x[nt][u + s], a0, a1, a2, a3, qf[nt][2 * w], qf[nt][2 * w + 1]);
          }
        }
      }
    }

    tile = take();
    if (!ok) break;
    float vsize = log2_of(vs);
    // a block of zeros, or one that needs no scale: its bytes tell
    if (vs == 1.f && all_zero<D, FMT>(tile, lo - x0, hi - x0)) vsize = kZeroExp;
    uint32_t pb[NT][kSubs][2];
    if constexpr (CHUNK) {
      // the slot a places after s_new (round the ring) holds position start - W + a: seen by rows below a
      const int a0 = x0 > s_new ? x0 - s_new : x0 - s_new + W;
      if (partial || a0 < n_rows || (x0 <= s_new && s_new < x0 + kQ8Block)) {
#pragma unroll
        for (int u = 0; u < kSubs; ++u) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int slot = x0 + u * kSub + i * 8 + g, a = slot > s_new ? slot - s_new : slot - s_new + W;
            const bool held = slot >= lo && slot < hi;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (!held || tok[nt][0] >= a) x[nt][u][2 * i] = -CUDART_INF_F;
              if (!held || tok[nt][1] >= a) x[nt][u][2 * i + 1] = -CUDART_INF_F;
            }
          }
        }
      }
    } else if (partial) {
#pragma unroll
      for (int u = 0; u < kSubs; ++u) {
        const int r0 = x0 + u * kSub + g, r1 = r0 + 8;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (r0 < lo || r0 >= hi) x[nt][u][0] = x[nt][u][1] = -CUDART_INF_F;
          if (r1 < lo || r1 >= hi) x[nt][u][2] = x[nt][u][3] = -CUDART_INF_F;
        }
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      softmax_step<D, kSubs, CHUNK>(st[nt], x[nt], score_factor(qs[nt][0], ks), score_factor(qs[nt][1], ks),
                                    vsize, pb[nt]);

#pragma unroll
    for (int u = 0; u < kSubs; u += 2) {
      uint32_t vw[2][4][F::kVWords];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          load_val8<D>(vw[s][i], tile, (u + s) * kSub + 2 * t + (i & 1) + (i >> 1) * 8, g);
      if (u + 2 == kSubs) done();
      if (partial) {                           // 0 times what a masked row holds must be 0
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int slot = x0 + (u + s) * kSub + 2 * t + (i & 1) + (i >> 1) * 8;
#pragma unroll
            for (int w = 0; w < F::kVWords; ++w) vw[s][i][w] = slot < lo || slot >= hi ? 0u : vw[s][i][w];
          }
        }
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int mt = 0; mt < F::kMTiles; ++mt) {
          // bytes 2 mt, 2 mt + 1 of rows (2t, 2t + 1) and (2t + 8, 2t + 9), paired by element
          const uint32_t sel = (mt & 1) ? 0x7362 : 0x5140;
          uint32_t a0, a1, a2, a3;
          q8::unpack4<FMT>(prmt(vw[s][0][mt / 2], vw[s][1][mt / 2], sel), a0, a1);
          q8::unpack4<FMT>(prmt(vw[s][2][mt / 2], vw[s][3][mt / 2], sel), a2, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(st[nt].o[mt], a0, a1, a2, a3, pb[nt][u + s][0], pb[nt][u + s][1]);
        }
      }
    }
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
  // in the rings, once every warp is done with its own: (m, r, l)[NW][G8], then O[NW][G8][D] with the
  // c-th four of a column h at c ^ (h / 2 & 3), so that the four columns of a store fall on different banks
  __syncthreads();
  constexpr int G8 = 8 * NT, D4 = D / 4;
  float4* sm_ml = reinterpret_cast<float4*>(smem_al);
  float4* sm_o = sm_ml + NW * G8;
  uint32_t* red = reinterpret_cast<uint32_t*>(smem_al + q8_ring_bytes<D, NT, NW, R>());
  // what the peers of a cluster send: O[rank][share], then (m, r, l)[rank][G8]
  float4* peer_o = reinterpret_cast<float4*>(smem_al + q8_ring_bytes<D, NT, NW, R>() + 16 + NW * R * 8);
  float4* peer_ml = peer_o + G8 * D4 + kMaxCluster;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float l0 = st[nt].l[0], l1 = st[nt].l[1];
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, off);
      l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int h = nt * 8 + 2 * t + e;
      if (g == 0) sm_ml[warp * G8 + h] = make_float4(st[nt].m[e], st[nt].r[e], e ? l1 : l0, 0.f);
      float4* o = sm_o + (warp * G8 + h) * D4;
      if constexpr (D == 16) {                 // two elements a lane
        reinterpret_cast<float2*>(o)[2 * ((g / 2) ^ t) + (g & 1)] = make_float2(st[nt].o[0][e], st[nt].o[0][2 + e]);
      } else {
#pragma unroll
        for (int mt = 0; mt < F::kMTiles; mt += 2)
          o[(g * (D / 32) + mt / 2) ^ t] =
              make_float4(st[nt].o[mt][e], st[nt].o[mt][2 + e], st[nt].o[mt + 1][e], st[nt].o[mt + 1][2 + e]);
      }
    }
  }
  __syncthreads();

  cluster_begun_wait();
  const int live = CHUNK ? min(cols, n_rows * G - c0) : cols;   // columns with a row
  for (int idx = threadIdx.x; idx < cols * D4; idx += NW * 32) {
    const int h = idx / D4, c = idx % D4;
    Four f;
    float4 ml[NW];
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      ml[w] = sm_ml[w * G8 + h];
      f.against(ml[w]);
    }
    if (c == 0 && h < live && fabsf(f.m) >= kMaxTop && f.m != -CUDART_INF_F) raise_status(p.status, SWA_ERR_DEVICE_ARG);
    if (f.m != -CUDART_INF_F) {
#pragma unroll
      for (int w = 0; w < NW; ++w) f.add(ml[w], sm_o[(w * G8 + h) * D4 + (c ^ (h / 2 & 3))]);
    }
    if (p.n_splits == 1) {
      if (h < live) f.store(p.out, row_of(h) * D4 + c, p.out_f32);
    } else if (CHUNK || p.cluster) {
      // each four to the CTA that merges it, (m, r, l) to all
      const int to = idx / per;
      send(at_rank(tc::smem_u32(peer_o + rank * per + idx - to * per), to), f.o, at_rank(peers_bar, to));
      for (int r = c; r < n_cl; r += D4)
        send(at_rank(tc::smem_u32(peer_ml + rank * G8 + h), r), make_float4(f.m, f.r, f.l, 0.f), at_rank(peers_bar, r));
    } else {
      const size_t part = row_of(h) * p.n_splits + split;
      reinterpret_cast<float4*>(p.ws_o)[part * D4 + c] = f.o;
      if (c == 0) reinterpret_cast<float4*>(p.ws_ml)[part] = make_float4(f.m, f.r, f.l, 0.f);
    }
  }

  bool late = false;
  if (p.cluster) {
    late = !tc::mbar_wait(peers_bar, 0, p.status);
    for (int idx = rank * per + threadIdx.x; !late && idx < (rank + 1) * per && idx < live * D4; idx += NW * 32) {
      const int h = idx / D4;
      Four f;
      for (int r = 0; r < n_cl; ++r) f.against(peer_ml[r * G8 + h]);
      for (int r = 0; r < n_cl; ++r) f.add(peer_ml[r * G8 + h], peer_o[r * per + idx - rank * per]);
      f.store(p.out, row_of(h) * D4 + idx % D4, p.out_f32);
    }
  }

  if (fills) {
    auto k_row = [&](int i) { return i == row_new ? kn : kt + (size_t)i * D; };
    auto v_row = [&](int i) { return i == row_new ? vn : vt + (size_t)i * D; };
    const size_t dst = (unit * W + blk0) * D;
    q8::round_block<D, FMT, NW * 32>(k_row, v_row, row_new + 1, p.ring.k8 + dst, p.ring.v8 + dst,
                                     p.ring.k_scale + unit * n_blocks + blk0 / kQ8Block,
                                     p.ring.v_scale + unit * n_blocks + blk0 / kQ8Block, red);
  }
  if (late) {
    // A peer's own wait has run out (raised in the status word) and it comes late: until it has ended its stores may
    // still arrive here.  Each thread has its own verdict, so this stands behind the last barrier of the CTA: threads
    // that saw the bytes land go on and leave, which the cluster's barrier counts as arrived.
    asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
    tc::mbar_wait(peers_bar, 0, p.status);
  }
}

// Merge of the per-split partials: grid B * Hq, a warp; lanes share the splits' (m, r, l), then each has four elements.
// (One pair of 1024 blocks: 15.5 us, and 23.4 with every lane going through all splits' sums.)
template <int D>
__global__ void __launch_bounds__(32) swa_q8_decode_combine_kernel(const Q8DecodeParams p) {
  __shared__ float weight[kSms];                     // a pair has at most a split for each SM
  wait_prior_grid();
  allow_next_grid();
  const size_t bh = blockIdx.x;
  if (p.pos[bh / p.n_q_heads] < 0) return;
  const int S = p.n_splits, lane = threadIdx.x;
  const float4* parts = reinterpret_cast<const float4*>(p.ws_ml) + bh * S;
  Four f;
  for (int s = lane; s < S; s += 32) f.against(parts[s]);
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    f.m = fmaxf(f.m, __shfl_xor_sync(0xffffffffu, f.m, off));
    f.r = fmaxf(f.r, __shfl_xor_sync(0xffffffffu, f.r, off));
  }
  for (int s = lane; s < S; s += 32) {
    const float4 part = parts[s];
    weight[s] = fast_exp2(part.x - f.m);
    f.l += fast_exp2(part.y - f.r) * part.z;
  }
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) f.l += __shfl_xor_sync(0xffffffffu, f.l, off);
  __syncwarp();
  if (lane >= D / 4) return;
  const float4* o = reinterpret_cast<const float4*>(p.ws_o) + bh * S * (D / 4) + lane;
#pragma unroll 8
  for (int s = 0; s < S; ++s) {
    const float4 x = o[(size_t)s * (D / 4)];
    f.o.x += weight[s] * x.x;
    f.o.y += weight[s] * x.y;
    f.o.z += weight[s] * x.z;
    f.o.w += weight[s] * x.w;
  }
  f.store(p.out, bh * (D / 4) + lane, p.out_f32);
}

namespace {

constexpr int kMaxDevices = 64;

template <int D, int NT, int V, int FMT, bool CHUNK>
cudaError_t launch_t(const Q8DecodeParams& p, const Q8DecodeMaps& maps, cudaStream_t stream) {
  constexpr int NW = kQ8Variants[V].warps, R = kQ8Variants[V].tiles;
  constexpr int smem = q8_smem_bytes<D, NT, NW, R>(V == 0);   // only variant 0 comes in clusters
  auto kern = swa_q8_decode_kernel<D, NT, NW, R, kQ8Variants[V].per_sm, FMT, CHUNK>;
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
  cfg.gridDim = dim3(p.n_splits, p.n_kv_heads * p.groups, p.batch);
  cfg.blockDim = dim3(NW * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster ? 2 : 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p, maps.k, maps.v);
  if (e != cudaSuccess || p.n_splits == 1 || p.cluster) return e;
  cudaLaunchConfig_t ccfg = {};
  ccfg.gridDim = dim3((unsigned)((size_t)p.batch * p.n_q_heads));
  ccfg.blockDim = dim3(32);
  ccfg.stream = stream;
  ccfg.attrs = attr;
  ccfg.numAttrs = 1;
  return cudaLaunchKernelEx(&ccfg, swa_q8_decode_combine_kernel<D>, p);
}

// Variant 2 needs a kernel of at most 168 registers: not two n-tiles, nor the rows of a chunk.
template <int D, int NT, int FMT, bool CHUNK>
cudaError_t launch_v(const Q8DecodeParams& p, const Q8DecodeMaps& maps, cudaStream_t stream) {
  if (p.variant == 0) return launch_t<D, NT, 0, FMT, CHUNK>(p, maps, stream);
  if (p.variant == 1) return launch_t<D, NT, 1, FMT, CHUNK>(p, maps, stream);
  if constexpr (NT == 1 && !CHUNK) {
    if (p.variant == 2) return launch_t<D, NT, 2, FMT, CHUNK>(p, maps, stream);
  }
  return cudaErrorInvalidValue;
}

template <int D, int FMT>
cudaError_t launch_f(const Q8DecodeParams& p, const Q8DecodeMaps& maps, cudaStream_t stream) {
  const int G = p.n_q_heads / p.n_kv_heads;
  if (p.n_tokens != nullptr)
    return p.max_tokens * G <= 8 ? launch_v<D, 1, FMT, true>(p, maps, stream) : launch_v<D, 2, FMT, true>(p, maps, stream);
  return G <= 8 ? launch_v<D, 1, FMT, false>(p, maps, stream) : launch_v<D, 2, FMT, false>(p, maps, stream);
}

template <int D>
cudaError_t launch_d(const Q8DecodeParams& p, const Q8DecodeMaps& maps, cudaStream_t stream) {
  return p.ring.format == SWA_Q8_E4M3 ? launch_f<D, SWA_Q8_E4M3>(p, maps, stream)
                                      : launch_f<D, SWA_Q8_INT8>(p, maps, stream);
}

}  // namespace
}  // namespace swa
