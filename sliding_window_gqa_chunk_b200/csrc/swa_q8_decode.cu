// swa_q8_decode.cu - how a decode step, or a chunk of few rows, over the 8-bit cache is
// spread over the SMs (the kernels are in swa_q8_decode.cuh).
#include "swa_internal.h"

namespace swa {

cudaError_t launch_q8_decode_16(const Q8DecodeParams& p, const Q8DecodeMaps& maps, cudaStream_t stream);
cudaError_t launch_q8_decode_64(const Q8DecodeParams& p, const Q8DecodeMaps& maps, cudaStream_t stream);
cudaError_t launch_q8_decode_128(const Q8DecodeParams& p, const Q8DecodeMaps& maps, cudaStream_t stream);

namespace {

// Blocks of a window from which the pairs, where there are fewer than 148 / 8, go over all SMs and are
// merged by a second kernel, not over clusters of 8: 8 pairs of 2048 blocks take 54 us and 61, of 512
// blocks 21 and 20, of 64 blocks 9.5 and 7.0.
constexpr int kLongBlocks = 512;

// Microseconds that `pairs` CTAs of variant v take in waves of what the SMs hold: a wave takes as long
// as its bytes from HBM (where rows are short and more pairs are read at once, a quarter longer), but
// at least as long as a CTA alone on its SM: 5 us to begin and to end, and `alone` a block.
double waves_us(int v, long long pairs, double blocks, int head_dim) {
  static const double alone[3] = {0.2, 0.35, 0.42};
  const double bytes_us = blocks * head_dim * 2 * kQ8Block / 6.8e6 * (v > 0 && head_dim < 128 ? 1.25 : 1.0);
  const double least = 5.0 + blocks * alone[v] * head_dim / 128;
  auto wave = [&](long long n) { return n * bytes_us > least ? n * bytes_us : least; };
  const long long slots = (long long)kSms * kQ8Variants[v].per_sm;
  return pairs / slots * wave(slots) + (pairs % slots ? wave(pairs % slots) : 0.0);
}

}  // namespace

// How the pairs (of a chunk: the CTAs' shares of their columns) are spread; a function of the shape
// alone.
//  - Fewer pairs than SMs: CTAs of 8 warps, one an SM, and the blocks of a pair over the CTAs of a cluster
//    of at most 8 as long as each warp has one, or, for one token in a long window, over all SMs and
//    merged by a second kernel.
//  - More: a CTA to a pair, of the variant that waves_us() likes best.  Measured (us; variants 0, 1, 2):
//    64 blocks, d = 128: 256 pairs 47, 47, 46; 320: 64, 75, 58; 512: 88, 84, 104; 768: 126, 123, 121;
//    1184: 186, 192, 184.  4 blocks, 1024 pairs: 42, 27, 24.  63 blocks, d = 64, 800 pairs: 70, 70, 70.
Q8DecodeSplit q8_decode_split(int batch, int n_kv_heads, int window, int head_dim, int groups, bool chunk, bool wide) {
  const long long units = (long long)batch * n_kv_heads * groups;
  const long long n_blocks = ((long long)window + kQ8Block - 1) / kQ8Block;
  Q8DecodeSplit s;
  long long splits = 1;
  s.variant = 0;
  s.cluster = 0;
  if (units < kSms) {
    splits = kSms / units;
    if (splits > kQ8MaxCluster && (chunk || n_blocks < kLongBlocks)) splits = kQ8MaxCluster;
    const long long useful = (n_blocks + kQ8Variants[0].warps - 1) / kQ8Variants[0].warps;
    if (splits > useful) splits = useful;
    s.cluster = splits <= kQ8MaxCluster;
  } else {
    const int variants = chunk || wide ? 2 : 3;   // those that have the registers
    for (int v = 1; v < variants; ++v)
      if (waves_us(v, units, (double)n_blocks, head_dim) < waves_us(s.variant, units, (double)n_blocks, head_dim))
        s.variant = v;
  }
  const long long per = (n_blocks + splits - 1) / splits;
  s.slots_per_split = (int)(per * kQ8Block);
  s.n_splits = (int)((n_blocks + per - 1) / per);
  if (s.n_splits == 1) s.cluster = 0;
  return s;
}

// Clusters do not cross the borders of the GPU's clusters of SMs, so of the larger sizes 148 SMs hold less than
// 148 CTAs (105 in clusters of 7, 120 of 8): pairs that do not all fit at once would take twice as long.
// 16 pairs of 64 blocks: 12.4 us in clusters of 8, 8.6 of 6; 48 pairs: 20.8 us of 3, 14.2 of 2.
Q8DecodeSplit q8_fit_clusters(Q8DecodeSplit s, long long units, int window) {
  const long long n_blocks = ((long long)window + kQ8Block - 1) / kQ8Block;
  for (int size = s.n_splits - 1; s.cluster && size >= 1; --size) {
    const int room = q8_clusters_at_once(s.n_splits);
    if (room == 0 || units <= room) break;
    const long long per = (n_blocks + size - 1) / size;
    s.slots_per_split = (int)(per * kQ8Block);
    s.n_splits = (int)((n_blocks + per - 1) / per);
    if (s.n_splits == 1) s.cluster = 0;
  }
  return s;
}

// A chunk's columns go straight over the ring's bytes, which each 16 of them read again, or the ring is
// written out in bf16 and attended to in tiles of 128 rows, which a CTA takes 35 us for in a window of 4096
// however few of them there are.  Over the bytes go up to 128 columns; what the SMs hold at once (up to 512
// rows, which one CTA of a pair reads alone); and up to 256 columns of up to 64 rows in two waves (of windows
// of up to 8192: the written-out way has less to do before the first key and less for each).  Measured over the
// bytes and written out (us, W = 4096, d = 128; 32 query heads over 8): 16 sequences x 4 rows 31, 208; 16 x 32
// rows 192, 212; 1 x 64 rows 28, 50; 2 x 64 50, 55; 4 x 33 57, 74; 4 x 48 83, 75; 1 x 128 53, 51.  4 over 1:
// 1 x 512 rows 39, 43; 1 x 1024 94, 43.  1 over 1: 1 x 512 26, 37; 1 x 1024 44, 38; 1 x 2048 75, 37.  In two
// waves: 8 over 8, W = 7215, 3 x 164 rows 91, 83; 16 over 4, W = 16270, 3 x 53 161, 116.
int q8_chunk_groups(long long rows, int group, long long pairs, int window) {
  const long long columns = rows * group, groups = columns > 8 ? (columns + 15) / 16 : 1, units = pairs * groups;
  const bool over_bytes = columns <= 128 || (units <= kSms && rows <= 512) ||
                          (units <= 2 * kSms && columns <= 256 && rows <= 64 && window <= 8192);
  return over_bytes ? (int)groups : 0;
}

cudaError_t launch_q8_decode(const Q8DecodeParams& p, const Q8DecodeMaps& maps, cudaStream_t stream) {
  switch (p.head_dim) {
    case 16: return launch_q8_decode_16(p, maps, stream);
    case 64: return launch_q8_decode_64(p, maps, stream);
    case 128: return launch_q8_decode_128(p, maps, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace swa
