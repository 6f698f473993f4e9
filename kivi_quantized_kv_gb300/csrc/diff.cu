// diff.cu — host side of the differential attention: launch shape and the
// launch itself.  The kernel is in diff_mma.cuh (design notes there);
// diff_b*.cu instantiate it per code width.
//
// Measured (heads of 128): 8 x 4096 tokens, 32/32 heads, 4 bits 55 us (3.0 TB/s
// of cache bytes; the plain decode of the same cache, half the products, 47);
// 4 x 32768, 32/8 heads, 2 bits 51 us (1.8 TB/s); 32 windows of 4096, 8 bits, groups
// of 64, 73 us (3.7 TB/s); one sequence of 256 tokens 9 us.  The first case at
// 1 to 8 bits: 67, 54, 69, 55, 79, 84, 80 and 60 us (bit streams read and shift
// more words a code).  The fused step takes 1 us more than the decode, a freezing
// step among 32 included.
// Bound by a group's instructions and their latencies: 28 M warp instructions
// for the first case (860 per warp and group of 32 tokens, some 240 of them for
// the codes), issue slots 52 % busy (35 % for the windows, ten warps an SM) with
// the sixteen warps that 128 registers allow, whose first stalls are fixed
// latencies (1.9 warps an issue), the math pipe and shared memory (1.0 each);
// tensor pipe 27 %, DRAM reads as many as the cache's bytes.
#include "diff_launch.cuh"

namespace kivi {

DiffShape diff_shape(const Geo& g) {
  DiffShape sh{};
  auto up = [](int64_t x, int64_t a) { return (x + a - 1) / a * a; };
  // a block, or a tail chunk (4 fp32 or 8 fp16 tokens, keys and values)
  const int64_t chunk = 32 * static_cast<int64_t>(g.d);
  const int64_t blk = up(g.block_bytes > chunk ? g.block_bytes : chunk, 128);
  const int64_t q_bytes = 2 * 16 * (g.d / 2 + 16);
  const int64_t slot = 2 * (g.d / 4 + 3) * 32 * 4;
  const int64_t xch = 8 * (g.G % 32 == 0 ? 512 : 256);
  const int64_t budget = 227 * 1024 - 2048;   // room for the static shared memory
  auto bytes = [&](int64_t np, int64_t ns) {
    return np * (ns * 2 * blk + xch + 8 * (ns > 1 ? ns : 3)) + q_bytes + (np / 2 > 0 ? np / 2 : 1) * slot;
  };
  // as many pairs as fit, then stages (up to four) while they fit: more warps
  // hide more than a second stage does (8 bits, groups of 64, 32 x 4096
  // tokens: 72 us with five pairs of one stage, 82 with three of two; 4 bits,
  // groups of 64, 8 x 8192: 36 with eight of one, 42 with five of two)
  int64_t np = mma::kDiffPairs, ns = 1;
  while (np > 1 && bytes(np, ns) > budget) --np;
  while (ns < 4 && bytes(np, ns + 1) <= budget) ++ns;
  sh.np = static_cast<int32_t>(np);
  sh.ns = static_cast<int32_t>(ns);
  sh.blk_off = static_cast<int32_t>(blk);
  sh.smem = static_cast<int32_t>(up(bytes(np, ns), 16));
  return sh;
}

cudaError_t launch_diff(DiffArgs a, int64_t num_sms, int64_t partial_floats, cudaStream_t stream) {
  const DiffShape sh = diff_shape(a.g);
  a.np = sh.np;
  a.ns = sh.ns;
  a.blk_off = sh.blk_off;
  // CTAs: at most one per SM, and at least four positions each.  Where all
  // units are alike, whole numbers of them per unit, so that no CTA ends one
  // unit and begins another (16 units of 74 positions: 11.3 us with 144 CTAs,
  // 15.6 with 152; 128 units of 142: 55.4 with 128, 58.0 with 152), unless the
  // blocks are so large that few pairs fit and an SM more counts for more (32
  // units of 64 positions, groups of 240 8-bit tokens: 128 us with 128, 109
  // with 152).
  // And about sqrt(2 uw) a unit at most: k CTAs take uw / k of the walk's time and
  // k of the merge's (4 units of 45 positions: 13.3 us with 10 CTAs each, 15.7
  // with 25, 22.4 with one; of 141: 16.7 with 10, 18.9 with 33).
  const int64_t records = partial_floats / diff_partial_floats(a.rows, a.g.d);   // of one unit and CTA
  const int64_t most = num_sms < (a.W + 3) / 4 ? num_sms : (a.W + 3) / 4;
  int64_t ctas = most < records / 2 ? most : records / 2;
  a.slots = 2;
  if (a.n_runs == 1) {
    const int64_t uw = a.r[0].uw, units = a.W / uw;
    int64_t k = 1;
    while ((k + 1) * (k + 1) <= 2 * uw) ++k;
    const int64_t whole = (most < records ? most : records) / units;   // CTAs a unit, one record each
    if (whole >= 1 && (sh.np >= 4 || whole > k)) {
      ctas = (whole < k ? whole : k) * units;
      a.slots = 1;
    }
  }
  if (ctas < 1 || a.W / ctas >= (int64_t{1} << 30)) return cudaErrorInvalidValue;
  if (injected_launch_failure()) return cudaErrorLaunchFailure;
  const dim3 grid(static_cast<unsigned>(ctas));
  const int threads = 64 * sh.np;
  switch (a.g.bits) {
    case 1: return mma::launch_diff_b1(a, grid, threads, sh.smem, stream);
    case 2: return mma::launch_diff_b2(a, grid, threads, sh.smem, stream);
    case 3: return mma::launch_diff_b3(a, grid, threads, sh.smem, stream);
    case 4: return mma::launch_diff_b4(a, grid, threads, sh.smem, stream);
    case 5: return mma::launch_diff_b5(a, grid, threads, sh.smem, stream);
    case 6: return mma::launch_diff_b6(a, grid, threads, sh.smem, stream);
    case 7: return mma::launch_diff_b7(a, grid, threads, sh.smem, stream);
    default: return mma::launch_diff_b8(a, grid, threads, sh.smem, stream);
  }
}

}  // namespace kivi
