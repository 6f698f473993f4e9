// diff_chunk.cu — launch of the differential attention of many query rows and
// of the merge of its parts.  The kernels are in diff_chunk.cuh (design notes
// there); diff_chunk_b*.cu instantiate the first per code width.
//
// Measured (heads of 128): 512 queries of 32/8 heads over 2 x 8192 tokens of 4 bits
// 271 us, 0.74 PFLOP/s (0.38 of the library's bf16 product): the first kernel
// 246, the merge 20; of 2 bits 273, of 8 bits 264; heads of 64 196.  Tensor pipe 35 %, issue slots 58 % of the 18 warps that 96
// registers allow.  Bound by the dequantizing groups, a CTA's busiest role (some
// 1800 warp instructions and 48 KB of shared-memory stores for a token tile of
// 2250 cycles, of which the products take 770): a third group of them, at 80
// registers, brought nothing, nor did the softmax without its exponentials.
#include "diff_chunk_launch.cuh"

namespace kivi {

// Word-rule widths (their codes unpack two at a time into fp16 with one
// AND-OR) and groups that divide a token tile, whose packed rows are whole
// (bulk copies).  The other caches keep the kernel of diff_mma.cuh, which walks the
// cache once for four query rows: 3.0 ms at 3 bits, 2.8 at 4 and 3.8 at 8 with
// groups of 128.
bool chunk_kernel_takes(const Geo& g) { return word_rule(g.bits) && kChunkTokens % g.G == 0; }

template <int D, int AHEAD>
static cudaError_t launch_merge(const ChunkArgs& a, cudaStream_t stream) {
  chunk::diff_chunk_merge_kernel<D, AHEAD><<<dim3(a.units / 2, kChunkRows / 32), 512, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_diff_chunk(const ChunkArgs& a, cudaStream_t stream) {
  if (a.ctas < 1 || a.ctas > a.W || a.units < 2 || a.n_tiles < 1) return cudaErrorInvalidValue;
  if (injected_launch_failure()) return cudaErrorLaunchFailure;
  cudaError_t e;
  if (a.g.bits == 2) e = chunk::launch_chunk_b2(a, stream);
  else if (a.g.bits == 4) e = chunk::launch_chunk_b4(a, stream);
  else if (a.g.bits == 8) e = chunk::launch_chunk_b8(a, stream);
  else return cudaErrorInvalidValue;
  if (e != cudaSuccess) return e;
  if (injected_launch_failure()) return cudaErrorLaunchFailure;
  // With a unit or more per CTA most have one part or two, and two merging CTAs
  // fit an SM (512 queries x 2 x 8192 tokens: 4 us less than with two parts
  // ahead); with fewer, a unit has many, whose latency is all there is (32
  // queries over 4096: 33.5 us, 35.4 with two ahead, 44.7 with one).
  const bool few = a.units >= a.ctas;
  if (a.g.d == 64) return few ? launch_merge<64, 1>(a, stream) : launch_merge<64, 4>(a, stream);
  return few ? launch_merge<128, 1>(a, stream) : launch_merge<128, 4>(a, stream);
}

}  // namespace kivi
