// pages.cu — copying, forking, compacting and freeing sequences of a cache.
//
// A sequence's state is its live bytes (sinks, ring tokens not yet frozen,
// frozen group blocks) at fixed offsets of its H_kv units, and its token
// count on the host.  Freeing is a count of zero; everything else is moving
// live bytes between sequences, in one cache or from one cache to another.
//
// In place, the new sequence b is the old sequence src[b] for all b at once:
// forks (one source, several destinations), chains and cycles.  A copy of
// some offset of a unit depends only on the same offset of other sequences, so a
// thread that owns an offset carries out the whole map there, in an order in
// which every old value is read before it is written over; it needs no
// scratch, no second pass and no other thread.  The host lays the map out as
// programs of steps (Step below), one program per connected part of the map:
// a source is loaded once and stored to all of its destinations, after the
// sources among those destinations have been through their own; a cycle is
// opened by keeping one member's old value in a register.  Parts run in
// parallel (gridDim.z).
//
// What bounds it: bytes, each live source byte read once and each live
// destination byte written once.  The blocks, nearly all of them, are one plain
// range of a unit: a CTA takes kCols x 2 KB of it, a thread kCols 16-byte
// offsets, whose loads go out together.  The sinks and the ring, whose rows
// are live one by one, have CTAs of their own (gridDim.x's last ones).
//
// Measured, read and written bytes: four sequences of up to 32768 tokens of 8
// bits into another cache (420 MB) 62 us, 6.8 TB/s (a plain copy's rate); two
// sequences of 4096 tokens forked to six others (168 MB) 27 us, 6.2 TB/s, eight of
// them turned round a cycle (336 MB) 54 us and swapped in pairs 52 us; one of 256
// tokens 2 us, a launch's own time.
#include "kivi_internal.cuh"

namespace kivi {
namespace {

// (small CTAs of few columns fill the SMs evenly: eight forks among 24 sequences
// of 2000 2-bit tokens 7.0 us, 9.4 with 256 threads and eight columns, long
// copies 2 % faster; two columns lose 3 % on those)
constexpr int kThreads = 128;
constexpr int kCols = 4;
constexpr int64_t kSpan = 16 * static_cast<int64_t>(kThreads) * kCols;   // bytes of a CTA

// Whether the 16 bytes at `off`, before the blocks, are live: in a sink or a
// ring row that holds a token.
__device__ __forceinline__ bool live_row(const PageArgs& a, const Step& s, int32_t off) {
  if (off < a.res_k) {
    const int32_t x = off >= a.sink_v ? off - static_cast<int32_t>(a.sink_v) : off;
    return x / (4 * a.d) < s.n_sink;
  }
  const int32_t x = off - static_cast<int32_t>(off >= a.res_v ? a.res_v : a.res_k);
  const int32_t rel = x / (2 * a.d) - s.rs0;
  return (rel < 0 ? rel + a.R : rel) < s.n_res;
}

// CYCLE: some program keeps a value (a cycle's opening).
template <bool CYCLE>
__global__ void __launch_bounds__(kThreads) pages_kernel(const __grid_constant__ PageArgs a, int32_t blk_ctas) {
  const int h = blockIdx.y;
  const int first = a.part[blockIdx.z], last = a.part[blockIdx.z + 1];
  const bool rows = static_cast<int>(blockIdx.x) >= blk_ctas;   // the sinks and the ring
  const int64_t off0 = rows ? (static_cast<int64_t>(blockIdx.x) - blk_ctas) * kSpan + 16 * static_cast<int>(threadIdx.x)
                            : a.groups + static_cast<int64_t>(blockIdx.x) * kSpan + 16 * static_cast<int>(threadIdx.x);
  constexpr int kNext = 16 * kThreads;   // bytes to the thread's next offset
  uint4 now[kCols], kept[CYCLE ? kCols : 1];
  uint32_t on = 0u;   // which of the thread's offsets are live at the step's source
  uint32_t held = 0u; // (checked build) which of them the kept value has
  for (int i = first; i < last; ++i) {
    const Step& s = a.step[i];
    if (s.src != kStepSame) {
      on = 0u;
#pragma unroll
      for (int k = 0; k < kCols; ++k) {
        const int64_t off = off0 + k * kNext;
        const bool l = rows ? off < a.groups && live_row(a, s, static_cast<int32_t>(off)) : off < s.end;
        on |= l ? 1u << k : 0u;
      }
    }
    if (s.src >= 0) {
      const uint8_t* p = a.src + (static_cast<int64_t>(s.src) * a.hkv + h) * a.src_unit + off0;
      if constexpr (kDebugChecks) {   // what may not be read is not stored either
        for (int k = 0; k < kCols; ++k)
          if ((on >> k & 1u) && !dbg_in_range(a.src_lo, a.src_hi, a.src_err, p + k * kNext, 16)) on &= ~(1u << k);
      }
#pragma unroll
      for (int k = 0; k < kCols; ++k)
        if (on >> k & 1u) now[k] = *reinterpret_cast<const uint4*>(p + k * kNext);
    } else if (CYCLE && s.src == kStepKept) {
#pragma unroll
      for (int k = 0; k < kCols; ++k) now[k] = kept[CYCLE ? k : 0];
      if constexpr (kDebugChecks) on &= held;
    }
    if (CYCLE && s.dst < 0) {
#pragma unroll
      for (int k = 0; k < kCols; ++k) kept[CYCLE ? k : 0] = now[k];
      if constexpr (kDebugChecks) held = on;
      continue;
    }
    uint8_t* p = a.dst + (static_cast<int64_t>(s.dst) * a.hkv + h) * a.dst_unit + off0;
#pragma unroll
    for (int k = 0; k < kCols; ++k)
      if ((on >> k & 1u) && dbg_in_range(a.dst_lo, a.dst_hi, a.dst_err, p + k * kNext, 16))
        *reinterpret_cast<uint4*>(p + k * kNext) = now[k];
  }
}

}  // namespace

cudaError_t launch_pages(const PageArgs& a, cudaStream_t s) {
  if (a.parts < 1) return cudaSuccess;
  const int64_t blk = a.end > a.groups ? (a.end - a.groups + kSpan - 1) / kSpan : 0;
  const dim3 grid(static_cast<unsigned>(blk + (a.groups + kSpan - 1) / kSpan), a.hkv, a.parts);
  bool cycle = false;
  for (int32_t i = 0; i < a.part[a.parts]; ++i) cycle = cycle || a.step[i].dst < 0;
  if (injected_launch_failure()) return cudaErrorLaunchFailure;
  if (cycle) pages_kernel<true><<<grid, kThreads, 0, s>>>(a, static_cast<int32_t>(blk));
  else pages_kernel<false><<<grid, kThreads, 0, s>>>(a, static_cast<int32_t>(blk));
  return cudaGetLastError();
}

}  // namespace kivi
