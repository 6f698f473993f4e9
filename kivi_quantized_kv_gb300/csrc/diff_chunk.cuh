// diff_chunk.cuh — differential attention of many query rows (chunks of a
// prompt) on the fifth-generation tensor cores.
//
// The formulas are those of diff_mma.cuh.  With many query rows a cache
// block's codes are worth turning into fp16 once for all of them, and the
// products are large enough for tcgen05: a unit is (128 query rows, sequence, kv
// pair, map), and a CTA walks the unit's token tiles of 64 tokens:
//   S = Q Kᵀ      128 x 64, Q in TMEM, K in shared memory, S into TMEM
//   P = 2^(S c - m)   rows in registers, back to TMEM as fp16
//   O += P V      128 x 2 d, P from TMEM, Vᵀ in shared memory
// TMEM at d = 128: O 256 columns, three S (P) buffers of 64, Q 64.  Keys are
// stored token by token and values channel by channel, which is K-major for
// both products, so the dequantized rows go to shared memory as they come, in
// the 128-byte swizzle.
//
// Roles, one CTA of 18 warps per SM:
//   warps 0-7    softmax, a thread per row: two groups of four warps, one for
//                even and one for odd tiles, that hand the rows' running max to
//                one another; it moves only when it grows by more than 2^8, so
//                O is rarely rescaled; at a unit's end they write its record
//   warp 8       one thread issues the MMAs: S of tile i + 2 before O of tile
//                i, so that no group waits for its S (three stages of K, V and
//                S: 268 us, 285 with S one tile ahead)
//   warp 9       one thread copies packed tiles into a ring of stages (bulk
//                copies: a group's keys with their scales, either head's values
//                with theirs)
//   warps 10-17  dequantize packed tiles into K (64 x d) and Vᵀ (2 d x 64): two
//                groups of four warps, one for even and one for odd tiles (a
//                tile's waits, fences and scales cost a warp as much as the
//                conversion of half of its rows: 373 us with eight warps on
//                every tile, 325 so)
// The roles' loops are short on purpose: unrolled over 128-token tiles, with
// the codes on their way in registers instead of the ring, the warps of an SM
// waited for instructions (2.8 warps an issue) more than for anything else
// (444 us against 384 for the same roles in this form; 512 queries x 2 x 8192
// tokens).
//
// Rounding.  K and V are rounded once to fp16 from code, step and minimum
// (one fused multiply-add), P once; each is half a step of 2^-11 relative,
// independent from element to element; Q is exact, S, O, the max and the sums
// are fp32.
//
// Work split: the units' token tiles laid end to end, one equal range per
// CTA.  Every part of a unit goes to a record in scratch (O by channel, so
// that rows are adjacent and the stores coalesce), and a second launch merges
// the parts of both maps, takes the difference, the norm and writes fp16: the
// two maps of a row are in different CTAs, and the records cost 2 x 130 KB
// per 128 rows and map against some hundreds of token tiles.
//
// Figures and what bounds it: beside the launch in diff_chunk.cu.
#pragma once

#include "decode_mma.cuh"

namespace kivi {
namespace chunk {

using mma::bulk_arm;
using mma::fence_mbar_init;
using mma::fence_proxy_async;
using mma::hfma2_u;
using mma::kLog2e;
using mma::kRescale;
using mma::kWaitNs;
using mma::mbar_arrive_if;
using mma::mbar_init;
using mma::mbar_wait;
using mma::pack_half2;
using mma::smem_addr;

constexpr int kSoftWarps = 8, kMmaWarp = 8, kCopyWarp = 9, kDeqWarp0 = 10, kDeqWarps = 8, kDeqGroup = 4;
constexpr int kThreads = 32 * (kDeqWarp0 + kDeqWarps);
constexpr int kTile = kChunkTokens;   // tokens of a tile

// ------------------------------------------------------------ PTX helpers
// A K-major operand in shared memory with the 128-byte swizzle: rows of 64
// fp16, groups of eight rows 1024 bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(1) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}
// fp16 x fp16 -> fp32, M = 128, both operands K-major
constexpr uint32_t instr_desc(int n) { return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24); }

// The whole warp comes here with the same operands and one elected lane issues:
// the instructions take their operands from uniform registers, which a
// single-lane branch, or a predicate of another kind, would have to fill through
// loops over the lanes (391 us against 325).
// `go` off in that lane: nothing is issued.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add, bool go) {
  asm volatile("{\n\t.reg .pred p, e, g;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 g, %5, 0;\n\telect.sync _|e, 0xFFFFFFFF;\n\t"
               "and.pred e, e, g;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
               :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add)), "r"(static_cast<uint32_t>(go)) : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar, bool go) {
  asm volatile("{\n\t.reg .pred e, g;\n\tsetp.ne.u32 g, %1, 0;\n\telect.sync _|e, 0xFFFFFFFF;\n\tand.pred e, e, g;\n\t"
               "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
               ::"r"(bar), "r"(static_cast<uint32_t>(go)) : "memory");
}
__device__ __forceinline__ void copy_one(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xFFFFFFFF;\n\t"
               "@e cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}"
               ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of the warp's 32 lanes
__device__ __forceinline__ void tmem_ld32(uint32_t (&v)[32], uint32_t addr) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
               "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
               "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                 "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
                 "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
                 "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
               : "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&v)[32]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
               "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
               "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
               :: "r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
                  "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
                  "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]),
                  "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
               : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               :: "r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void bar_sync(int id) { asm volatile("bar.sync %0, 256;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void bar_arrive(int id) { asm volatile("bar.arrive %0, 256;" ::"r"(id) : "memory"); }
// two fp32 at once
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// --------------------------------------------------------------- layout
template <int D>
struct Smem {
  static constexpr int kAtomK = kTile * 128;            // 64 channels of a key tile
  static constexpr int kK = kTile * D * 2;              // D / 64 atoms
  static constexpr int kV = 2 * D * kTile * 2;          // one atom: 2 D rows x 128 bytes
  static constexpr int kStages = 3;
  static constexpr int oV = kStages * kK, oMax = oV + kStages * kV;
  static constexpr int oBar = oMax + 2 * kChunkRows * 4;
  // barriers: K full, V full, K free and V free (per stage), S full and P full
  // (per buffer, as many), O done (by tile parity), Q full, unit done, raw full
  // and empty (per raw stage), all products done
  static constexpr int kMaxRaw = 6;
  static constexpr int kBars = 6 * kStages + 5 + 2 * kMaxRaw;
  static constexpr int oMisc = oBar + 8 * kBars;
  static constexpr int oRaw = (oMisc + 16 + 127) / 128 * 128;
};
// TMEM columns
template <int D>
struct Tmem {
  static constexpr int kO = 0, kS = 2 * D, kQ = kS + 3 * kTile;   // S and P of buffer b at kS + 64 b
  static constexpr int kCols = 512;                               // 2 D + 192 + D / 2 in use
};
// byte offset of 16-byte part x of row `row` in a swizzled atom
__device__ __forceinline__ uint32_t swz(int row, int x) {
  return static_cast<uint32_t>((row >> 3) * 1024 + (row & 7) * 128 + ((x ^ (row & 7)) << 4));
}

struct Part {       // a CTA's part of one unit
  int u, tile;      // the unit, its row tile
  int b, j, m;
  int first, last;  // its token tiles
};

// Walks a CTA's range of work positions unit by unit; every role does so alike.
struct Walk {
  int pos, end, ti;
  __device__ __forceinline__ Walk(const ChunkArgs& a) {
    pos = static_cast<int>(static_cast<int64_t>(blockIdx.x) * a.W / a.ctas);
    end = static_cast<int>(static_cast<int64_t>(blockIdx.x + 1) * a.W / a.ctas);
    ti = 0;
  }
  __device__ __forceinline__ bool next(const ChunkArgs& a, Part& p) {
    if (pos >= end) return false;
    while (ti + 1 < a.n_tiles && a.t[ti + 1].pos0 <= pos) ++ti;
    const ChunkTile& t = a.t[ti];
    const int kvp = a.g.hkv / 2;
    const int l = (pos - t.pos0) / t.w;
    p.tile = ti;
    p.u = t.ubase + l;
    p.m = l & 1;
    p.j = (l >> 1) % kvp;
    p.b = t.b0 + (l >> 1) / kvp;
    const int base = t.pos0 + l * t.w;
    p.first = pos - base;
    p.last = min(t.w, end - base);
    pos = base + p.last;
    return true;
  }
};

// What a token tile holds: n0 sinks from s0 on, then n1 tokens; those are
// frozen tokens from f on, or (tail) ring tokens from i0 on.
struct Tokens {
  bool tail;
  int n0, n1, s0, f, i0;
  int64_t pos;      // position of the first of the n1 tokens
};
__device__ __forceinline__ Tokens tokens_of(const ChunkArgs& a, const ChunkTile& t, const ChunkRun& r, int i) {
  Tokens k;
  k.tail = i >= t.n_frozen;
  k.s0 = k.i0 = k.f = k.n0 = 0;
  if (!k.tail) {
    k.f = t.f_begin + kTile * i;
    k.n1 = min(kTile, r.frozen - k.f);
    k.pos = a.g.S + r.g_first * a.g.G + k.f;
  } else {
    k.s0 = kTile * (i - t.n_frozen);
    k.n0 = max(0, min(kTile, t.n_sink - k.s0));
    k.i0 = max(0, k.s0 - t.n_sink);
    k.n1 = max(0, min(kTile - k.n0, t.n_ring - k.i0));
    k.pos = r.ring_pos0 + k.i0;
  }
  return k;
}

// fp16 pair p of a packed slice, codes as fp16 integers (exact)
template <int BITS>
__device__ __forceinline__ uint32_t code_half2(const uint32_t* w, int p) {
  const uint32_t x = mma::code_pair<BITS>(w, p) | 0x64006400u;   // 1024 + code 2^kb
  const uint32_t kb = mma::pair_kb<BITS>(p);
  const uint32_t sc = (15u - kb) << 10, off = 0x8000u | ((25u - kb) << 10);   // 2^-kb, -2^(10 - kb)
  return hfma2_u(x, sc | (sc << 16), off | (off << 16));
}

// The largest code times its step, rounded up at quantization, may carry past
// fp16's range where the values nearly fill it: such a step is taken one unit
// in the last place lower, which brings it back (the true range is finite, and
// the step was at most half a unit too large).
__device__ __forceinline__ uint32_t safe_step(uint32_t step, uint32_t min, uint32_t top) {
  const uint32_t r = hfma2_u(top, step, min);
  return step - ((r & 0xFFFFu) == 0x7C00u ? 1u : 0u) - ((r >> 16) == 0x7C00u ? 0x10000u : 0u);
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// The columns of a token tile that a row sees (positions lo to hi), as bits:
// sinks (no lower end), then the other tokens.  Out of line: only the tiles at the ends
// of what a row tile sees, and tails, need it.
static __device__ __noinline__ uint64_t seen_columns(const ChunkArgs& a, int tile, int i, int64_t lo, int64_t hi) {
  const ChunkTile& t = a.t[tile];
  const Tokens tk = tokens_of(a, t, a.r[t.run], i);
  auto near = [](int64_t x) { return static_cast<int>(min(static_cast<int64_t>(kTile), max(static_cast<int64_t>(0), x))); };
  auto bits = [](int a0, int a1) -> uint64_t { return a1 > a0 ? (~0ull >> (64 - (a1 - a0))) << a0 : 0ull; };   // [a0, a1)
  const int y0 = tk.n0 + near(lo - tk.pos), y1 = tk.n0 + min(tk.n1, near(hi - tk.pos + 1));
  return bits(0, min(tk.n0, near(hi - tk.s0 + 1))) | bits(y0, y1);
}

// A dequantizing warp's share of a tail tile's rows (sinks fp32, ring fp16, both
// exact in fp16): keys, 16 tokens a warp, or values of a head, D / 2 channels a
// warp.  Out of line: it takes no registers from the loop.
template <int D>
static __device__ __noinline__ void tail_rows(const ChunkArgs& a, const Part q, int i, int dw, bool value, uint32_t at) {
  const Geo& g = a.g;
  const ChunkTile& t = a.t[q.tile];
  const ChunkRun& rn = a.r[t.run];
  const Tokens tk = tokens_of(a, t, rn, i);
  const int lane = threadIdx.x & 31, head = value ? dw >> 1 : q.m;
  const uint8_t* unit = a.arena + (static_cast<int64_t>(q.b) * g.hkv + 2 * q.j + head) * g.unit_bytes;
  // row of token x of the tile; null past the last one
  auto row = [&](int x, bool& sink) -> const uint8_t* {
    sink = x < tk.n0;
    if (sink) return unit + (value ? g.sink_v : g.sink_k) + static_cast<int64_t>(tk.s0 + x) * D * 4;
    x -= tk.n0;
    if (x >= tk.n1) return nullptr;
    int slot = rn.rs0 + tk.i0 + x;
    if (slot >= g.R) slot -= g.R;
    return unit + (value ? g.res_v : g.res_k) + static_cast<int64_t>(slot) * D * 2;
  };
  // eight channels of a row as fp16
  auto eight = [&](int x, int part) -> uint4 {
    bool sink;
    const uint8_t* p = row(x, sink);
    if constexpr (kDebugChecks) {   // a row outside the cache reads as zeros
      if (p && !dbg_in_region(g, p, sink ? 4 * D : 2 * D)) p = nullptr;
    }
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (p && sink) {
      const float4 f = reinterpret_cast<const float4*>(p)[2 * part], h = reinterpret_cast<const float4*>(p)[2 * part + 1];
      v = make_uint4(pack_half2(f.x, f.y), pack_half2(f.z, f.w), pack_half2(h.x, h.y), pack_half2(h.z, h.w));
    } else if (p) {
      v = reinterpret_cast<const uint4*>(p)[part];
    }
    return v;
  };
  if (!value) {
    constexpr int KL = D / 8, KX = D / 16;
    const int part = lane % KL;
    uint4 v[KX];
#pragma unroll
    for (int x = 0; x < KX; ++x) v[x] = eight(16 * dw + lane / KL + x * (32 / KL), part);
#pragma unroll
    for (int x = 0; x < KX; ++x)
      sts128(at + (part >> 3) * Smem<D>::kAtomK + swz(16 * dw + lane / KL + x * (32 / KL), part & 7), v[x].x, v[x].y, v[x].z, v[x].w);
  } else {
    // two tokens x eight channels a step, turned into eight rows' pairs
    constexpr int VP = D / 16;   // octets of the warp's channels
#pragma unroll 1
    for (int x0 = lane; x0 < 32 * VP; x0 += 128) {
      uint4 v[4][2];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int x = x0 + 32 * y, t0 = 2 * (x / VP), part = (D / 16) * (dw & 1) + x % VP;
        v[y][0] = eight(t0, part);
        v[y][1] = eight(t0 + 1, part);
      }
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int x = x0 + 32 * y, tp = x / VP, ch = head * D + (D / 2) * (dw & 1) + 8 * (x % VP);
        const uint32_t w0[4] = {v[y][0].x, v[y][0].y, v[y][0].z, v[y][0].w}, w1[4] = {v[y][1].x, v[y][1].y, v[y][1].z, v[y][1].w};
#pragma unroll
        for (int c = 0; c < 8; ++c)
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + swz(ch + c, tp >> 2) + 4 * (tp & 3)),
                       "r"(mma::prmt(w0[c >> 1], w1[c >> 1], (c & 1) ? 0x7632u : 0x5410u)) : "memory");
      }
    }
  }
}

template <int D, int BITS>
__global__ void __launch_bounds__(kThreads, 1) diff_chunk_kernel(const __grid_constant__ ChunkArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  using S = Smem<D>;
  using T = Tmem<D>;
  const Geo& g = a.g;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = smem_addr(smem);
  const uint32_t bars = base + S::oBar;
  auto k_full = [&](int s) { return bars + 8 * s; };
  auto v_full = [&](int s) { return bars + 8 * (S::kStages + s); };
  auto k_free = [&](int s) { return bars + 8 * (2 * S::kStages + s); };
  auto v_free = [&](int s) { return bars + 8 * (3 * S::kStages + s); };
  auto s_full = [&](int b) { return bars + 8 * (4 * S::kStages + b); };
  auto p_full = [&](int b) { return bars + 8 * (5 * S::kStages + b); };
  auto o_done = [&](int b) { return bars + 8 * (6 * S::kStages + b); };
  const uint32_t q_full = o_done(2), u_done = q_full + 8;
  auto raw_full = [&](int s) { return u_done + 8 + 8 * s; };
  auto raw_empty = [&](int s) { return u_done + 8 + 8 * (S::kMaxRaw + s); };
  const uint32_t m_done = u_done + 8 + 8 * 2 * S::kMaxRaw;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::oMisc);

  if (base & 1023u) {   // the swizzled atoms need it; the kernel has no static shared memory in front
    if (tid == 0) atomicOr(a.error, mma::kErrCopy);
    return;
  }
  if (tid == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(k_full(s), kDeqGroup);
      mbar_init(v_full(s), kDeqGroup);
      mbar_init(k_free(s), 1);
      mbar_init(v_free(s), 1);
      mbar_init(s_full(s), 1);
      mbar_init(p_full(s), 16 * kSoftWarps);
    }
    for (int b = 0; b < 2; ++b) mbar_init(o_done(b), 1);
    mbar_init(q_full, 32 * kSoftWarps);
    mbar_init(u_done, 1);
    mbar_init(m_done, 1);
    for (int s = 0; s < a.raw_stages; ++s) {
      mbar_init(raw_full(s), 1);
      mbar_init(raw_empty(s), kDeqGroup);
    }
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)), "n"(T::kCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);

  // Every wait is bounded: the copying warp's by a.wait_ns, the others', whose
  // lanes give up one by one, by kWaitNs, which no test makes shorter.  A warp
  // whose wait ran out waits no more, issues and copies nothing more, and goes on
  // through the barriers; the others' waits for it run out in turn, and the launch
  // ends with the error bit set.
  bool gone = false;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (gone || mbar_wait(bar, parity, kWaitNs)) return;
    gone = true;
    atomicOr(a.error, mma::kErrCopy);
  };
  // where `gone` decides what a whole warp does its lanes have to agree (a vote
  // in every role's waits would cost 46 us of 265; the issuing warp, 15 of them,
  // goes on whatever happens, with its instructions off)
  auto wait_alike = [&](uint32_t bar, uint32_t parity, unsigned long long limit) {
    if (gone || __all_sync(0xffffffffu, mbar_wait(bar, parity, limit))) return;
    gone = true;
    if (lane == 0) atomicOr(a.error, mma::kErrCopy);
  };

  Walk walk(a);
  Part pt;
  if (warp < kSoftWarps) {
    // ------------------------------------------------------------ softmax
    const int half = warp >> 2, row = 32 * (warp & 3) + lane;   // the group's tiles; the warp's TMEM lanes are its rows
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    float* s_max = reinterpret_cast<float*>(smem + S::oMax);    // [tile parity][row]: the running max after a tile
    const float scale = kLog2e * rsqrtf(static_cast<float>(D));
    const int tiles = walk.end - walk.pos;
    int it = 0, units = 0;   // token tiles and parts of units of this CTA so far
    int sb = 0;              // the tile's S buffer
    uint32_t sph = 0;
    while (walk.next(a, pt)) {
      const ChunkTile& t = a.t[pt.tile];
      const ChunkRun& rn = a.r[t.run];
      const int rep = g.rep;
      // Q of the unit, half a row a thread: its last reader was the S product
      // of the tile before, which every softmax thread has waited for
      {
        const int vr = t.row0 + min(row, t.nrow - 1);
        const int64_t at = (static_cast<int64_t>(pt.b) * a.q_rows + vr / rep) * g.hq +
                           2 * (static_cast<int64_t>(pt.j) * rep + vr % rep) + pt.m;
        const uint4* q = reinterpret_cast<const uint4*>(a.q + at * D + half * (D / 2));
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {   // 16 channels, 8 columns
          const uint4 u = __ldg(q + 2 * x), v = __ldg(q + 2 * x + 1);
          dbg_check_finite(g, u);
          dbg_check_finite(g, v);
          const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
          tmem_st8(t_lane + T::kQ + half * (D / 4) + 8 * x, w);
        }
        wait_st();
        fence_before();
        mbar_arrive_if(true, q_full);
      }

      const int64_t hi = rn.q_pos0 + (t.row0 + min(row, t.nrow - 1)) / rep;
      const int64_t lo = g.window > 0 ? hi + 1 - g.window : 0;
      // frozen tiles [i_lo, i_hi) are seen whole by every row of the tile (kept
      // in registers: the plan's indexed constants are slow to read)
      const int64_t f_pos = g.S + rn.g_first * g.G + t.f_begin;   // position of tile 0's first token
      const int64_t hi_min = rn.q_pos0 + t.row0 / rep + 1 - f_pos;
      const int64_t lo_max = g.window > 0 ? rn.q_pos0 + (t.row0 + t.nrow - 1) / rep + 1 - g.window - f_pos : 0;
      const int i_hi = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(rn.frozen - t.f_begin), hi_min)) / kTile);
      const int i_lo = static_cast<int>(max(static_cast<int64_t>(0), lo_max) + kTile - 1) / kTile;
      const int tile = pt.tile, first = pt.first, last = pt.last;
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int i = first; i < last; ++i, ++it) {
        const int b = sb;
        const uint32_t bph = sph;
        if (++sb == S::kStages) { sb = 0; sph ^= 1u; }
        if ((it & 1) != half) continue;
        const uint32_t t_s = t_lane + T::kS + kTile * b;
        uint32_t see0 = ~0u, see1 = ~0u;
        if (i >= i_hi || i < i_lo) {
          const uint64_t see = seen_columns(a, tile, i, lo, hi);
          see0 = static_cast<uint32_t>(see);
          see1 = static_cast<uint32_t>(see >> 32);
        }
        wait(s_full(b), bph);
        fence_after();
        uint32_t s[2][32];
        tmem_ld32(s[0], t_s);
        tmem_ld32(s[1], t_s + 32);
        wait_ld();
        if ((see0 & see1) != ~0u) {
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            if (!(see0 >> c & 1u)) s[0][c] = 0xFF800000u;
            if (!(see1 >> c & 1u)) s[1][c] = 0xFF800000u;
          }
        }
        float m4[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) m4[c] = __uint_as_float(s[0][c]);
#pragma unroll
        for (int c = 4; c < 64; ++c) m4[c & 3] = fmaxf(m4[c & 3], __uint_as_float(s[c >> 5][c & 31]));
        const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * scale;
        // the running max after the tile before, from the other group, and on to it
        if (it > 0) bar_sync(1 + (half ^ 1));
        const float before = i > first ? s_max[(half ^ 1) * kChunkRows + row] : -INFINITY;
        const bool up = mx > before + kRescale || (before == -INFINITY && mx > -INFINITY);
        const float now = up ? mx : before;
        s_max[half * kChunkRows + row] = now;
        if (it + 1 < tiles) bar_arrive(1 + half);
        if (now > m) {   // since this group's last tile
          l *= m == -INFINITY ? 0.f : mma::ex2(m - now);
          m = now;
        }
        const float ref = m == -INFINITY ? 0.f : m;
        // P over the first half of S's columns
        {
          const uint64_t sc2 = pair_of(scale, scale), rf2 = pair_of(-ref, -ref);
          uint64_t l2[2] = {0ull, 0ull};
#pragma unroll
          for (int c0 = 0; c0 < 64; c0 += 16) {
            uint32_t p[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const int y = c0 + 2 * c;
              float e0, e1;
              unpair(fma2(pair_of(__uint_as_float(s[y >> 5][y & 31]), __uint_as_float(s[y >> 5][(y & 31) + 1])), sc2, rf2), e0, e1);
              e0 = mma::ex2(e0);
              e1 = mma::ex2(e1);
              l2[c & 1] = add2(l2[c & 1], pair_of(e0, e1));
              p[c] = pack_half2(e0, e1);
            }
            tmem_st8(t_s + c0 / 2, p);
          }
          float a0, a1;
          unpair(add2(l2[0], l2[1]), a0, a1);
          l += a0 + a1;
        }
        // O of the tile before is complete (it comes before this one's in the
        // tensor pipe anyway); the rows whose max moved bring it along
        if (it > 0) wait(o_done(half ^ 1), ((it - 1) >> 1) & 1);
        if (i > first && __any_sync(0xffffffffu, up)) {
          const float corr = !up ? 1.f : before == -INFINITY ? 0.f : mma::ex2(before - now);
          fence_after();
#pragma unroll 1
          for (int c = 0; c < 2 * D; c += 32) {
            uint32_t o[32];
            const uint32_t at = t_lane + T::kO + c;
            tmem_ld32(o, at);
            wait_ld();
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * corr);
            tmem_st32(at, o);
          }
        }
        wait_st();
        fence_before();
        mbar_arrive_if(true, p_full(b));
      }
      // the part's record: channels by rows, then either group's max and sum
      // (the max only grows, so O's is the larger of the two)
      wait(u_done, units & 1);
      ++units;
      fence_after();
      float* rec = a.records + (static_cast<int64_t>(pt.u) + blockIdx.x) * ((2 * D + 4) * kChunkRows) + row;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        tmem_ld32(o, t_lane + T::kO + half * D + c);
        wait_ld();
#pragma unroll
        for (int x = 0; x < 32; ++x) rec[(half * D + c + x) * kChunkRows] = __uint_as_float(o[x]);
      }
      rec[(2 * D + 2 * half) * kChunkRows] = m;
      rec[(2 * D + 2 * half + 1) * kChunkRows] = l;
      fence_before();   // the next unit's first O product comes after its Q's arrivals
    }
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- MMA
    const uint64_t kd = operand_desc(base), vd = operand_desc(base + S::oV);   // + bytes / 16
    int it = 0, units = 0;
    int ks = 0, vs = 0;   // stages of the next S (keys, S itself) and of the next O (values, P)
    uint32_t kph = 0, vph = 0;
    // the next S, which also frees its keys' stage
    auto s_product = [&]() {
      wait(k_full(ks), kph);
      fence_after();
      const bool go = !gone;
      const uint64_t k0 = kd + static_cast<uint32_t>(ks * (S::kK >> 4));
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        mma_ts(tmem + T::kS + kTile * ks, tmem + T::kQ + 8 * k,
               k0 + static_cast<uint32_t>(((k >> 2) * S::kAtomK + (k & 3) * 32) >> 4), instr_desc(kTile), k > 0, go);
      mma_commit(s_full(ks), go);
      mma_commit(k_free(ks), go);
      if (++ks == S::kStages) { ks = 0; kph ^= 1u; }
    };
    while (walk.next(a, pt)) {
      wait(q_full, units & 1);
      ++units;
      s_product();
      if (pt.first + 1 < pt.last) s_product();
#pragma unroll 1
      for (int i = pt.first; i < pt.last; ++i, ++it) {
        if (i + 2 < pt.last) s_product();
        wait(v_full(vs), vph);
        wait(p_full(vs), vph);
        fence_after();
        const bool go = !gone;
        const uint64_t v0 = vd + static_cast<uint32_t>(vs * (S::kV >> 4));
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          mma_ts(tmem + T::kO, tmem + T::kS + kTile * vs + 8 * k, v0 + static_cast<uint32_t>(2 * k), instr_desc(2 * D),
                 i > pt.first || k > 0, go);
        mma_commit(o_done(it & 1), go);
        mma_commit(v_free(vs), go);
        if (++vs == S::kStages) { vs = 0; vph ^= 1u; }
      }
      mma_commit(u_done, !gone);
    }
    // no product is in flight when TMEM and shared memory are given back, also
    // after a wait that ran out
    mma_commit(m_done, true);
    mbar_wait(m_done, 0, kWaitNs);
    __syncwarp();
  } else if (warp == kCopyWarp) {
    // --------------------------------------------------------------- copy
    {
      const int ng = kTile / g.G;   // groups of a tile
      const uint32_t kb = static_cast<uint32_t>(g.blk_vq), vb = static_cast<uint32_t>(g.blk_vs + 4 * g.G - g.blk_vq);
      int rt = 0, rs = 0;
      uint32_t ph = 1;   // a fresh barrier's phase before the first counts as complete
      while (walk.next(a, pt)) {
        const ChunkTile& t = a.t[pt.tile];
        const ChunkRun& rn = a.r[t.run];
        const uint8_t* k0 = a.arena + (static_cast<int64_t>(pt.b) * g.hkv + 2 * pt.j) * g.unit_bytes + g.groups;
        const uint8_t* kk = k0 + pt.m * g.unit_bytes;
        int grp = (t.f_begin + kTile * pt.first) / g.G;
        for (int i = pt.first; i < pt.last && i < t.n_frozen; ++i, ++rt) {
          wait_alike(raw_empty(rs), ph, a.wait_ns);
          if (gone) break;
          const int n = min(ng, rn.frozen / g.G - grp);
          const uint32_t dst = base + S::oRaw + rs * a.raw_bytes, bar = raw_full(rs);
          if (lane == 0) bulk_arm(bar, n * (kb + 2 * vb));
          __syncwarp();
          for (int x = 0; x < n; ++x) {
            uint32_t slot = rn.slot0 + static_cast<uint32_t>(grp + x);
            if (g.window > 0 && slot >= static_cast<uint32_t>(g.n_slots)) slot -= static_cast<uint32_t>(g.n_slots);
            const int64_t at = static_cast<int64_t>(slot) * g.block_bytes;
            // (checked build: where an address is outside the cache, the
            // cache's first block is read instead, as the barrier counts bytes)
            const bool ok = dbg_in_region(g, k0 + at, g.block_bytes) && dbg_in_region(g, k0 + g.unit_bytes + at, g.block_bytes);
            const uint8_t* first = a.arena + g.groups;
            copy_one(dst + x * kb, ok ? kk + at : first, kb, bar);
            copy_one(dst + ng * kb + x * vb, (ok ? k0 + at : first) + g.blk_vq, vb, bar);
            copy_one(dst + ng * (kb + vb) + x * vb, (ok ? k0 + g.unit_bytes + at : first) + g.blk_vq, vb, bar);
          }
          grp += ng;
          if (++rs == a.raw_stages) { rs = 0; ph ^= 1u; }
        }
      }
      // after a wait that ran out: the copies in flight land (bounded) before
      // the shared memory is given back
      if (gone) {
        for (int x = max(0, rt - a.raw_stages); x < rt; ++x)
          mbar_wait(raw_full(x % a.raw_stages), static_cast<uint32_t>(x / a.raw_stages) & 1u, kWaitNs);
      }
    }
    __syncwarp();
  } else {
    // --------------------------------------------------------- dequantize
    // A thread owns eight channels of a key row (keys: step and min go by
    // channel) or eight tokens of a value row (step and min go by token): it
    // keeps their eight steps and minima in registers and walks the rows, so
    // eight lanes write one whole 128-byte row of an atom.
    const int dw = (warp - kDeqWarp0) % kDeqGroup, grp = (warp - kDeqWarp0) / kDeqGroup;   // the group: its stage
    constexpr int KL = D / 8, KE = 32 / KL;   // lanes of a key row; rows a step
    const int G = g.G, ng = kTile / G, lg = 31 - __clz(G);   // G 16, 32 or 64
    const uint32_t kb = static_cast<uint32_t>(g.blk_vq), vb = static_cast<uint32_t>(g.blk_vs + 4 * G - g.blk_vq);
    const uint32_t vrow = static_cast<uint32_t>(G) * BITS / 8;
    // eight codes of octet o of a row: two words at 8 bits, one at 4; at 2 bits
    // a byte of either half of a word, which is shifted down for the odd octet
    auto octet_at = [](int o) -> uint32_t { return BITS == 2 ? 4 * (o >> 1) : BITS * o; };
    constexpr uint32_t kTop1 = 0x6400u + (1u << BITS) - 1u;   // 1024 + the largest code
    const uint32_t top = hfma2_u(kTop1 * 0x10001u, 0x3C003C00u, 0xE400E400u);
    struct Octet {
      uint32_t w[BITS == 8 ? 2 : 1];
    };
    // (all of a warp's loads of a kind come before its stores: neither moves
    // past the other)
    auto get = [&](uint32_t from, int sh) -> Octet {
      Octet c;
      if constexpr (BITS == 8) {
        const uint2 x = mma::lds64(from);
        c.w[0] = x.x;
        c.w[1] = x.y;
      } else {
        c.w[0] = mma::lds32(from) >> (BITS == 2 ? sh : 0);
      }
      return c;
    };
    auto put = [&](uint32_t at, const Octet& c, const uint32_t (&dd)[4], const uint32_t (&mm)[4]) {
      uint32_t o[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) o[y] = hfma2_u(code_half2<BITS>(c.w, y), dd[y], mm[y]);
      sts128(at, o[0], o[1], o[2], o[3]);
    };
    // keys: tokens 16 dw + ke + KE x, channels 8 kp ..
    constexpr int KX = 16 / KE;
    const int kp = lane % KL, ke = lane / KL, kgrp = (16 * dw) >> lg;
    const uint32_t k_from = kgrp * kb + (16 * dw - (kgrp << lg) + ke) * (D * BITS / 8) + octet_at(kp);
    const uint32_t k_scale = kgrp * kb + static_cast<uint32_t>(g.blk_ks) + 16 * kp;
    const uint32_t k_to = (kp >> 3) * S::kAtomK + (16 * dw + ke) * 128;
    const int k_sh = 8 * (kp & 1);
    // values: channels v_ch + 4 x of the half's head, tokens 8 vp ..
    const int vp = lane & 7, ve = lane >> 3, v_half = dw >> 1, v_ch = (D / 2) * (dw & 1) + ve;
    constexpr int VX = D / 8;
    const int vgrp = (8 * vp) >> lg, voff = 8 * vp - (vgrp << lg);
    const uint32_t v_blk = ng * kb + (v_half * ng + vgrp) * vb;
    const uint32_t v_from = v_blk + v_ch * vrow + octet_at(voff >> 3);
    const uint32_t v_scale = v_blk + static_cast<uint32_t>(g.blk_vs - g.blk_vq) + 4 * voff;
    const uint32_t v_to = (v_half * D + v_ch) * 128;
    const int v_sh = 8 * ((voff >> 3) & 1);

    int it = 0, rs = 0, ds = 0;   // tile; its raw stage; its stage
    uint32_t ph = 0, dph = 1;     // dph: the phase in which the stage became free (a fresh barrier's before the first)
    while (walk.next(a, pt)) {
      const ChunkTile& t = a.t[pt.tile];
      const int frozen = a.r[t.run].frozen - t.f_begin, n_frozen = t.n_frozen;
#pragma unroll 1
      for (int i = pt.first; i < pt.last; ++i, ++it) {
        const int r0 = rs;
        const uint32_t p0 = ph;
        if (i < n_frozen && ++rs == a.raw_stages) { rs = 0; ph ^= 1u; }
        const int d0 = ds;
        const uint32_t empty = dph;
        if (++ds == S::kStages) { ds = 0; dph ^= 1u; }
        if ((it & 1) != grp) continue;
        const uint32_t ks = base + d0 * S::kK, vs = base + S::oV + d0 * S::kV;
        if (i >= n_frozen) {
          wait(k_free(d0), empty);
          tail_rows<D>(a, pt, i, dw, false, ks);
          fence_proxy_async();
          __syncwarp();
          mbar_arrive_if(lane == 0, k_full(d0));
          wait(v_free(d0), empty);
          tail_rows<D>(a, pt, i, dw, true, vs);
          fence_proxy_async();
          __syncwarp();
          mbar_arrive_if(lane == 0, v_full(d0));
          continue;
        }
        const int left = frozen - kTile * i;   // frozen tokens from the tile's first on
        const uint32_t raw = base + S::oRaw + r0 * a.raw_bytes;
        wait(raw_full(r0), p0);
        wait(k_free(d0), empty);
        {
          const uint4 d4 = mma::lds128(raw + k_scale), m4 = mma::lds128(raw + k_scale + 2 * D);
          Octet c[KX];
#pragma unroll
          for (int x = 0; x < KX; ++x) c[x] = get(raw + k_from + x * KE * (D * BITS / 8), k_sh);
          uint32_t dd[4] = {d4.x, d4.y, d4.z, d4.w}, mm[4] = {m4.x, m4.y, m4.z, m4.w};
          const bool none = 16 * dw >= left;   // tokens that do not exist read as zeros
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            dd[y] = none ? 0u : safe_step(dd[y], mm[y], top);
            mm[y] = none ? 0u : mm[y];
          }
#pragma unroll
          for (int x = 0; x < KX; ++x)   // rows ke + KE x of the warp's 16
            put(ks + k_to + x * KE * 128 + (((kp & 7) ^ ke ^ (KE * x & 7)) << 4), c[x], dd, mm);
        }
        fence_proxy_async();
        __syncwarp();
        mbar_arrive_if(lane == 0, k_full(d0));

        wait(v_free(d0), empty);
        {
          const uint4 a4 = mma::lds128(raw + v_scale), b4 = mma::lds128(raw + v_scale + 16);
          Octet c[VX];
          uint32_t from = raw + v_from;
#pragma unroll
          for (int x = 0; x < VX; ++x, from += 4 * vrow) c[x] = get(from, v_sh);
          const uint32_t pr[8] = {a4.x, a4.y, a4.z, a4.w, b4.x, b4.y, b4.z, b4.w};
          uint32_t dd[4], mm[4];
          const bool none = 8 * vp >= left;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            mm[y] = mma::prmt(pr[2 * y], pr[2 * y + 1], 0x7632u);
            dd[y] = none ? 0u : safe_step(mma::prmt(pr[2 * y], pr[2 * y + 1], 0x5410u), mm[y], top);
            mm[y] = none ? 0u : mm[y];
          }
          // rows ve + 4 x: the low row bits are ve, then ve ^ 4
          const uint32_t to0 = vs + v_to + ((vp ^ ve) << 4), to1 = vs + v_to + 512 + ((vp ^ ve ^ 4) << 4);
#pragma unroll
          for (int x = 0; x < VX; ++x) put(((x & 1) ? to1 : to0) + (x >> 1) * 1024, c[x], dd, mm);
        }
        fence_proxy_async();
        __syncwarp();
        mbar_arrive_if(lane == 0, v_full(d0));
        mbar_arrive_if(lane == 0, raw_empty(r0));
      }
    }
  }

  fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(T::kCols) : "memory");
  }
}

// Merges the parts of both maps of 32 rows of a (row tile, sequence, kv pair),
// takes the difference and the norm.  512 threads: lane = row, a warp = D / 8
// channels of both maps; AHEAD parts' loads go out together.
template <int D, int AHEAD>
__global__ void __launch_bounds__(512, AHEAD == 1 ? 2 : 1) diff_chunk_merge_kernel(const __grid_constant__ ChunkArgs a) {
  constexpr int C = D / 8, kWarps = 16;
  __shared__ float s_ss[kWarps][32];
  __shared__ float s_lam[2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int u0 = 2 * blockIdx.x;   // the unit of map 0
  int ti = 0;
  while (ti + 1 < a.n_tiles && a.t[ti + 1].ubase <= u0) ++ti;
  const ChunkTile& t = a.t[ti];
  const int row = 32 * blockIdx.y + lane;
  if (32 * static_cast<int>(blockIdx.y) >= t.nrow) return;   // uniform
  if (warp < 2) {
    float x = 0.f;
    for (int i = lane; i < D; i += 32) x = fmaf(a.lambdas[2 * warp * D + i], a.lambdas[(2 * warp + 1) * D + i], x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (lane == 0) s_lam[warp] = expf(x);
  }

  constexpr int64_t step = static_cast<int64_t>(2 * D + 4) * kChunkRows;
  float v[2][C], L[2];
#pragma unroll
  for (int mp = 0; mp < 2; ++mp) {
    const int u = u0 + mp;
    const int64_t p0 = t.pos0 + static_cast<int64_t>(u - t.ubase) * t.w;
    const int first = mma::owner_of(p0, a.W, a.ctas), n = mma::owner_of(p0 + t.w - 1, a.W, a.ctas) - first + 1;
    const float* rec = a.records + (static_cast<int64_t>(u) + first) * step + row;
    float M = -INFINITY;
    L[mp] = 0.f;
#pragma unroll
    for (int x = 0; x < C; ++x) v[mp][x] = 0.f;
    for (int c0 = 0; c0 < n; c0 += AHEAD) {
      float m0[AHEAD], l0[AHEAD], m1[AHEAD], l1[AHEAD], o[AHEAD][C];
#pragma unroll
      for (int c = 0; c < AHEAD; ++c) {
        m0[c] = m1[c] = -INFINITY;
        l0[c] = l1[c] = 0.f;
#pragma unroll
        for (int x = 0; x < C; ++x) o[c][x] = 0.f;
        if (c0 + c < n) {
          const float* r = rec + (c0 + c) * step;
          m0[c] = r[2 * D * kChunkRows];
          l0[c] = r[(2 * D + 1) * kChunkRows];
          m1[c] = r[(2 * D + 2) * kChunkRows];
          l1[c] = r[(2 * D + 3) * kChunkRows];
#pragma unroll
          for (int x = 0; x < C; ++x) o[c][x] = r[(warp * C + x) * kChunkRows];
        }
      }
      float Mn = M;
#pragma unroll
      for (int c = 0; c < AHEAD; ++c) Mn = fmaxf(Mn, fmaxf(m0[c], m1[c]));
      const float keep = M == -INFINITY ? 0.f : mma::ex2(M - Mn);
      M = Mn;
      L[mp] *= keep;
#pragma unroll
      for (int x = 0; x < C; ++x) v[mp][x] *= keep;
#pragma unroll
      for (int c = 0; c < AHEAD; ++c) {
        const float f0 = m0[c] == -INFINITY ? 0.f : mma::ex2(m0[c] - M), f1 = m1[c] == -INFINITY ? 0.f : mma::ex2(m1[c] - M);
        L[mp] = fmaf(l0[c], f0, fmaf(l1[c], f1, L[mp]));
        const float f = fmaxf(f0, f1);   // O's: the max only grows over a part
#pragma unroll
        for (int x = 0; x < C; ++x) v[mp][x] = fmaf(f == 0.f ? 0.f : o[c][x], f, v[mp][x]);
      }
    }
  }
  __syncthreads();   // λ
  const float lam = s_lam[0] - s_lam[1] + a.lambda_init;
  const float i0 = L[0] > 0.f ? 1.f / L[0] : 0.f, i1 = L[1] > 0.f ? lam / L[1] : 0.f;
  float o[C], ss = 0.f;
#pragma unroll
  for (int x = 0; x < C; ++x) {
    o[x] = fmaf(v[0][x], i0, -(v[1][x] * i1));
    ss = fmaf(o[x], o[x], ss);
  }
  if (a.weight != nullptr) {
    s_ss[warp][lane] = ss;
    __syncthreads();
    ss = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) ss += s_ss[w][lane];
    // a row of zeros (nothing seen, say) stays one, also where eps is 0
    const float f = ss == 0.f ? 0.f : rsqrtf(ss * (1.f / (2 * D)) + a.eps) * (1.f - a.lambda_init);
#pragma unroll
    for (int x = 0; x < C; ++x) o[x] *= f * __ldg(a.weight + warp * C + x);
  }
  if (row >= t.nrow) return;
  const int kvp = a.g.hkv / 2, rep = a.g.rep;
  const int l = (u0 - t.ubase) >> 1, vr = t.row0 + row;
  const int64_t at = (static_cast<int64_t>(t.b0 + l / kvp) * a.q_rows + vr / rep) * (a.g.hq / 2) +
                     static_cast<int64_t>(l % kvp) * rep + vr % rep;
  __half* to = a.out + at * (2 * D) + warp * C;
#pragma unroll
  for (int x = 0; x < C; x += 8)
    *reinterpret_cast<uint4*>(to + x) = make_uint4(pack_half2(o[x], o[x + 1]), pack_half2(o[x + 2], o[x + 3]),
                                                   pack_half2(o[x + 4], o[x + 5]), pack_half2(o[x + 6], o[x + 7]));
}

}  // namespace chunk
}  // namespace kivi
