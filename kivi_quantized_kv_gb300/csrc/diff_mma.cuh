// diff_mma.cuh — differential attention over the packed cache on tensor cores.
//
// A head of differential attention has two query rows, two key rows and one
// value row of 2 d channels:
//   o = softmax(q1 K1ᵀ / sqrt(d)) V - λ softmax(q2 K2ᵀ / sqrt(d)) V,
//   λ = exp(λq1 · λk1) - exp(λq2 · λk2) + λ_init,
// then, with a norm, o w (1 - λ_init) / sqrt(mean o² + eps).  In the cache a
// "kv pair" is two neighbouring kv heads: head 2j holds K1 and the first half
// of V, head 2j + 1 K2 and the second half, so a pair's tokens freeze,
// quantize and travel as any other head's.
//
// Both maps need all of V, so the attention of decode_mma.cuh, run head by
// head, would read every value block twice.  Here two warps work on a pair's
// two blocks of the same tokens: warp w makes the scores of map w from block
// w's keys and the products of both maps with block w's values.  The only
// thing they trade is P': each warp writes its map's probabilities, times the
// value steps of either block, into the pair's shared exchange, meets the
// other at a named barrier, and reads the eight columns (four query rows x
// two maps) that its value MMAs take.  The exchange is double buffered by
// chunk, so one barrier a chunk is enough, and the same barrier says that the
// stage before is free for the next copy.  Large blocks leave a pair one stage,
// which is then refilled by halves: a block's keys during its last values, its
// values during the next keys (8 bits, groups of 64, 4 x 32768 tokens: 65 us;
// 70 when the whole stage waits for the pair).
//
// The scores, the code tricks and the value scale are those of decode_mma.cuh
// (codes as exact fp16 subnormals, the folded query in hi and lo columns, the
// running max rescaled lazily).  P' too is split exactly into hi and lo fp16;
// the value MMA's columns being the two maps, the lo parts take a second MMA
// over the same unpacked codes (without them each P' would be off by up to
// 2^-11 of itself).  A warp keeps the running max, sum and Σ p min of its own map
// only, and follows the other map's max through the exchange to keep its
// accumulators in step.
//
// Work split: as decode_mma.cuh, unit = (sequence, kv pair, pass of up to four
// query rows), the units' work positions (frozen groups, then the tail chunks)
// laid end to end and cut into one range per CTA, one CTA per SM with up to
// eight pairs, which take the positions of a range in turn.  At a unit's end the
// pairs' states meet in a tree over shared memory; a unit inside one CTA is
// finished there, else the CTA writes a partial record (a CTA shares at most
// its first and its last unit, so two records a CTA, or one where the launch
// gives each unit whole CTAs), and the last CTA to sign in merges: the difference and the norm need both maps and all 2 d
// channels, so they come last, once.
//
// Bound by: the instructions of a group and their latencies at sixteen warps an
// SM (each code is unpacked once for all query rows and both maps; issue slots
// are half busy); the figures are beside the launch in diff.cu.
#pragma once

#include "decode_mma.cuh"

namespace kivi {
namespace mma {

constexpr int kDiffPairs = 8;   // warp pairs of a CTA, at most

template <int D, int CH>
struct DiffSmem {
  using WS = WarpSmem<D, CH>;
  static constexpr int kState = D / 4 + 3;                    // accumulators of a lane, its two maxima and its sum
  static constexpr int kSlot = 2 * kState * 32 * 4;           // a pair's state
  static constexpr int kXch = 8 * WS::kXch;                   // two buffers of hi and lo P' for either value block
  static constexpr int kRow = 2 * D;                          // floats of an output row
};

__device__ __forceinline__ void pair_sync(int pair) {
  __syncwarp();
  asm volatile("bar.sync %0, 64;" ::"r"(pair + 1) : "memory");
}

template <int D, int BITS, int CH, bool ONE>
__global__ void __launch_bounds__(kDiffPairs * 64, 1) diff_mma_kernel(const __grid_constant__ DiffArgs a) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  using WS = WarpSmem<D, CH>;
  using DS = DiffSmem<D, CH>;
  constexpr int RK = D * BITS / 8;          // key row bytes
  constexpr int QD = D / 4;                 // channels of a lane's quarter
  constexpr int NP = QD / 2;                // channel pairs of a lane's quarter
  constexpr int NKC = D / 16;               // k-chunks over channels
  constexpr int QV = CH * BITS / 4;         // bits of a lane's value quarter per chunk
  constexpr int VW = QV >= 32 ? QV / 32 : 1;
  constexpr int TPL = CH / 8;               // tokens per score lane per chunk
  constexpr int NCT = D / 16;               // channel tiles of a value half
  constexpr int NKT = CH / 16;
  constexpr int REC = 2 * D + 4;            // floats of a partial record
  constexpr bool one = ONE;                 // one stage a pair

  const Geo& g = a.g;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pair = warp >> 1, w = warp & 1;   // w: the warp's map and value half
  const int r = lane >> 2, c = lane & 3;
  const int np = a.np, rep = g.rep, kvp = g.hkv / 2;
  const int64_t P = gridDim.x;
  const int64_t c_start = static_cast<int64_t>(blockIdx.x) * a.W / P;
  const int64_t c_end = static_cast<int64_t>(blockIdx.x + 1) * a.W / P;
  if (c_start >= c_end) return;   // uniform; the host launches no more CTAs than positions
  const int range = static_cast<int>(c_end - c_start);

  // shared memory: stages | q of both maps | slots (also the output rows) | exchange | barriers
  const uint32_t stage_bytes = 2 * static_cast<uint32_t>(a.blk_off);
  uint8_t* stages = smem_raw + static_cast<size_t>(pair) * a.ns * stage_bytes;
  uint8_t* q_all = smem_raw + static_cast<size_t>(np) * a.ns * stage_bytes;
  float* slots = reinterpret_cast<float*>(q_all + 2 * WS::kQ);
  const int n_slots_c = np / 2 > 0 ? np / 2 : 1;
  uint8_t* xch = reinterpret_cast<uint8_t*>(slots) + n_slots_c * DS::kSlot;
  uint64_t* bars = reinterpret_cast<uint64_t*>(xch + np * DS::kXch);
  uint8_t* xw = xch + pair * DS::kXch;
  __shared__ float s_qf[8];                        // query prescale 2^e of each row (map, head)
  __shared__ float s_max[kDiffPairs][2][2][4];     // pair, buffer, map, head: the running max
  __shared__ float s_mn[kDiffPairs][2][4][2];      // pair, map, head, value half: Σ p min
  __shared__ float s_l[8];                         // row sums of the unit being finished
  __shared__ float s_lam;
  __shared__ unsigned s_flag;

  // a barrier a stage, one arrival of either warp; with one stage a pair has
  // one for either warp's keys and one for both blocks' values
  const uint32_t bar0 = smem_addr(bars + pair * (one ? 3 : a.ns)), bar_k = bar0 + 8 * w, bar_v = bar0 + 16;
  if (w == 0 && lane == 0) {
    if (one) {
      mbar_init(bar0, 1);
      mbar_init(bar0 + 8, 1);
      mbar_init(bar_v, 2);
    } else {
      for (int s = 0; s < a.ns; ++s) mbar_init(bar0 + 8 * s, 2);
    }
    fence_mbar_init();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncthreads();
  // the launch before in the stream has completed and its writes are visible
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ------------------------------------------------------------- units
  auto run_of = [&](int u, int k) -> int {
    while (k + 1 < a.n_runs && u >= a.r[k + 1].ubase) ++k;
    return k;
  };
  int k0 = 0;
  while (k0 + 1 < a.n_runs && a.r[k0 + 1].pos0 <= c_start) ++k0;
  const int u_first = a.r[k0].ubase + static_cast<int>((c_start - a.r[k0].pos0) / a.r[k0].uw);
  // first position of unit u_first, relative to the range
  const int rel0 = static_cast<int>(a.r[k0].pos0 + static_cast<int64_t>(u_first - a.r[k0].ubase) * a.r[k0].uw - c_start);
  struct Unit {
    int b, j, pass;
  };
  auto unit_parts_of = [&](int u, const DiffRun& rn) -> Unit {
    Unit x;
    const int l = u - rn.ubase;
    x.pass = l % rn.npass;
    const int bj = l / rn.npass;
    x.b = rn.b0 + bj / kvp;
    x.j = bj % kvp;
    return x;
  };
  // row of map 0's query of row hh (map 1: the next row); half of it is the output's
  auto q_row_of = [&](const Unit& x, int hh) -> int64_t {
    const int v = 4 * x.pass + hh;
    return (static_cast<int64_t>(x.b) * a.q_rows + v / rep) * g.hq + 2 * (static_cast<int64_t>(x.j) * rep + v % rep);
  };

  // ---------------------------------------------------------- producer
  // lane 0 of either warp copies its block of the pair's next item; the walk
  // over the units is the whole warp's, so that a frozen group (nearly every
  // item) costs no branch
  int p_it = 0, p_st = 0, p_u = u_first - 1, p_k = k0, p_end = rel0;
  const uint8_t* p_unit = nullptr;   // own kv head's unit
  bool aborted = false;
  int ab_it = 0;   // the item whose wait ran out; one stage: 2 + ph_v if its values were on their way
  const uint32_t dst0 = smem_addr(stages) + w * a.blk_off;
  // to the pair's next item; false behind the range's end
  auto walk = [&]() -> bool {
    const int rel = pair + p_it * np;
    if (aborted || rel >= range) return false;
    if (rel >= p_end) {
      do {
        ++p_u;
        p_k = run_of(p_u, p_k);
        p_end += a.r[p_k].uw;
      } while (rel >= p_end);
      const Unit x = unit_parts_of(p_u, a.r[p_k]);
      p_unit = a.arena + (static_cast<int64_t>(x.b) * g.hkv + 2 * x.j + w) * g.unit_bytes;
    }
    return true;
  };
  auto block_of = [&](const DiffRun& rn, int pos) -> const uint8_t* {
    uint32_t slot = rn.slot0 + static_cast<uint32_t>(pos);
    if (g.window > 0 && slot >= static_cast<uint32_t>(g.n_slots)) slot -= static_cast<uint32_t>(g.n_slots);
    return p_unit + g.groups + static_cast<int64_t>(slot) * g.block_bytes;
  };
  auto copy_tail = [&](const DiffRun& rn, int pos, uint32_t dst, uint32_t bar) {   // lane 0
    const TailChunk tk = tail_chunk(pos - rn.n_vis, rn.n_sink, rn.n_res, a.k_fresh != nullptr);
    if (tk.n == 0) {
      mbar_arrive_if(true, bar);   // an empty cache: nothing to copy or to attend to
    } else if (tk.fresh) {
      const int64_t row = (p_unit - a.arena) / g.unit_bytes * D;
      bulk_arm(bar, 4 * D);
      bulk_copy(dst, a.k_fresh + row, 2 * D, bar);
      bulk_copy(dst + 16 * D, a.v_fresh + row, 2 * D, bar);
    } else if (tk.sink) {
      const uint32_t bytes = static_cast<uint32_t>(tk.n) * D * 4;
      const uint8_t* sk = p_unit + g.sink_k + static_cast<int64_t>(tk.first) * D * 4;
      const uint8_t* sv = p_unit + g.sink_v + static_cast<int64_t>(tk.first) * D * 4;
      if (dbg_in_region(g, sk, bytes) && dbg_in_region(g, sv, bytes)) {
        bulk_arm(bar, 2 * bytes);
        bulk_copy(dst, sk, bytes, bar);
        bulk_copy(dst + 16 * D, sv, bytes, bar);
      } else {
        mbar_arrive_if(true, bar);
      }
    } else {
      int s0 = rn.rs0 + tk.first;
      if (s0 >= g.R) s0 -= g.R;
      const int n1 = min(tk.n, g.R - s0), n2 = tk.n - n1;   // the ring may wrap
      const uint8_t* rk = p_unit + g.res_k + static_cast<int64_t>(s0) * D * 2;
      const uint8_t* rv = p_unit + g.res_v + static_cast<int64_t>(s0) * D * 2;
      if (dbg_in_region(g, rk, n1 * D * 2) && dbg_in_region(g, rv, n1 * D * 2)) {
        bulk_arm(bar, static_cast<uint32_t>(tk.n) * D * 4);
        bulk_copy(dst, rk, n1 * D * 2, bar);
        bulk_copy(dst + 16 * D, rv, n1 * D * 2, bar);
        if (n2 > 0) {
          bulk_copy(dst + n1 * D * 2, p_unit + g.res_k, n2 * D * 2, bar);
          bulk_copy(dst + 16 * D + n1 * D * 2, p_unit + g.res_v, n2 * D * 2, bar);
        }
      } else {
        mbar_arrive_if(true, bar);
      }
    }
  };
  auto issue = [&]() {   // several stages
    if (!walk()) return;
    const DiffRun& rn = a.r[p_k];
    const int pos = pair + p_it * np - (p_end - rn.uw);
    const uint32_t dst = dst0 + p_st * stage_bytes;
    const uint32_t bar = bar0 + 8 * p_st;
    if (pos < rn.n_vis) {
      const uint8_t* src = block_of(rn, pos);
      if (dbg_in_region(g, src, g.block_bytes))
        bulk_load_if(lane == 0, dst, src, static_cast<uint32_t>(g.block_bytes), bar);
      else mbar_arrive_if(lane == 0, bar);
    } else if (lane == 0) {
      copy_tail(rn, pos, dst, bar);
    }
    __syncwarp();
    ++p_it;
    if (++p_st == a.ns) p_st = 0;
  };
  // One stage: a warp reads its own block's keys alone, and either block's
  // value steps before the pair meets, so the next item's keys come as soon as
  // the last chunk's scores are made and its values as soon as the last
  // products are, without another meeting.  Tail chunks come with the values'
  // turn, both parts on the keys' barrier.
  const uint8_t* p_src = nullptr;   // the block whose keys were asked for and whose values were not
  auto issue_keys = [&]() {
    if (!walk()) return;
    const DiffRun& rn = a.r[p_k];
    const int pos = pair + p_it * np - (p_end - rn.uw);
    if (pos >= rn.n_vis) return;
    p_src = block_of(rn, pos);
    if (dbg_in_region(g, p_src, g.block_bytes)) bulk_load_if(lane == 0, dst0, p_src, static_cast<uint32_t>(g.blk_vq), bar_k);
    else mbar_arrive_if(lane == 0, bar_k);
  };
  auto issue_values = [&]() {
    if (aborted) return;
    if (p_src != nullptr) {
      if (dbg_in_region(g, p_src, g.block_bytes))
        bulk_load_if(lane == 0, dst0 + static_cast<uint32_t>(g.blk_vq), p_src + g.blk_vq,
                     static_cast<uint32_t>(g.block_bytes - g.blk_vq), bar_v);
      else mbar_arrive_if(lane == 0, bar_v);
      p_src = nullptr;
    } else {
      if (!walk()) return;
      const DiffRun& rn = a.r[p_k];
      if (lane == 0) copy_tail(rn, pair + p_it * np - (p_end - rn.uw), dst0, bar_k);
    }
    __syncwarp();
    ++p_it;
  };
  if (one) {
    issue_keys();
    issue_values();
  } else {
    for (int s = 0; s < a.ns; ++s) issue();
  }

  // ---------------------------------------------------------- consumer
  const uint32_t partmask = (r & 1) ? 0xFFFFFFFFu : 0u;
  const int hh_col = r >> 1;   // value column r: query row r >> 1, map r & 1; score column: hi or lo
  float vscl[TPL];             // 2^-k of the lane's tokens' codes (decode_mma.cuh)
#pragma unroll
  for (int i = 0; i < TPL; ++i) {
    const int l = (TPL * r + i) % (CH / 4);
    const int kb = stream_bits<BITS>() ? 0 : (BITS * ((l / 2) % (16 / (stream_bits<BITS>() ? 1 : BITS)))) % 8;
    vscl[i] = __uint_as_float(static_cast<uint32_t>(127 - kb) << 23);
  }
  const float qscale = kLog2e * rsqrtf(static_cast<float>(D));
  constexpr bool kSwap = (RK == 64);
  const int sw = kSwap ? (r & 1) : 0;
  const uint32_t q_off = static_cast<uint32_t>(c * (RK / 4));
  const int ksh = static_cast<int>(8 * (q_off & 3u));
  const uint32_t o_k0 = static_cast<uint32_t>(g.blk_kq) + (TPL * r + sw) * RK + (q_off & ~3u);
  const uint32_t o_k1 = static_cast<uint32_t>(g.blk_kq) + (TPL * r + 1 - sw) * RK + (q_off & ~3u);
  const uint32_t o_ds = static_cast<uint32_t>(g.blk_ks) + c * (D / 2);
  const uint32_t o_vs = static_cast<uint32_t>(g.blk_vs) + TPL * r * 4;
  const uint32_t vrow = static_cast<uint32_t>(g.G) * BITS / 8;
  constexpr bool kStream = stream_bits<BITS>();
  const uint32_t o_vq = kStream ? static_cast<uint32_t>(g.blk_vq) + r * vrow + 4 * ((8 * c * BITS) >> 5)
                                : static_cast<uint32_t>(g.blk_vq) + r * vrow +
                                      (QV >= 32 ? c * (QV / 8) : ((c * QV) / 32) * 4);
  const int vsh = kStream ? (8 * c * BITS) & 31 : (QV >= 32 ? 0 : ((c * QV) % 32) / 2);
  const uint32_t q_s = smem_addr(q_all + w * WS::kQ + hh_col * WS::kQRow + c * WS::kQS);

  float oacc[NCT][4];   // channels 16 ct + r (0, 1) and + 8 (2, 3) of the value half; head c, map 0 (0, 2) and 1 (1, 3)
  float res_m, res_l, mn_a, mn_b;   // own map, head c: max, sum, Σ p min of either value half
  float par_m;                      // the other map's max the accumulators are at
  float f_a, f_b;                   // value scales 2^F of the unit (0: not chosen)
  bool o_real;
  auto scale_map = [&](int m, float f) {
    const float f0 = m ? 1.f : f, f1 = m ? f : 1.f;
#pragma unroll
    for (int i = 0; i < NCT; ++i) { oacc[i][0] *= f0; oacc[i][1] *= f1; oacc[i][2] *= f0; oacc[i][3] *= f1; }
  };
  // the other map's max moved: bring its columns of the accumulators along
  auto follow = [&](int buf) {
    const float m = s_max[pair][buf][1 - w][c];
    if (__any_sync(0xffffffffu, m != par_m)) {
      scale_map(1 - w, par_m == -INFINITY ? 0.f : ex2(par_m - m));   // 1 where it did not
      par_m = m;
    }
  };
  auto raise = [&](float corr) {   // own map's reference moved by log2(1 / corr)
    res_l *= corr;
    mn_a *= corr;
    mn_b *= corr;
    scale_map(w, corr);
  };

  int it = 0, st = 0, buf = 0;
  uint32_t ph = 0, ph_v = 0;   // ph_v: of the values' barrier (one stage)
  auto look = [&](uint32_t bar, uint32_t parity, bool frozen) {
    if (!aborted && !__all_sync(0xffffffffu, mbar_wait(bar, parity, a.wait_ns))) {
      // give up: go on through the barriers with whatever the stage holds
      // (the outputs are invalid and say so), without waiting or copying
      aborted = true;
      ab_it = !one ? it : frozen ? 2 + static_cast<int>(ph_v) : 0;
      if (lane == 0) atomicOr(a.error, kErrCopy);
    }
  };
  bool have_lam = false;
  int k = k0, u_rel = rel0;
  for (int u = u_first; u_rel < range; ++u) {
    k = run_of(u, k);
    const DiffRun& rn = a.r[k];
    const Unit un = unit_parts_of(u, rn);
    const int nh = min(4, rn.nq * rep - 4 * un.pass);
    const int seg_end = min(range, u_rel + rn.uw);
    const bool masked = rn.nq > 1 || g.window > 0;
    const int64_t hi = rn.q_pos0 + (4 * un.pass + c) / rep;   // the last position head c sees
    const int64_t lo = g.window > 0 ? hi + 1 - g.window : INT64_MIN;
    res_m = par_m = -INFINITY;
    res_l = mn_a = mn_b = f_a = f_b = 0.f;
    o_real = false;
#pragma unroll
    for (int i = 0; i < NCT; ++i) oacc[i][0] = oacc[i][1] = oacc[i][2] = oacc[i][3] = 0.f;

    // the unit's query rows, both maps: quarter rows padded, rows past nh zero,
    // a row whose largest |q_c| exceeds 1 scaled by 2^-e (decode_mma.cuh)
    for (int kk = tid; kk < D; kk += static_cast<int>(blockDim.x)) {   // 8 rows of D / 8 16-byte parts
      const int m = kk / (D / 2), hh = (kk / (D / 8)) & 3, idx = kk % (D / 8);
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (hh < nh) v = *reinterpret_cast<const uint4*>(a.q + (q_row_of(un, hh) + m) * D + idx * 8);
      uint32_t mb = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                             __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
      mb = max(mb & 0xFFFFu, mb >> 16);
#pragma unroll
      for (int o = 1; o < D / 8; o <<= 1) mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, o));
      const int e = mb > 0x3C00u ? static_cast<int>(mb >> 10) - 14 : 0;
      if constexpr (kDebugChecks) {
        if (mb >= 0x7C00u) atomicOr(a.error, kErrNonFinite);
      }
      if (e > 0) {
        const uint32_t h = e <= 14 ? static_cast<uint32_t>(15 - e) << 10 : 1u << (24 - e);
        const uint32_t s2 = h | (h << 16);
        v.x = hmul2_u(v.x, s2); v.y = hmul2_u(v.y, s2); v.z = hmul2_u(v.z, s2); v.w = hmul2_u(v.w, s2);
      }
      *reinterpret_cast<uint4*>(q_all + m * WS::kQ + hh * WS::kQRow + (idx / (QD / 8)) * WS::kQS +
                                (idx % (QD / 8)) * 16) = make_uint4(v.x, v.z, v.y, v.w);
      if (idx == 0) s_qf[4 * m + hh] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    }
    __syncthreads();
    const float qf = s_qf[4 * w + c];

    for (; pair + it * np < seg_end; ++it) {
      const int pos = pair + it * np - u_rel;
      look(one ? bar_k : bar0 + 8 * st, ph, pos < rn.n_vis);
      const uint32_t stage = smem_addr(stages) + st * stage_bytes;
      const uint32_t blk = stage + w * a.blk_off;
      if (pos < rn.n_vis) {
        // ---------------------------------------------------- a frozen group
        const int64_t a_grp = g.S + (rn.g_first + pos) * g.G;
        uint32_t bq[NP], q2[NP];
#pragma unroll
        for (int i = 0; i < NP / 4; ++i) {
          const uint4 v = lds128(q_s + 16 * i);
          q2[4 * i] = v.x; q2[4 * i + 1] = v.z; q2[4 * i + 2] = v.y; q2[4 * i + 3] = v.w;
        }
#pragma unroll
        for (int i = 0; i < NP / 4; ++i) {
          const uint4 dv = lds128(blk + o_ds + 16 * i);
          const uint32_t dw[4] = {dv.x, dv.y, dv.z, dv.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t h2 = hmul2_u(q2[4 * i + j], dw[j]);
            bq[4 * i + j] = hfma2_u(q2[4 * i + j], dw[j], (h2 ^ 0x80008000u) & partmask);
          }
        }
        float cst_a[4] = {0.f, 0.f, 0.f, 0.f}, cst_b[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NP / 4; ++i) {
          const uint4 mv = lds128(blk + o_ds + 2 * D + 16 * i);
          mma16816(cst_a, mv.x, mv.y, mv.z, mv.w, q2[4 * i], q2[4 * i + 2]);
          mma16816(cst_b, mv.x, mv.y, mv.z, mv.w, q2[4 * i + 1], q2[4 * i + 3]);
        }
        const float cst_h = (cst_a[0] + cst_b[2]) * (qscale * qf);
        const float scs = qscale * kTwo24 * qf;

        for (int s0 = 0; s0 < g.G; s0 += CH) {
          float sv[TPL];
          chunk_scores<D, BITS, CH>(bq, blk + o_k0 + s0 * RK, blk + o_k1 + s0 * RK, scs, cst_h, sw, ksh, sv);
          if (masked) {
#pragma unroll
            for (int i = 0; i < TPL; ++i) {
              const int64_t t = a_grp + s0 + TPL * r + i;
              if (t < lo || t > hi) sv[i] = -INFINITY;
            }
          }
          float mx = sv[0];
#pragma unroll
          for (int i = 1; i < TPL; ++i) mx = fmaxf(mx, sv[i]);
          if (__any_sync(0xffffffffu, mx > res_m + kRescale)) {
            mx = warp_max_rows(mx);
            float corr = 1.f;
            if (mx > res_m + kRescale) {   // uniform over the lanes of head c
              corr = (res_m == -INFINITY) ? 0.f : ex2(res_m - mx);
              res_m = mx;
            }
            raise(corr);
          }
          const float mref = (res_m == -INFINITY) ? 0.f : res_m;
          if (one) {
            if (s0 + CH >= g.G) {
              __syncwarp();
              issue_keys();
            }
            if (s0 == 0) look(bar_v, ph_v, true);
          }
          float da[2 * TPL], db[2 * TPL];   // (Δ, min) of the lane's tokens in either block
#pragma unroll
          for (int hb = 0; hb < 2; ++hb) {
            const uint32_t addr = stage + hb * a.blk_off + o_vs + 4 * s0;
            float (&dm)[2 * TPL] = hb ? db : da;
            if constexpr (TPL == 4) {
              const uint4 x = lds128(addr);
              const uint32_t xv[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) { const float2 f = h2f(xv[i]); dm[2 * i] = f.x; dm[2 * i + 1] = f.y; }
            } else {
              const uint2 x = lds64(addr);
              const float2 f0 = h2f(x.x), f1 = h2f(x.y);
              dm[0] = f0.x; dm[1] = f0.y; dm[2] = f1.x; dm[3] = f1.y;
            }
          }
          if (f_a == 0.f) {   // the pair's first frozen chunk of the unit: both warps choose alike
            float xa = da[0], xb = db[0];
#pragma unroll
            for (int i = 1; i < TPL; ++i) { xa = fmaxf(xa, da[2 * i]); xb = fmaxf(xb, db[2 * i]); }
            xa = warp_max_rows(xa);
            xb = warp_max_rows(xb);
            int ea = 0, eb = 0;
            frexpf(xa, &ea);
            frexpf(xb, &eb);
            f_a = __uint_as_float(static_cast<uint32_t>(127 + (ea < 6 ? 6 - ea : 0)) << 23);
            f_b = __uint_as_float(static_cast<uint32_t>(127 + (eb < 6 ? 6 - eb : 0)) << 23);
          }
          float pa[TPL], pb[TPL], pm = 0.f;
#pragma unroll
          for (int i = 0; i < TPL; ++i) {
            const float p = ex2(sv[i] - mref);
            res_l += p;
            mn_a = fmaf(p, da[2 * i + 1], mn_a);
            mn_b = fmaf(p, db[2 * i + 1], mn_b);
            const float ps = p * vscl[i];
            pa[i] = ps * (da[2 * i] * f_a);
            pb[i] = ps * (db[2 * i] * f_b);
            pm = fmaxf(pm, fmaxf(pa[i], pb[i]));
          }
          // fp16 range of P': the head's reference raised by a power of two
          // where it would be passed (decode_mma.cuh)
          if (__any_sync(0xffffffffu, pm > 65504.f)) {
            pm = warp_max_rows(pm);
            int ex = 0;
            frexpf(pm, &ex);
            const int E = pm > 65504.f ? ex - 15 : 0;
            const float corr = __uint_as_float(static_cast<uint32_t>(127 - E) << 23);
            res_m += static_cast<float>(E);
            raise(corr);
#pragma unroll
            for (int i = 0; i < TPL; ++i) { pa[i] *= corr; pb[i] *= corr; }
          }
          // hi and lo halves of P' for either block's value warp
          const uint32_t xo = xch_off<CH>(c, w, TPL * r);
#pragma unroll
          for (int hb = 0; hb < 2; ++hb) {
            const float (&pp)[TPL] = hb ? pb : pa;
            uint32_t hw[TPL / 2], lw[TPL / 2];
#pragma unroll
            for (int i = 0; i < TPL / 2; ++i) {
              hw[i] = rope_split(pp[2 * i], pp[2 * i + 1], false);
              lw[i] = rope_split(pp[2 * i], pp[2 * i + 1], true);
            }
            uint8_t* x = xw + (4 * buf + 2 * hb) * WS::kXch + xo;
            if constexpr (TPL == 4) {
              *reinterpret_cast<uint2*>(x) = make_uint2(hw[0], hw[1]);
              *reinterpret_cast<uint2*>(x + WS::kXch) = make_uint2(lw[0], lw[1]);
            } else {
              *reinterpret_cast<uint32_t*>(x) = hw[0];
              *reinterpret_cast<uint32_t*>(x + WS::kXch) = lw[0];
            }
          }
          if (r == 0) s_max[pair][buf][w][c] = res_m;
          pair_sync(pair);
          if (s0 == 0 && it > 0 && !one) issue();   // the stage before is free
          follow(buf);
          // Oᵀ += Vᵀ P' of the warp's value half
          uint32_t bp[2][NKT][2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint8_t* xr = xw + (4 * buf + 2 * w + e) * WS::kXch;
            if constexpr (NKT == 2) {
              const uint4 x = *reinterpret_cast<const uint4*>(xr + xch_off<CH>(hh_col, r & 1, 8 * c));
              bp[e][0][0] = x.x; bp[e][0][1] = x.y; bp[e][1][0] = x.z; bp[e][1][1] = x.w;
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(xr + xch_off<CH>(hh_col, r & 1, 4 * c));
              bp[e][0][0] = x.x; bp[e][0][1] = x.y;
            }
          }
          buf ^= 1;
          const uint32_t vq = blk + o_vq + s0 * BITS / 8;
#pragma unroll
          for (int ct = 0; ct < NCT; ++ct) {
            uint32_t v0[kStream ? 2 : VW], v1[kStream ? 2 : VW];
            const uint32_t rowa = vq + ct * 16 * vrow, rowb = rowa + 8 * vrow;
            if constexpr (kStream) {   // the lane's 8 codes: a 64-bit window from three words
              const uint32_t a0 = lds32(rowa), a1 = lds32(rowa + 4), a2 = lds32(rowa + 8);
              const uint32_t b0 = lds32(rowb), b1 = lds32(rowb + 4), b2 = lds32(rowb + 8);
              v0[0] = __funnelshift_r(a0, a1, vsh); v0[1] = __funnelshift_r(a1, a2, vsh);
              v1[0] = __funnelshift_r(b0, b1, vsh); v1[1] = __funnelshift_r(b1, b2, vsh);
            } else if constexpr (VW == 2) {
              const uint2 x = lds64(rowa), y = lds64(rowb);
              v0[0] = x.x; v0[1] = x.y; v1[0] = y.x; v1[1] = y.y;
            } else if constexpr (QV >= 32) {
              v0[0] = lds32(rowa);
              v1[0] = lds32(rowb);
            } else {
              v0[0] = lds32(rowa) >> vsh;
              v1[0] = lds32(rowb) >> vsh;
            }
#pragma unroll
            for (int kc = 0; kc < NKT; ++kc) {
              const uint32_t a0 = code_pair<BITS>(v0, 2 * kc), a1 = code_pair<BITS>(v1, 2 * kc);
              const uint32_t a2 = code_pair<BITS>(v0, 2 * kc + 1), a3 = code_pair<BITS>(v1, 2 * kc + 1);
              mma16816(oacc[ct], a0, a1, a2, a3, bp[0][kc][0], bp[0][kc][1]);
              mma16816(oacc[ct], a0, a1, a2, a3, bp[1][kc][0], bp[1][kc][1]);
            }
          }
        }
        if (one) {
          __syncwarp();
          issue_values();
          ph_v ^= 1u;
        }
      } else {
        // ------------------------------------------------------ a tail chunk
        const TailChunk tk = tail_chunk(pos - rn.n_vis, rn.n_sink, rn.n_res, a.k_fresh != nullptr);
        const uint8_t* kst = stages + st * stage_bytes + w * a.blk_off;
        const uint8_t* vst = kst + 16 * D;
        if (!o_real) {   // from here on the accumulators hold real-scale values
          const float f = w ? f_b : f_a;
          const float to_real = f == 0.f ? kTwo24 : kTwo24 / f;
          scale_map(0, to_real);
          scale_map(1, to_real);
          o_real = true;
        }
        uint32_t ka[NP];   // keys of token r (zero past the chunk), pair order of quarter c
        if (r < tk.n) {
          if (tk.sink) {
            const float* kr = reinterpret_cast<const float*>(kst) + r * D + c * QD;
#pragma unroll
            for (int i = 0; i < NP / 2; ++i) {
              const float4 f = reinterpret_cast<const float4*>(kr)[i];
              ka[2 * i] = pack_half2(f.x, f.y);
              ka[2 * i + 1] = pack_half2(f.z, f.w);
            }
          } else {
            const uint8_t* kr = kst + (r * D + c * QD) * 2;
#pragma unroll
            for (int i = 0; i < NP / 4; ++i) {
              const uint4 v = reinterpret_cast<const uint4*>(kr)[i];
              ka[4 * i] = v.x; ka[4 * i + 1] = v.y; ka[4 * i + 2] = v.z; ka[4 * i + 3] = v.w;
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < NP; ++i) ka[i] = 0u;
        }
        float acc0[4] = {0.f, 0.f, 0.f, 0.f}, acc1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NP / 4; ++i) {
          const uint4 v = lds128(q_s + 16 * i);   // pairs 4i, 4i + 2, 4i + 1, 4i + 3
          mma16816(acc0, ka[4 * i], 0u, ka[4 * i + 1], 0u, v.x, v.z);
          mma16816(acc1, ka[4 * i + 2], 0u, ka[4 * i + 3], 0u, v.y, v.w);
        }
        float s = (r < tk.n) ? (acc0[0] + acc1[0]) * (qscale * qf) : -INFINITY;
        if (rn.nq > 1) {   // the ring and the sinks lie inside any window of the newest query
          const int64_t t = tk.fresh ? rn.fresh_pos
                          : tk.sink  ? static_cast<int64_t>(tk.first) + r
                                     : g.S + (rn.g_first + rn.n_vis) * g.G + tk.first + r;
          if (t > hi || (t >= g.S && t < lo)) s = -INFINITY;
        }
        const float mx = warp_max_rows(s);
        float corr = 1.f;
        if (mx > res_m + kRescale) {
          corr = (res_m == -INFINITY) ? 0.f : ex2(res_m - mx);
          res_m = mx;
        }
        if (__any_sync(0xffffffffu, corr != 1.f)) raise(corr);
        const float p = s == -INFINITY ? 0.f : ex2(s - res_m);
        res_l += p;
        {
          const float h = __uint_as_float(__float_as_uint(p) & 0xFFFFE000u);
          uint8_t* x = xw + 4 * buf * WS::kXch + xch_off<CH>(c, w, r);
          *reinterpret_cast<__half*>(x) = __float2half_rn(h);
          *reinterpret_cast<__half*>(x + WS::kXch) = __float2half_rn(p - h);
        }
        if (r == 0) s_max[pair][buf][w][c] = res_m;
        pair_sync(pair);
        if (it > 0 && !one) issue();
        follow(buf);
        const uint8_t* xr = xw + 4 * buf * WS::kXch + xch_off<CH>(hh_col, r & 1, 2 * c);
        const uint32_t tmask = (2 * c < tk.n ? 0x0000FFFFu : 0u) | (2 * c + 1 < tk.n ? 0xFFFF0000u : 0u);
        const uint32_t b0 = *reinterpret_cast<const uint32_t*>(xr) & tmask;
        const uint32_t b1 = *reinterpret_cast<const uint32_t*>(xr + WS::kXch) & tmask;   // lo: the upper k half
        buf ^= 1;
        if (tk.sink) {
          const float* vr = reinterpret_cast<const float*>(vst);
#pragma unroll
          for (int ct = 0; ct < NCT; ++ct) {
            uint32_t a0 = 0u, a1 = 0u;
            if (2 * c < tk.n) {
              const float* v0r = vr + (2 * c) * D + 16 * ct + r;
              const float x0 = v0r[0], y0 = (2 * c + 1 < tk.n) ? v0r[D] : 0.f;
              const float x1 = v0r[8], y1 = (2 * c + 1 < tk.n) ? v0r[D + 8] : 0.f;
              a0 = pack_half2(x0, y0);
              a1 = pack_half2(x1, y1);
            }
            mma16816(oacc[ct], a0, a1, a0, a1, b0, b1);
          }
        } else {
          const uint32_t vbase = smem_addr(vst) + (lane & 7) * D * 2 + ((lane >> 3) & 1) * 16;
#pragma unroll
          for (int ct = 0; ct < NCT; ++ct) {
            uint32_t a0, a1;
            ldsm_x2_trans(a0, a1, vbase + 32 * ct);
            a0 &= tmask;
            a1 &= tmask;
            mma16816(oacc[ct], a0, a1, a0, a1, b0, b1);
          }
        }
        if (tk.fresh && un.pass == 0) {
          // fused step: the token into its sink slot (widened to fp32) or its
          // ring slot; nothing this launch reads lives there
          uint8_t* base = const_cast<uint8_t*>(a.arena) +
                          (static_cast<int64_t>(un.b) * g.hkv + 2 * un.j + w) * g.unit_bytes;
          const int64_t fp = rn.fresh_pos;
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            for (int e = 4 * lane; e < D; e += 128) {
              const uint2 x = *reinterpret_cast<const uint2*>(kst + part * 16 * D + 2 * e);
              dbg_check_finite(g, make_uint4(x.x, x.y, 0u, 0u));
              if (fp < g.S) {
                const float2 f0 = h2f(x.x), f1 = h2f(x.y);
                uint8_t* to = base + (part ? g.sink_v : g.sink_k) + (fp * D + e) * 4;
                if (dbg_in_region(g, to, 16)) *reinterpret_cast<float4*>(to) = make_float4(f0.x, f0.y, f1.x, f1.y);
              } else {
                uint8_t* to = base + (part ? g.res_v : g.res_k) + ((fp - g.S) % g.R * D + e) * 2;
                if (dbg_in_region(g, to, 8)) *reinterpret_cast<uint2*>(to) = x;
              }
            }
          }
        }
        if (one) {
          __syncwarp();
          issue_keys();
          issue_values();
        }
      }
      if (one || ++st == a.ns) { st = 0; ph ^= 1u; }
    }

    // ------------------------------------------------------ the unit's end
    res_l = warp_sum_rows(res_l);
    mn_a = warp_sum_rows(mn_a);
    mn_b = warp_sum_rows(mn_b);
    if (r == 0) {
      s_mn[pair][w][c][0] = mn_a;
      s_mn[pair][w][c][1] = mn_b;
    }
    pair_sync(pair);
    {
      const float m0 = s_mn[pair][0][c][w], m1 = s_mn[pair][1][c][w];
      const float f = w ? f_b : f_a;
      const float osc = (o_real ? 1.f : kTwo24) / ((o_real || f == 0.f) ? 1.f : f);
#pragma unroll
      for (int i = 0; i < NCT; ++i) {
        oacc[i][0] = fmaf(oacc[i][0], osc, m0);
        oacc[i][1] = fmaf(oacc[i][1], osc, m1);
        oacc[i][2] = fmaf(oacc[i][2], osc, m0);
        oacc[i][3] = fmaf(oacc[i][3], osc, m1);
      }
    }
    // the pairs' states, halved in number until pair 0 has all
    for (int active = np; active > 1;) {
      const int half = (active + 1) / 2;
      if (pair >= half && pair < active) {
        float* so = slots + (pair - half) * (DS::kSlot / 4) + w * DS::kState * 32 + lane;
#pragma unroll
        for (int i = 0; i < NCT; ++i) {
#pragma unroll
          for (int j = 0; j < 4; ++j) so[(4 * i + j) * 32] = oacc[i][j];
        }
        so[4 * NCT * 32] = res_m;
        so[(4 * NCT + 1) * 32] = par_m;
        so[(4 * NCT + 2) * 32] = res_l;
      }
      __syncthreads();
      if (pair < active - half) {
        const float* so = slots + pair * (DS::kSlot / 4) + w * DS::kState * 32 + lane;
        const float m2 = so[4 * NCT * 32], q2 = so[(4 * NCT + 1) * 32], l2 = so[(4 * NCT + 2) * 32];
        const float mo = fmaxf(res_m, m2), mp = fmaxf(par_m, q2);
        const float fo = res_m == -INFINITY ? 0.f : ex2(res_m - mo), fo2 = m2 == -INFINITY ? 0.f : ex2(m2 - mo);
        const float fp = par_m == -INFINITY ? 0.f : ex2(par_m - mp), fp2 = q2 == -INFINITY ? 0.f : ex2(q2 - mp);
        res_l = fmaf(l2, fo2, res_l * fo);
        const float f0 = w ? fp : fo, f1 = w ? fo : fp, g0 = w ? fp2 : fo2, g1 = w ? fo2 : fp2;
#pragma unroll
        for (int i = 0; i < NCT; ++i) {
          oacc[i][0] = fmaf(so[(4 * i) * 32], g0, oacc[i][0] * f0);
          oacc[i][1] = fmaf(so[(4 * i + 1) * 32], g1, oacc[i][1] * f1);
          oacc[i][2] = fmaf(so[(4 * i + 2) * 32], g0, oacc[i][2] * f0);
          oacc[i][3] = fmaf(so[(4 * i + 3) * 32], g1, oacc[i][3] * f1);
        }
        res_m = mo;
        par_m = mp;
      }
      active = half;
      __syncthreads();
    }
    // λ, by a warp that the tree has left idle (its loads would hold up the
    // first unit if they came first)
    if (!have_lam && warp == (np > 1 ? 2 : 1)) {
      float d1 = 0.f, d2 = 0.f;
      for (int i = lane; i < D; i += 32) {
        d1 = fmaf(a.lambdas[i], a.lambdas[D + i], d1);
        d2 = fmaf(a.lambdas[2 * D + i], a.lambdas[3 * D + i], d2);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        d1 += __shfl_xor_sync(0xffffffffu, d1, o);
        d2 += __shfl_xor_sync(0xffffffffu, d2, o);
      }
      if (lane == 0) s_lam = expf(d1) - expf(d2) + a.lambda_init;
    }
    have_lam = true;
    const int64_t u_base = c_start + u_rel;
    const int first = owner_of(u_base, a.W, P);
    const int total = owner_of(u_base + rn.uw - 1, a.W, P) - first + 1;
    float* rows = slots;   // [8][2 D]: unnormalised outputs, row 4 map + head
    if (pair == 0 && c < nh) {
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        float* to = rows + (4 * m + c) * DS::kRow;
        if (total > 1) {
          const int slot = a.slots * static_cast<int>(blockIdx.x) + (u == u_first ? 0 : 1);
          to = a.partials + (static_cast<int64_t>(slot) * a.rows + (a.rows / 2) * m + c) * REC;
          if (m == w && r == 0) { to[2 * D] = res_m; to[2 * D + 1] = res_l; }
        } else if (m == w && r == 0) {
          s_l[4 * m + c] = res_l;
        }
#pragma unroll
        for (int i = 0; i < NCT; ++i) {
          to[w * D + 16 * i + r] = oacc[i][m];
          to[w * D + 16 * i + r + 8] = oacc[i][m + 2];
        }
      }
    }
    bool finish = true;
    if (total > 1) {
      __threadfence();
      __syncthreads();
      if (tid == 0) s_flag = (atomicAdd(a.counters + u, 1u) == static_cast<unsigned>(total - 1)) ? 1u : 0u;
      __syncthreads();
      finish = s_flag != 0u;
      if (finish) {
        __threadfence();
        // Σ over the CTAs: record s is CTA first + s's, its second one when the
        // unit is not that CTA's first
        const int late = (static_cast<int64_t>(first) * a.W / P) < u_base ? 1 : 0;
        for (int i = tid; i < 2 * nh * D; i += static_cast<int>(blockDim.x)) {
          const int row = i / D, ch = 2 * (i % D);
          const int m = row / nh, hh = row % nh;
          const float* base = a.partials + (static_cast<int64_t>(a.slots * first) * a.rows + (a.rows / 2) * m + hh) * REC;
          const int64_t unit = static_cast<int64_t>(a.rows) * REC, step = a.slots * unit;
          float M = -INFINITY, L = 0.f;
          float2 O = make_float2(0.f, 0.f);
          for (int s0 = 0; s0 < total; s0 += kMergeBatch) {
            float2 ml[kMergeBatch], o[kMergeBatch];
#pragma unroll
            for (int s = 0; s < kMergeBatch; ++s) {
              ml[s] = make_float2(-INFINITY, 0.f);
              o[s] = make_float2(0.f, 0.f);
              if (s0 + s < total) {
                const float* ps = base + (s0 + s) * step + ((s0 + s == 0 && late) ? unit : 0);
                ml[s] = __ldcg(reinterpret_cast<const float2*>(ps + 2 * D));
                o[s] = __ldcg(reinterpret_cast<const float2*>(ps + ch));
              }
            }
            float mb = M;
#pragma unroll
            for (int s = 0; s < kMergeBatch; ++s) mb = fmaxf(mb, ml[s].x);
            if (mb == -INFINITY) continue;
            const float sc = M == -INFINITY ? 0.f : ex2(M - mb);
            O.x *= sc;
            O.y *= sc;
            L *= sc;
            M = mb;
#pragma unroll
            for (int s = 0; s < kMergeBatch; ++s) {
              const float f = ml[s].x == -INFINITY ? 0.f : ex2(ml[s].x - M);
              O.x = fmaf(o[s].x, f, O.x);
              O.y = fmaf(o[s].y, f, O.y);
              L = fmaf(ml[s].y, f, L);
            }
          }
          *reinterpret_cast<float2*>(rows + (4 * m + hh) * DS::kRow + ch) = O;
          if (ch == 0) s_l[4 * m + hh] = L;
        }
        if (tid == 0) a.counters[u] = 0u;
      }
    }
    __syncthreads();
    // row hh: the difference of the maps, its norm, the output
    for (int hh = warp; finish && hh < nh; hh += 2 * np) {
      const float l1 = s_l[hh], l2 = s_l[4 + hh];
      const float i1 = l1 > 0.f ? 1.f / l1 : 0.f, i2 = l2 > 0.f ? s_lam / l2 : 0.f;
      float2 o[D / 32];
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int ch = 2 * (lane + 32 * i);
        const float2 x = *reinterpret_cast<const float2*>(rows + hh * DS::kRow + ch);
        const float2 y = *reinterpret_cast<const float2*>(rows + (4 + hh) * DS::kRow + ch);
        o[i] = make_float2(fmaf(x.x, i1, -(y.x * i2)), fmaf(x.y, i1, -(y.y * i2)));
        ss = fmaf(o[i].x, o[i].x, fmaf(o[i].y, o[i].y, ss));
      }
      if (a.weight != nullptr) {
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, x);
        // a row of zeros (nothing seen, say) stays one, also where eps is 0
        const float f = ss == 0.f ? 0.f : rsqrtf(ss * (1.f / (2 * D)) + a.eps) * (1.f - a.lambda_init);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const float2 wt = __ldg(reinterpret_cast<const float2*>(a.weight) + lane + 32 * i);
          o[i].x *= f * wt.x;
          o[i].y *= f * wt.y;
        }
      }
      __half* to = a.out + (q_row_of(un, hh) / 2) * (2 * D);
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
        reinterpret_cast<__half2*>(to)[lane + 32 * i] = __floats2half2_rn(o[i].x, o[i].y);
    }
    u_rel += rn.uw;
  }

  // after a wait that ran out: the copies in flight land (bounded) before the
  // shared memory is given back
  if (aborted) {
    if (one) {
      mbar_wait(bar_k, static_cast<uint32_t>(p_it - (p_src != nullptr ? 0 : 1)) & 1u, kWaitNs);
      if (ab_it & 2) mbar_wait(bar_v, ab_it & 1, kWaitNs);
    } else {
      for (; ab_it < p_it; ++ab_it)
        mbar_wait(bar0 + 8 * (ab_it % a.ns), static_cast<uint32_t>(ab_it / a.ns) & 1u, kWaitNs);
    }
  }
}

}  // namespace mma
}  // namespace kivi
