// rope_qkv.cu — rotary positions with several axes, and the layout the cache
// takes: the query, key and value rows of new tokens as a projection leaves
// them ([B][n][heads][d] with strides) become the attention's q
// [B][n][H_q][d] and the append's k and v [B][H_kv][n][d], fp16, the first
// two turned.
//
// The mathematics.  Pair i of a head's channels is turned by the angle
// p θ_i, p the token's position on the axis that owns the pair and
// θ_i = base^(-i / pairs):
//   (x, y) -> (x cos - y sin, x sin + y cos).
// The angle is reduced in fixed point: F_i = 2^64 θ_i / 2π, rounded as a
// double, comes with the launch; p F_i mod 2^64 is the fraction of a turn
// exactly (integer products wrap by themselves, for negative positions too),
// off by at most |p| 2^-54 turns for F_i's rounding, where an fp32 product
// p θ would lose |p| 2^-24.  Its top 32 bits, as a signed fraction of a half turn, go through
// sincospif.  The products are fp32; one rounding to fp16 at the end.
//
// What bounds it: bytes (read once, written once, nothing computed twice but
// the angles).  A CTA takes a few tokens, its threads make the tokens'
// cos and sin once in shared memory (64 a token, against 48 rows of 128
// channels that use them), then walk the tokens' rows: a thread owns 16
// channels (the eight of both halves, or sixteen adjacent ones), so every
// load and store is 16 bytes, and keeps kBatch rows' loads in flight, the first
// ones while the angles are made.
//
// Measured (48 rows of 128 a token): 32768 tokens in fp32 178 us, 6.8 TB/s (a
// plain copy's rate); 3 x 777 tokens of 24 rows in fp16 6 us; one token of eight
// sequences 2.9 us, a launch's own time.
#include "kivi_internal.cuh"

#include <cuda_bf16.h>

namespace kivi {
namespace {

constexpr int kThreads = 256;
// Rows of a thread in flight, and CTAs an SM: as many rows as leave the registers
// for more CTAs (32768 tokens in fp32: 178 us with two rows and three CTAs, 185
// with three and two; 20000 in bf16: 79 with three and four, 84 with three rows
// and as many CTAs as fit without a bound).
template <class T>
constexpr int kBatch = sizeof(T) == 4 ? 2 : 3;
template <class T, int MODE>
constexpr int kCtas = MODE == 2 ? 2 : sizeof(T) == 4 ? 3 : 4;

// Sixteen channels of a row as 16-byte loads: 0..7 from `a`, 8..15 from `b`.
template <class T>
struct Raw {
  static constexpr int kVec = 8 * sizeof(T) / 16;
  uint4 a[kVec], b[kVec];
  __device__ __forceinline__ void load(const T* pa, const T* pb) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      a[i] = __ldcs(reinterpret_cast<const uint4*>(pa) + i);
      b[i] = __ldcs(reinterpret_cast<const uint4*>(pb) + i);
    }
  }
};
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(float x) { return x; }

template <class T, int N>
__device__ __forceinline__ void widen(const uint4 (&v)[N], float (&f)[8]) {
  T x[8];
  memcpy(x, v, sizeof(x));
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = to_f(x[i]);
}

__device__ __forceinline__ void store8(__half* p, const float (&f)[8]) {
  uint4 v;
  __half2 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
  memcpy(&v, h, 16);
  *reinterpret_cast<uint4*>(p) = v;
}

// MODE 0: pairs (i, i + pairs), pairs a multiple of 8: a thread's two vectors
//         are the two halves of eight pairs (beyond the pairs: two vectors of
//         untouched channels).
// MODE 1: pairs (2i, 2i + 1), a multiple of 8 of them: a thread's two vectors
//         are eight whole pairs.
// MODE 2: pairs (i, i + pairs), any number of pairs: sixteen adjacent channels,
//         whose partners are read one by one.
// MODE 3: pairs (2i, 2i + 1), any number of pairs: as mode 1, but the thread of
//         the last pair leaves the channels past it as they came (turned by
//         nothing, an infinity's neighbour would be NaN).
// Modes 0 and 2 give the same numbers, and so do 1 and 3 where both can.  Mode 2
// reads 16 more elements a thread (20000 tokens in bf16: 227 us, where mode 0
// takes 79), mode 3 tests each pair (3 x 777 tokens of 24 rows in fp16: 6.0 us,
// 5.8 in mode 1; 20000 in bf16 79 in both), so they take only the sections that
// the others cannot.
template <class T, int MODE>
__global__ void __launch_bounds__(kThreads, kCtas<T, MODE>) rope_qkv_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float4 tab[kRopeTokens][4][8];   // token, pair (2 j, 2 j + 1) of an item, item: (cos, sin) twice
  const int b = blockIdx.y, tid = threadIdx.x;
  const int64_t n_b = a.ragged ? a.counts[b] : a.n;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tokens;
  if (t0 >= n_b) return;   // uniform over the block
  const int nt = static_cast<int>(n_b - t0 < a.tokens ? n_b - t0 : a.tokens);
  const int64_t bb = a.b0 + b;

  const int items = a.d / 16, item = tid % items, slots = kThreads / items;
  const int heads = a.hq + 2 * a.hk;
  const int row1 = nt * heads;
  int c0, c1;   // first channels of the thread's two vectors
  bool turned;
  if constexpr (MODE == 0) {
    turned = 8 * item < a.pairs;
    c0 = turned ? 8 * item : 16 * item;
    c1 = turned ? a.pairs + 8 * item : c0 + 8;
  } else {
    c0 = 16 * item;
    c1 = c0 + 8;
    turned = c0 < 2 * a.pairs;
  }
  const int left = a.pairs - 8 * item;   // MODE 3: turned pairs from the thread's first on

  // rows of this CTA, split over gridDim.z when there are few tokens; the first
  // ones' loads go out before the angles are made
  const int lane_row = tid / items, stride = slots * gridDim.z;
  Raw<T> raw[kBatch<T>];
  const T* src[kBatch<T>];
  auto fetch = [&](int r0) {
#pragma unroll
    for (int k = 0; k < kBatch<T>; ++k) {
      const int r = r0 + k * stride;
      if (r >= row1) break;
      const int t = r / heads, h = r % heads;
      const int64_t tt = t0 + t;
      const T* p;
      if (h < a.hq) p = static_cast<const T*>(a.q) + bb * a.qs_b + tt * a.qs_t + static_cast<int64_t>(h) * a.d;
      else if (h < a.hq + a.hk) p = static_cast<const T*>(a.k) + bb * a.ks_b + tt * a.ks_t + static_cast<int64_t>(h - a.hq) * a.d;
      else p = static_cast<const T*>(a.v) + bb * a.vs_b + tt * a.vs_t + static_cast<int64_t>(h - a.hq - a.hk) * a.d;
      src[k] = p;
      raw[k].load(p + c0, p + c1);
    }
  };
  int r0 = blockIdx.z * slots + lane_row;
  fetch(r0);

  for (int x = tid; x < nt * 64; x += kThreads) {
    const int t = x >> 6, p = x & 63;
    float sn = 0.f, cs = 1.f;   // pairs past the last (not read)
    if (p < a.pairs) {
      const int64_t pos = a.positions[(static_cast<int64_t>(a.axis[p]) * a.B + bb) * a.n + t0 + t];
      const uint64_t turn = static_cast<uint64_t>(pos) * a.turn[p];
      sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &sn, &cs);
    }
    reinterpret_cast<float2*>(&tab[t][(p & 7) >> 1][p >> 3])[p & 1] = make_float2(cs, sn);
  }
  __syncthreads();

  for (; r0 < row1; r0 += stride * kBatch<T>, fetch(r0)) {
#pragma unroll
    for (int k = 0; k < kBatch<T>; ++k) {
      const int r = r0 + k * stride;
      if (r >= row1) break;
      const int t = r / heads, h = r % heads;
      const int64_t tt = t0 + t;
      float x[8], y[8];
      widen<T>(raw[k].a, x);
      widen<T>(raw[k].b, y);
      if (turned && h < a.hq + a.hk) {
        if constexpr (MODE == 2) {
          // channel c of a pair: x of pair c below `pairs`, y of pair c - pairs from there on
          float xo[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int c = c0 + j;
            const float own = j < 8 ? x[j & 7] : y[j & 7];
            xo[j] = own;
            if (c < 2 * a.pairs) {
              const int p = c < a.pairs ? c : c - a.pairs;
              const float2 w = reinterpret_cast<const float2*>(&tab[t][(p & 7) >> 1][p >> 3])[p & 1];
              const float other = to_f(src[k][c < a.pairs ? c + a.pairs : p]);
              xo[j] = c < a.pairs ? fmaf(own, w.x, -other * w.y) : fmaf(other, w.y, own * w.x);
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) { x[j] = xo[j]; y[j] = xo[8 + j]; }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 w = tab[t][j][item];   // pairs 8 item + 2 j, + 1
            if constexpr (MODE == 0) {
              const float x0 = x[2 * j], x1 = x[2 * j + 1], y0 = y[2 * j], y1 = y[2 * j + 1];
              x[2 * j] = fmaf(x0, w.x, -y0 * w.y);
              y[2 * j] = fmaf(x0, w.y, y0 * w.x);
              x[2 * j + 1] = fmaf(x1, w.z, -y1 * w.w);
              y[2 * j + 1] = fmaf(x1, w.w, y1 * w.z);
            } else {
              float (&z)[8] = j < 2 ? x : y;
              const int o = 4 * (j & 1);
              const float u0 = z[o], v0 = z[o + 1], u1 = z[o + 2], v1 = z[o + 3];
              if (MODE == 1 || 2 * j < left) {
                z[o] = fmaf(u0, w.x, -v0 * w.y);
                z[o + 1] = fmaf(u0, w.y, v0 * w.x);
              }
              if (MODE == 1 || 2 * j + 1 < left) {
                z[o + 2] = fmaf(u1, w.z, -v1 * w.w);
                z[o + 3] = fmaf(u1, w.w, v1 * w.z);
              }
            }
          }
        }
      }
      __half* dst;
      if (h < a.hq) dst = a.q_out + ((bb * a.n + tt) * a.hq + h) * a.d;
      else if (h < a.hq + a.hk) dst = a.k_out + ((bb * a.hk + (h - a.hq)) * a.n + tt) * a.d;
      else dst = a.v_out + ((bb * a.hk + (h - a.hq - a.hk)) * a.n + tt) * a.d;
      store8(dst + c0, x);
      store8(dst + c1, y);
    }
  }
}

template <class T>
void launch_mode(const RopeArgs& a, int mode, dim3 grid, cudaStream_t s) {
  if (mode == 0) rope_qkv_kernel<T, 0><<<grid, kThreads, 0, s>>>(a);
  else if (mode == 1) rope_qkv_kernel<T, 1><<<grid, kThreads, 0, s>>>(a);
  else if (mode == 2) rope_qkv_kernel<T, 2><<<grid, kThreads, 0, s>>>(a);
  else rope_qkv_kernel<T, 3><<<grid, kThreads, 0, s>>>(a);
}

}  // namespace

cudaError_t launch_rope_qkv(RopeArgs a, int dtype, bool adjacent, int num_sms, const int64_t* n_tokens,
                            cudaStream_t s) {
  const int mode = adjacent ? (a.pairs % 8 == 0 ? 1 : 3) : a.pairs % 8 == 0 ? 0 : 2;
  const int slots = kThreads / (a.d / 16), heads = a.hq + 2 * a.hk;
  // Four tokens a CTA share its start (2400 tokens of 48 rows in bf16 11.4 us,
  // 14.1 with one; 20000 79 and 107); one where four would leave SMs with little
  // (600 tokens 4.7 us, 5.6 with four), and with fewer tokens than SMs a token's
  // rows are split over gridDim.z (8 tokens 3.0 us, 3.3 without).
  const int64_t total = static_cast<int64_t>(a.B) * a.n;
  a.tokens = total >= 8 * static_cast<int64_t>(num_sms) ? kRopeTokens : 1;
  const int passes = (a.tokens * heads + slots - 1) / slots;
  int64_t z = 1;
  if (total < num_sms) z = num_sms / total < passes ? num_sms / total : passes;
  a.ragged = n_tokens != nullptr;
  // the counts of a ragged batch travel with the launch, kRopeCounts at most
  const int32_t most = a.ragged ? kRopeCounts : a.B;
  for (int32_t b0 = 0; b0 < a.B; b0 += most) {
    const int32_t nb = a.B - b0 < most ? a.B - b0 : most;
    a.b0 = b0;
    int64_t longest = a.n;
    if (a.ragged) {
      longest = 0;
      for (int32_t b = 0; b < nb; ++b) {
        a.counts[b] = n_tokens[b0 + b];
        longest = a.counts[b] > longest ? a.counts[b] : longest;
      }
      if (longest == 0) continue;
    }
    if (injected_launch_failure()) return cudaErrorLaunchFailure;
    const dim3 grid(static_cast<unsigned>((longest + a.tokens - 1) / a.tokens), nb, static_cast<unsigned>(z));
    if (dtype == KIVI_F16) launch_mode<__half>(a, mode, grid, s);
    else if (dtype == KIVI_BF16) launch_mode<__nv_bfloat16>(a, mode, grid, s);
    else launch_mode<float>(a, mode, grid, s);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace kivi
