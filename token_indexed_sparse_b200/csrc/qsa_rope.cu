// Rotary positions, their gradient, and the write of new K/V rows into a paged
// cache with the rotation on the way.
//
// Pair i of a head turns by the angle pos * f_i and grows by m:
//   y1 = m (x1 cos a - x2 sin a),  y2 = m (x1 sin a + x2 cos a),
// pairs being dims (2i, 2i + 1) (interleaved) or (i, i + R / 2) (half layout),
// i < R / 2; dims R and up pass unchanged.  The map is m times a rotation, so
// the gradient is m times the opposite rotation: the same kernel with -sin.
//
// Angles: pos * f_i reaches 1e6 radians, where 32 bits keep 0.06 of a radian.
// The turn count f_i / (2 pi) mod 1 is taken in two 64-bit floating-point parts (one
// alone leaves 2^-25 of a turn at position 2^31 for f = 1, and more for faster pairs)
// as a fraction of 2^64, right to a unit; times the integer position, modulo 2^64, it
// is the angle's fraction of a turn with no range reduction, right to 2^-33.  Its top
// 32 bits as half-turns, rounded to FP32, go to sincospi: 2^-26 of a turn, 1e-7 of a
// radian, is what that leaves.
//
// Bound by memory: every 16-byte piece is read and written once, past the caches
// (evict-first; with default stores the append of 16 k tokens took 94 us, not 91).
// A block takes a few tokens, as many as give each thread its units (four, two in
// the append; fewer leave too little in flight: 12 + 1 heads of 16384 tokens took
// 47 us with two tokens a block, 42 with four).  Each thread first issues the loads
// of its units, then the block computes the cosines and sines of its (token, pair)s
// into shared memory for all heads, then each thread rotates its units in FP32 and
// rounds once.  A unit is two 16-byte pieces of one head that hold eight whole pairs
// in either layout.  26 heads of 32768 tokens: 139 us, 6.3 TB/s (133 us at the rate
// of a plain copy).
#include "qsa_cache.cuh"
#include "qsa_device.cuh"
#include "qsa_internal.h"

namespace qsa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxTok = 8;                       // tokens per block at most
constexpr int kUnits = kHeadDim / 16;            // two-piece units per head
constexpr int kAhead = 4, kAppendAhead = 2;      // units whose loads a thread holds
constexpr int kCsUnit = 9;                       // a unit's eight (cos, sin) and one of padding: no bank conflicts
constexpr double kTurnHi = 0x1.45f306dc9c883p-3, kTurnLo = -0x1.6b01ec5417056p-57;  // 1 / (2 pi), in two parts

// Fraction of a turn of one position step, in units of 2^-64 modulo 2^64: each part's distance to the
// nearest whole number (exact), rounded to a unit.
__device__ __forceinline__ unsigned long long turn_step(double f) {
  const double hi = __dmul_rn(f, kTurnHi), lo = __fma_rn(f, kTurnLo, __fma_rn(f, kTurnHi, -hi));
  return static_cast<unsigned long long>(__double2ll_rn((hi - rint(hi)) * 18446744073709551616.0)) +
         static_cast<unsigned long long>(__double2ll_rn((lo - rint(lo)) * 18446744073709551616.0));
}

// cos and sin of pos * f, times m.
__device__ __forceinline__ float2 turned(double f, int64_t pos, float m) {
  const unsigned long long a = turn_step(f) * static_cast<unsigned long long>(pos);
  const int top = static_cast<int>((a + 0x80000000ull) >> 32);  // signed: [-1/2, 1/2) of a turn
  float s, c;
  sincospif(static_cast<float>(top) * 4.656612873077392578125e-10f, &s, &c);  // 2^-31: half-turns
  return make_float2(c * m, s * m);
}

// The two 16-byte pieces (indices within the head's 32) of unit j.
__device__ __forceinline__ int2 unit_pieces(int j, int rot, bool inter) {
  return !inter && j < rot / 16 ? make_int2(j, j + rot / 16) : make_int2(2 * j, 2 * j + 1);
}

// Rotates unit j's eight pairs: cs[0..8) are their (cos, sin) m.
__device__ __forceinline__ void rotate_unit(uint4& a, uint4& b, const float2* cs, bool inter, float sign) {
  uint32_t* pa = reinterpret_cast<uint32_t*>(&a);
  uint32_t* pb = reinterpret_cast<uint32_t*>(&b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (inter) {  // each 32-bit word is a pair
      const float2 ca = cs[i], cb = cs[4 + i];
      const float a1 = bf16_lo(pa[i]), a2 = bf16_hi(pa[i]), b1 = bf16_lo(pb[i]), b2 = bf16_hi(pb[i]);
      const float sa = sign * ca.y, sb = sign * cb.y;
      pa[i] = pack_bf16(a1 * ca.x - a2 * sa, a1 * sa + a2 * ca.x);
      pb[i] = pack_bf16(b1 * cb.x - b2 * sb, b1 * sb + b2 * cb.x);
    } else {  // word i of both pieces: pairs 2i and 2i + 1
      const float2 c0 = cs[2 * i], c1 = cs[2 * i + 1];
      const float x0 = bf16_lo(pa[i]), x1 = bf16_hi(pa[i]), y0 = bf16_lo(pb[i]), y1 = bf16_hi(pb[i]);
      const float s0 = sign * c0.y, s1 = sign * c1.y;
      pa[i] = pack_bf16(x0 * c0.x - y0 * s0, x1 * c1.x - y1 * s1);
      pb[i] = pack_bf16(x0 * s0 + y0 * c0.x, x1 * s1 + y1 * c1.x);
    }
  }
}

__device__ __forceinline__ const uint4* piece(const HeadRows& x, int64_t t, int h) {
  return reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(x.p) + t * x.ts + h * x.hs);
}

// cos and sin (times m) of the block's tokens and pairs.
template <class Pos>
__device__ __forceinline__ void fill_turns(float2 (*cs)[kUnits * kCsUnit], const double* inv_freq, Pos pos, int n_tok,
                                           int rot, float m) {
  const int pairs = rot / 2;
  for (int i = threadIdx.x; i < n_tok * pairs; i += kRopeThreads) {
    const int tok = i / pairs, f = i - tok * pairs;
    cs[tok][(f >> 3) * kCsUnit + (f & 7)] = turned(__ldg(inv_freq + f), pos(tok), m);
  }
}

// A block's units, `ahead` per thread and round: unit u is unit j of head h of token tok.  They are counted in
// 32 bits: a block has 1024 at most or one token's heads, which the entry points bound.
struct Unit {
  int tok, h, j;
};
__device__ __forceinline__ Unit unit_at(int u, int heads) {
  const int r = u / kUnits, tok = r / heads;
  return {tok, r - tok * heads, u % kUnits};
}

// Rotates q (H heads) and k (G heads) of T tokens, n_blk a block.
__global__ void __launch_bounds__(kRopeThreads)
rope_kernel(HeadRows q, HeadRows k, HeadRows qo, HeadRows ko, const int32_t* __restrict__ positions,
            const double* __restrict__ inv_freq, int64_t T, int H, int G, int rot, bool inter, float m, float sign,
            int n_blk) {
  __shared__ float2 cs[kMaxTok][kUnits * kCsUnit];
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * n_blk;
  const int n_tok = static_cast<int>(min(static_cast<int64_t>(n_blk), T - t0));
  const int units = n_tok * (H + G) * kUnits;
  for (int u0 = 0; u0 < units; u0 += kAhead * kRopeThreads) {
    uint4 a[kAhead], b[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int u = u0 + i * kRopeThreads + threadIdx.x;
      if (u >= units) continue;
      const Unit x = unit_at(u, H + G);
      const uint4* src = x.h < H ? piece(q, t0 + x.tok, x.h) : piece(k, t0 + x.tok, x.h - H);
      const int2 pc = unit_pieces(x.j, rot, inter);
      a[i] = __ldcs(src + pc.x);
      b[i] = __ldcs(src + pc.y);
    }
    if (u0 == 0) {
      fill_turns(cs, inv_freq, [&](int tok) { return static_cast<int64_t>(__ldg(positions + t0 + tok)); }, n_tok, rot, m);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int u = u0 + i * kRopeThreads + threadIdx.x;
      if (u >= units) continue;
      const Unit x = unit_at(u, H + G);
      if (x.j < rot / 16) rotate_unit(a[i], b[i], cs[x.tok] + kCsUnit * x.j, inter, sign);
      uint4* dst = const_cast<uint4*>(x.h < H ? piece(qo, t0 + x.tok, x.h) : piece(ko, t0 + x.tok, x.h - H));
      const int2 pc = unit_pieces(x.j, rot, inter);
      __stcs(dst + pc.x, a[i]);
      __stcs(dst + pc.y, b[i]);
    }
  }
}

// Writes a packed batch's new K (rotated) and V rows into their pages, and the
// rotated q rows (when nq > 0; nq = H, or 0 without q) to qo.  Rows of no sequence
// are left alone; a row whose position has no page gets its q but no K/V row.
__global__ void __launch_bounds__(kRopeThreads, 6)
append_kernel(HeadRows q, HeadRows k, HeadRows v, HeadRows qo, __nv_bfloat16* __restrict__ k_pages,
              __nv_bfloat16* __restrict__ v_pages, CacheView c, const double* __restrict__ inv_freq, int64_t T, int nq,
              int G, int rot, bool inter, float m, int n_blk) {
  __shared__ float2 cs[kMaxTok][kUnits * kCsUnit];
  __shared__ int64_t s_pos[kMaxTok];
  __shared__ int s_row[kMaxTok];  // pool row, -1 without a page, -2 for a row of no sequence
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * n_blk;
  const int n_tok = static_cast<int>(min(static_cast<int64_t>(n_blk), T - t0));
  const int heads = nq + 2 * G;  // in the order q, k, v
  const int units = n_tok * heads * kUnits;
  for (int u0 = 0; u0 < units; u0 += kAppendAhead * kRopeThreads) {
    uint4 a[kAppendAhead], b[kAppendAhead];
    auto pieces = [&](const Unit& x) { return unit_pieces(x.j, x.h < nq + G ? rot : 0, inter); };
#pragma unroll
    for (int i = 0; i < kAppendAhead; ++i) {
      const int u = u0 + i * kRopeThreads + threadIdx.x;
      if (u >= units) continue;
      const Unit x = unit_at(u, heads);
      const uint4* src = x.h < nq ? piece(q, t0 + x.tok, x.h)
                                  : (x.h < nq + G ? piece(k, t0 + x.tok, x.h - nq) : piece(v, t0 + x.tok, x.h - nq - G));
      const int2 pc = pieces(x);
      a[i] = __ldcs(src + pc.x);
      b[i] = __ldcs(src + pc.y);
    }
    if (u0 == 0) {
      const int tok = threadIdx.x >> 5;  // a warp per token looks its place up
      static_assert(kMaxTok <= kRopeThreads / 32, "a warp per token");
      if (tok < n_tok) {
        const int seq = cache_seq(c, t0 + tok);
        const int64_t pos = seq < 0 ? 0 : cache_pos(c, seq, t0 + tok);
        s_pos[tok] = pos;
        s_row[tok] = seq < 0 ? -2 : cache_row(c, seq, pos);
      }
      __syncthreads();
      fill_turns(cs, inv_freq, [&](int tok) { return s_pos[tok]; }, n_tok, rot, m);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kAppendAhead; ++i) {
      const int u = u0 + i * kRopeThreads + threadIdx.x;
      if (u >= units) continue;
      const Unit x = unit_at(u, heads);
      const int row = s_row[x.tok];
      if (row < (x.h < nq ? -1 : 0)) continue;
      if (x.j < rot / 16 && x.h < nq + G) rotate_unit(a[i], b[i], cs[x.tok] + kCsUnit * x.j, inter, 1.f);
      uint4* dst;
      if (x.h < nq) {
        dst = const_cast<uint4*>(piece(qo, t0 + x.tok, x.h));
      } else {
        const int g = x.h < nq + G ? x.h - nq : x.h - nq - G;
        dst = reinterpret_cast<uint4*>((x.h < nq + G ? k_pages : v_pages) + (static_cast<int64_t>(row) * G + g) * kHeadDim);
      }
      const int2 pc = pieces(x);
      __stcs(dst + pc.x, a[i]);
      __stcs(dst + pc.y, b[i]);
    }
  }
}

// Tokens per block: `ahead` units a thread, but one token where there are few (a block per SM and more).
int tokens_per_block(int64_t T, int heads, int ahead) {
  int n = ahead * kRopeThreads / (heads * kUnits);
  n = n < 1 ? 1 : (n > kMaxTok ? kMaxTok : n);
  while (n > 1 && (T + n - 1) / n < 4 * sm_count()) n /= 2;
  return n;
}

}  // namespace

cudaError_t launch_rope(const HeadRows& q, const HeadRows& k, const HeadRows& qo, const HeadRows& ko,
                        const int32_t* positions, const double* inv_freq, int64_t T, int H, int G, int rot, bool inter,
                        float m, bool backward, cudaStream_t s) {
  const int n = tokens_per_block(T, H + G, kAhead);
  rope_kernel<<<static_cast<unsigned>((T + n - 1) / n), kRopeThreads, 0, s>>>(
      q, k, qo, ko, positions, inv_freq, T, H, G, rot, inter, m, backward ? -1.f : 1.f, n);
  return cudaGetLastError();
}

cudaError_t launch_cache_append(const HeadRows& q, const HeadRows& k, const HeadRows& v, const HeadRows& qo,
                                void* k_pages, void* v_pages, const CacheView& c, const double* inv_freq, int64_t T,
                                int nq, int G, int rot, bool inter, float m, cudaStream_t s) {
  const int n = tokens_per_block(T, nq + 2 * G, kAppendAhead);
  append_kernel<<<static_cast<unsigned>((T + n - 1) / n), kRopeThreads, 0, s>>>(
      q, k, v, qo, static_cast<__nv_bfloat16*>(k_pages), static_cast<__nv_bfloat16*>(v_pages), c, inv_freq, T, nq, G,
      rot, inter, m, n);
  return cudaGetLastError();
}

}  // namespace qsa
