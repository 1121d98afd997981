// Attention of a packed batch's new tokens over a paged K/V cache, one query
// token at a time: the 12 heads of a (token, KV group) pair against a list of
// keys, by route IDs (the row's sorted, de-duplicated list) or by position (a
// window and first tokens, or everything up to the token).
//
// The arithmetic is the forward's (softmax of scaled dot products with a running
// maximum that may lag by 2^8, P rounded to BF16 for P V, FP32 sums; empty rows
// give zero output and -inf LSE).  What differs is where a key lies: its position
// goes through the sequence's block table to a pool row as its copy is issued,
// one key per lane, and a key without a row (a position at or past kv_len, an
// unmapped page) is zero-filled and masked.  So a value outside the visible set
// is never read, whatever it holds.
//
// Few tokens (a decode step) leave most SMs idle when one CTA takes a whole
// list, so a list is cut into `splits` runs of chunks whose unnormalised sums
// go to a workspace, and a second kernel joins them in run order (bit for bit
// reproducible).
#include "qsa_internal.h"
#include "qsa_device.cuh"

namespace qsa {
namespace {

constexpr int kNw = 2, kCps = 4;             // warps per CTA, CTAs per SM (the forward's shape)
constexpr int kThreads = kNw * 32;
constexpr int kKeys = 8 * kNw;               // keys per chunk
constexpr int kNt = kHeadDim / kNw / 8;      // n8 tiles of P V per warp
constexpr int kTile = kKeys * 512;
constexpr int kStageBytes = 2 * kTile + kHeadsPerGroup * 512;  // K | V | Q rows
constexpr int kPStride = kKeys + 8;
constexpr int kOffZero = 2 * kStageBytes;    // 512 zero bytes: Q rows 12..15
constexpr int kOffP = kOffZero + 512;
constexpr int kOffMax = kOffP + kRowTile * kPStride * 2;
constexpr int kOffSum = kOffMax + kNw * kRowTile * 4;
constexpr int kOffDesc = kOffSum + kNw * kRowTile * 4;
constexpr int kOffLive = kOffDesc + 2 * 16;  // [stage][warp]: which of the warp's 8 keys have a row
constexpr int kOffJump = kOffLive + 2 * kNw * 4;
constexpr int kSmem = kOffJump + ((kNw * 4 + 15) / 16) * 16;
static_assert((kSmem + 1024) * kCps <= 233472, "shared memory per SM");
constexpr int kFirst = 1, kLast = 2, kEnd = 4;
constexpr float kLag = 8.f;
constexpr int kPartRow = kHeadDim;           // FP32 sums per head of a part, then (max, sum) pairs
constexpr int kPartFloats = kHeadsPerGroup * (kPartRow + 2);

__device__ __forceinline__ float p_of(float s, float m) { return s == -INFINITY ? 0.f : exp2f(s - m); }

// Where the keys of an item come from.
struct RouteKeys {
  const int32_t* row_cnt;
  const int32_t* row_cols;
  int n_sel;
};
struct Keys {  // the keys of one row: key i is cols[i], or i < n_first ? i : base + i
  const int32_t* cols;
  int64_t base;
  int n_first, cnt;
  int64_t limit;  // positions at or above it are not visible
};
__device__ __forceinline__ Keys row_keys(const RouteKeys& r, const CacheView& c, int seq, int64_t t) {
  Keys k;
  k.cols = r.row_cols + t * r.n_sel;
  k.base = 0;
  k.n_first = 0;
  k.cnt = __ldg(r.row_cnt + t);
  k.limit = __ldg(c.kv_len + seq);
  return k;
}
template <class Source>
__global__ void __launch_bounds__(kThreads, kCps)
paged_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
             const __nv_bfloat16* __restrict__ v, CacheView cache, Source src, unsigned n_items, int G, int splits,
             float scale_log2, float* __restrict__ partial, __nv_bfloat16* __restrict__ out,
             float* __restrict__ lse) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gq = lane >> 2, cq = lane & 3, mi = lane >> 3;
  const int H = G * kHeadsPerGroup;
  int4* desc = reinterpret_cast<int4*>(smem + kOffDesc);
  __nv_bfloat16* sP = reinterpret_cast<__nv_bfloat16*>(smem + kOffP);
  float* sMax = reinterpret_cast<float*>(smem + kOffMax);
  float* sSum = reinterpret_cast<float*>(smem + kOffSum);
  unsigned* sLive = reinterpret_cast<unsigned*>(smem + kOffLive);
  int* sJump = reinterpret_cast<int*>(smem + kOffJump);
  if (tid < 32) reinterpret_cast<uint4*>(smem + kOffZero)[tid] = make_uint4(0, 0, 0, 0);

  // The chunk to issue next: item (t, g, split), chunk ch of [ch, ch_end), its row's keys.
  unsigned it = blockIdx.x;
  int64_t t = 0;
  int g = 0, seq = -1, ch = 0, ch_first = 0, ch_end = 0;
  Keys keys{};
  auto enter = [&]() {  // item `it`
    if (it >= n_items) return;
    const unsigned r = it / splits;
    t = r / G;
    g = static_cast<int>(r - static_cast<unsigned>(t) * G);
    const unsigned part = it - r * splits;
    seq = cache_seq(cache, t);
    ch = ch_first = 0;
    ch_end = 1;  // an empty run has one chunk without keys
    if (seq >= 0) {
      keys = row_keys(src, cache, seq, t);
      const int64_t n = (static_cast<int64_t>(keys.cnt) + kKeys - 1) / kKeys;
      ch = ch_first = static_cast<int>(n * part / splits);
      ch_end = static_cast<int>(n * (part + 1) / splits);
      if (ch_end == ch) {
        keys.cnt = 0;
        ch_end = ch + 1;
      }
    } else {
      keys.cnt = 0;
    }
  };
  // Lane j (and j + 8, ...) holds the pool row of the warp's key j in the chunk, -1 without one.
  auto rows_of = [&]() {
    if (it >= n_items) return -1;
    const int64_t i = static_cast<int64_t>(ch) * kKeys + 8 * warp + (lane & 7);
    if (i >= keys.cnt) return -1;
    const int64_t j = keys.cols ? __ldg(keys.cols + i) : (i < keys.n_first ? i : keys.base + i);
    return j < keys.limit ? cache_row(cache, seq, j) : -1;
  };
  enter();
  int row = rows_of();
  // Issues the chunk into `stage`, records its descriptor, advances.
  auto issue = [&](int stage) {
    const uint32_t st = sbase + stage * kStageBytes;
    if (it < n_items) {
      const bool any = static_cast<int64_t>(ch) * kKeys < keys.cnt;
      if (any) {
        const unsigned live = __ballot_sync(0xffffffffu, row >= 0) & 0xff;
        if (lane == 0) sLive[stage * kNw + warp] = live;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const __nv_bfloat16* base = (kv ? v : k) + lane * 8;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int rj = __shfl_sync(0xffffffffu, row, j);
            const int r = 8 * warp + j;
            const int64_t off = (static_cast<int64_t>(max(rj, 0)) * G + g) * kHeadDim;
            cp_async16(st + kv * kTile + swz512(r, lane), base + off, rj >= 0);
          }
        }
        if (ch == ch_first) {
          const __nv_bfloat16* qs = q + (t * H + g * kHeadsPerGroup) * kHeadDim;
#pragma unroll
          for (int r = 0; r < kHeadsPerGroup; r += kNw)
            cp_async16(st + 2 * kTile + swz512(r + warp, lane), qs + (r + warp) * kHeadDim + lane * 8, true);
        }
      }
      // x: item, y: row's head offset in units of 12, or -1 for a row of no sequence
      if (tid == 0)
        desc[stage] = make_int4(static_cast<int>(it), seq < 0 ? -1 : 0, any ? 1 : 0,
                                (ch == ch_first ? kFirst : 0) | (ch == ch_end - 1 ? kLast : 0));
    } else if (tid == 0) {
      desc[stage] = make_int4(0, 0, 0, kEnd);
    }
    cp_async_commit();
    if (it < n_items && ++ch == ch_end) {
      it += gridDim.x;
      enter();
    }
    row = rows_of();
  };
  issue(0);

  uint32_t qa[16][4];
  float o[kNt][4];
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  const uint32_t spa = smem_u32(sP);

  for (int c = 0;; ++c) {
    const int stage = c & 1;
    const uint32_t st = sbase + stage * kStageBytes;
    cp_async_wait<0>();
    __syncthreads();  // chunk c has landed; every warp is done with chunk c - 1
    const int4 d = desc[stage];
    const unsigned live = sLive[stage * kNw + warp];
    issue(stage ^ 1);
    if (d.w & kEnd) break;
    const unsigned vi = static_cast<unsigned>(d.x);
    const int64_t qrow0 = static_cast<int64_t>(vi / splits) * kHeadsPerGroup;  // [T, H] rows of the item's heads
    float* part = partial + static_cast<int64_t>(vi) * kPartFloats;
    if (d.z == 0) {  // no keys: a run of one chunk
      if (d.y < 0) continue;
      if (splits > 1) {
        if (tid < kHeadsPerGroup) {  // maximum -inf: the join reads no sums
          part[kHeadsPerGroup * kPartRow + 2 * tid] = -INFINITY;
          part[kHeadsPerGroup * kPartRow + 2 * tid + 1] = 0.f;
        }
      } else {
        uint4* orow = reinterpret_cast<uint4*>(out + qrow0 * kHeadDim);
        for (int i = tid; i < kHeadsPerGroup * 32; i += kThreads) orow[i] = make_uint4(0, 0, 0, 0);
        if (tid < kHeadsPerGroup) lse[qrow0 + tid] = -INFINITY;
      }
      continue;
    }
    if (d.w & kFirst) {
#pragma unroll
      for (int ks = 0; ks < 16; ++ks) {
        const int r = ((mi & 1) << 3) + (lane & 7);
        const int cc = 2 * ks + (mi >> 1);
        ldsm_x4(qa[ks], r < kHeadsPerGroup ? st + 2 * kTile + swz512(r, cc) : sbase + kOffZero + (cc << 4));
      }
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt) o[nt][0] = o[nt][1] = o[nt][2] = o[nt][3] = 0.f;
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.f;
    }
    // S = Q K^T for this warp's 8 keys, as four independent accumulation chains
    float s[4];
    {
      float sp[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) sp[j][0] = sp[j][1] = sp[j][2] = sp[j][3] = 0.f;
#pragma unroll
      for (int ks = 0; ks < 16; ks += 2) {
        uint32_t b[4];
        ldsm_x4(b, st + swz512(warp * 8 + (lane & 7), 2 * ks + mi));
        mma_16816(sp[(ks >> 1) & 3], qa[ks], b[0], b[1]);
        mma_16816(sp[(ks >> 1) & 3], qa[ks + 1], b[2], b[3]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = (sp[0][i] + sp[1][i]) + (sp[2][i] + sp[3][i]);
    }
    const int key0 = warp * 8 + 2 * cq;
    const bool v0 = live >> (2 * cq) & 1, v1 = live >> (2 * cq + 1) & 1;
    s[0] = v0 ? s[0] * scale_log2 : -INFINITY;
    s[1] = v1 ? s[1] * scale_log2 : -INFINITY;
    s[2] = v0 ? s[2] * scale_log2 : -INFINITY;
    s[3] = v1 ? s[3] * scale_log2 : -INFINITY;
    // P against the running maximum as it stands; it is replaced only when a
    // score exceeds it by more than kLag (then every warp rescales together)
    const bool jump = fmaxf(s[0], s[1]) > m0 + kLag || fmaxf(s[2], s[3]) > m1 + kLag;
    const unsigned any_jump = __any_sync(0xffffffffu, jump);
    float p0 = p_of(s[0], m0), p1 = p_of(s[1], m0), p2 = p_of(s[2], m1), p3 = p_of(s[3], m1);
    if (!any_jump) {
      *reinterpret_cast<uint32_t*>(sP + gq * kPStride + key0) = pack_bf16(p0, p1);
      *reinterpret_cast<uint32_t*>(sP + (gq + 8) * kPStride + key0) = pack_bf16(p2, p3);
    }
    float x0 = fmaxf(s[0], s[1]), x1 = fmaxf(s[2], s[3]);
    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
    if (cq == 0) {
      sMax[warp * kRowTile + gq] = x0;
      sMax[warp * kRowTile + gq + 8] = x1;
    }
    if (lane == 0) sJump[warp] = any_jump ? 1 : 0;
    __syncthreads();
    bool rescale = false;
#pragma unroll
    for (int w = 0; w < kNw; ++w) rescale |= sJump[w] != 0;
    if (rescale) {  // CTA-uniform
      float n0 = m0, n1 = m1;
#pragma unroll
      for (int w = 0; w < kNw; ++w) {
        n0 = fmaxf(n0, sMax[w * kRowTile + gq]);
        n1 = fmaxf(n1, sMax[w * kRowTile + gq + 8]);
      }
      const float a0 = n0 == -INFINITY ? 1.f : exp2f(m0 - n0), a1 = n1 == -INFINITY ? 1.f : exp2f(m1 - n1);
      m0 = n0;
      m1 = n1;
      l0 *= a0;
      l1 *= a1;
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt) {
        o[nt][0] *= a0;
        o[nt][1] *= a0;
        o[nt][2] *= a1;
        o[nt][3] *= a1;
      }
      p0 = p_of(s[0], m0);
      p1 = p_of(s[1], m0);
      p2 = p_of(s[2], m1);
      p3 = p_of(s[3], m1);
      *reinterpret_cast<uint32_t*>(sP + gq * kPStride + key0) = pack_bf16(p0, p1);
      *reinterpret_cast<uint32_t*>(sP + (gq + 8) * kPStride + key0) = pack_bf16(p2, p3);
      __syncthreads();
    }
    l0 += p0 + p1;  // this lane's part of the row sums
    l1 += p2 + p3;
    {
      uint32_t pa[4];
      ldsm_x4(pa, spa + (((((mi & 1) << 3) + (lane & 7)) * kPStride + ((mi >> 1) << 3)) << 1));
#pragma unroll
      for (int nt = 0; nt < kNt; nt += 2) {
        uint32_t b[4];
        ldsm_x4_t(b, st + kTile + swz512(((mi & 1) << 3) + (lane & 7), warp * kNt + nt + (mi >> 1)));
        mma_16816(o[nt], pa, b[0], b[1]);
        mma_16816(o[nt + 1], pa, b[2], b[3]);
      }
    }
    if (d.w & kLast) {  // CTA-uniform
      float c0 = l0, c1 = l1;
      c0 += __shfl_xor_sync(0xffffffffu, c0, 1);
      c0 += __shfl_xor_sync(0xffffffffu, c0, 2);
      c1 += __shfl_xor_sync(0xffffffffu, c1, 1);
      c1 += __shfl_xor_sync(0xffffffffu, c1, 2);
      if (cq == 0) {
        sSum[warp * kRowTile + gq] = c0;
        sSum[warp * kRowTile + gq + 8] = c1;
      }
      __syncthreads();
      float t0 = 0.f, t1 = 0.f;
#pragma unroll
      for (int w = 0; w < kNw; ++w) {
        t0 += sSum[w * kRowTile + gq];
        t1 += sSum[w * kRowTile + gq + 8];
      }
      const bool second = gq + 8 < kHeadsPerGroup;
      if (splits > 1) {
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt) {
          const int dim = warp * (kNt * 8) + nt * 8 + 2 * cq;
          *reinterpret_cast<float2*>(part + gq * kPartRow + dim) = make_float2(o[nt][0], o[nt][1]);
          if (second) *reinterpret_cast<float2*>(part + (gq + 8) * kPartRow + dim) = make_float2(o[nt][2], o[nt][3]);
        }
        if (warp == 0 && cq == 0) {
          float2* ml = reinterpret_cast<float2*>(part + kHeadsPerGroup * kPartRow);
          ml[gq] = make_float2(m0, t0);
          if (second) ml[gq + 8] = make_float2(m1, t1);
        }
      } else {
        // a zero sum: every listed key was without a row
        const float i0 = t0 == 0.f ? 0.f : 1.f / t0, i1 = t1 == 0.f ? 0.f : 1.f / t1;
        __nv_bfloat16* orow = out + qrow0 * kHeadDim;
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt) {
          const int dim = warp * (kNt * 8) + nt * 8 + 2 * cq;
          *reinterpret_cast<uint32_t*>(orow + gq * kHeadDim + dim) = pack_bf16(o[nt][0] * i0, o[nt][1] * i0);
          if (second)
            *reinterpret_cast<uint32_t*>(orow + (gq + 8) * kHeadDim + dim) = pack_bf16(o[nt][2] * i1, o[nt][3] * i1);
        }
        if (warp == 0 && cq == 0) {
          lse[qrow0 + gq] = t0 == 0.f ? -INFINITY : (m0 + log2f(t0)) * kLn2;
          if (second) lse[qrow0 + gq + 8] = t1 == 0.f ? -INFINITY : (m1 + log2f(t1)) * kLn2;
        }
      }
    }
  }
  cp_async_wait<0>();
}

// Joins the parts of head `blockIdx.x % 12` of one (token, group): one warp per
// quarter of the parts, 8 dims per lane, the quarters added in order.
constexpr int kJoinWarps = 4;
__global__ void __launch_bounds__(kJoinWarps * 32)
paged_join_kernel(const float* __restrict__ partial, CacheView cache, int G, int splits,
                  __nv_bfloat16* __restrict__ out, float* __restrict__ lse) {
  __shared__ float sO[kJoinWarps][kHeadDim];
  __shared__ float sL[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned item = blockIdx.x / kHeadsPerGroup, h = blockIdx.x - item * kHeadsPerGroup;
  if (cache_seq(cache, item / G) < 0) return;
  const float* base = partial + static_cast<int64_t>(item) * splits * kPartFloats;
  const float* ml = base + kHeadsPerGroup * kPartRow + 2 * h;
  float m = -INFINITY;
  for (int i = lane; i < splits; i += 32) m = fmaxf(m, ml[static_cast<int64_t>(i) * kPartFloats]);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  const int a = splits * warp / kJoinWarps, z = splits * (warp + 1) / kJoinWarps;
  float l = 0.f, o[8] = {};
#pragma unroll 4
  for (int i = a; i < z; ++i) {
    const float2 x = *reinterpret_cast<const float2*>(ml + static_cast<int64_t>(i) * kPartFloats);
    if (x.x == -INFINITY && x.y == 0.f) continue;  // a part without visible keys wrote no sums
    const float w = x.x == -INFINITY ? 1.f : exp2f(x.x - m);
    const float4* p = reinterpret_cast<const float4*>(base + static_cast<int64_t>(i) * kPartFloats + h * kPartRow) + 2 * lane;
    const float4 u = p[0], y = p[1];
    l += x.y * w;
    o[0] += u.x * w, o[1] += u.y * w, o[2] += u.z * w, o[3] += u.w * w;
    o[4] += y.x * w, o[5] += y.y * w, o[6] += y.z * w, o[7] += y.w * w;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) sO[warp][8 * lane + i] = o[i];
  if (lane == 0) sL[warp] = l;
  __syncthreads();
  float total = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) total += sL[w];
  const float inv = total == 0.f ? 0.f : 1.f / total;
  const int64_t row = static_cast<int64_t>(item) * kHeadsPerGroup + h;
  const int d = 2 * threadIdx.x;
  float y0 = 0.f, y1 = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    y0 += sO[w][d];
    y1 += sO[w][d + 1];
  }
  *reinterpret_cast<uint32_t*>(out + row * kHeadDim + d) = pack_bf16(y0 * inv, y1 * inv);
  if (threadIdx.x == 0) lse[row] = total == 0.f ? -INFINITY : (m + log2f(total)) * kLn2;
}

template <class Source>
cudaError_t launch(const void* q, const void* k, const void* v, const CacheView& c, const Source& src, int64_t T, int G,
                   float scale, int splits, void* partial, void* out, float* lse, cudaStream_t s) {
  auto kern = paged_kernel<Source>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const int64_t n_items = T * G * splits;
  const int64_t slots = static_cast<int64_t>(kCps) * sm_count();
  kern<<<static_cast<unsigned>(n_items < slots ? n_items : slots), kThreads, kSmem, s>>>(
      static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v),
      c, src, static_cast<unsigned>(n_items), G, splits, scale * kLog2e, static_cast<float*>(partial),
      static_cast<__nv_bfloat16*>(out), lse);
  e = cudaGetLastError();
  if (e != cudaSuccess || splits == 1) return e;
  paged_join_kernel<<<static_cast<unsigned>(T * G * kHeadsPerGroup), kJoinWarps * 32, 0, s>>>(
      static_cast<const float*>(partial), c, G, splits, static_cast<__nv_bfloat16*>(out), lse);
  return cudaGetLastError();
}

}  // namespace

// Parts per row: enough to fill the resident CTAs of a 148-SM device when there
// are few rows, never under 64 keys a part.
int paged_splits(int64_t T, int G, int64_t max_keys) {
  const int64_t slots = 148 * kCps, items = T * G;
  const int64_t fill = slots / items, most = (max_keys + 63) / 64;
  const int64_t n = fill < most ? fill : most;
  return n < 1 ? 1 : static_cast<int>(n);
}

size_t paged_partial_bytes(int64_t T, int G, int splits) {
  return splits > 1 ? static_cast<size_t>(T) * G * splits * kPartFloats * sizeof(float) : 0;
}

cudaError_t launch_paged_forward(const void* q, const void* k_pages, const void* v_pages, const CacheView& c,
                                 const int32_t* row_cnt, const int32_t* row_cols, int64_t T, int G, int n_sel,
                                 float scale, int splits, void* partial, void* out, float* lse, cudaStream_t s) {
  return launch(q, k_pages, v_pages, c, RouteKeys{row_cnt, row_cols, n_sel}, T, G, scale, splits, partial, out, lse, s);
}

}  // namespace qsa
