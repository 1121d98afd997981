// Route-set attention of a packed batch's new tokens over a paged K/V cache.
//
// First the pool rows of every row's route set (paged_rows_kernel), then the forward's arithmetic
// over them, the 12 heads of a (token, KV group) pair at a time (softmax of scaled dot products with
// a running maximum that may lag by 2^8, P rounded to BF16 for P V, FP32 sums; empty rows give zero
// output and -inf LSE): chunks of 16 keys through a two-stage ring of 16-byte cp.async copies, four
// CTAs of two warps per SM.  Rows outside the set are never read, whatever they hold.
//
// A (token, key, group) costs 1 KB of K and V.  The gather runs at 30 B/clk/SM (512 tokens with 2048 routes
// over 131072: 139 us, L2 hit rate 41 %, DRAM 3.9 TB/s; 2048 tokens: 464 us), where a bare cp.async gather
// reaches 46 from L2 with 8 warps an SM and 25, the HBM limit, past it.  At those 8 warps, all that 254 registers
// a thread leave, the instructions of a 16-key chunk set the pace (413 a warp at 4.3 cycles each).
//
// P is BF16 because the tensor cores take P and V in one type, and V is BF16: a relative 2^-8 a term at most,
// 2.3e-3 of an output against 64 bits where rounding the output alone gives 1.7e-3.  Row sums are taken before it.
//
// Few tokens (a decode step) leave most SMs idle when one CTA takes a whole list, so a list is cut
// into `splits` parts whose unnormalised sums go to a workspace, and a second kernel joins them in
// part order (bit for bit reproducible).
#include "qsa_internal.h"
#include "qsa_device.cuh"
#include "qsa_launch.cuh"

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
constexpr int kOffJump = kOffDesc + 2 * 16;
constexpr int kSmem = kOffJump + ((kNw * 4 + 15) / 16) * 16;
static_assert((kSmem + 1024) * kCps <= 233472, "shared memory per SM");
constexpr int kFirst = 1, kLast = 2, kEnd = 4, kNone = 8;
constexpr float kLag = 8.f;
constexpr int kPartRow = kHeadDim;           // FP32 sums per head of a part, then (max, sum) pairs
constexpr int kPartFloats = kHeadsPerGroup * (kPartRow + 2);

__device__ __forceinline__ float p_of(float s, float m) { return s == -INFINITY ? 0.f : exp2f(s - m); }

// Pool rows of every row of route IDs: the IDs that name a position of the row's sequence with a
// page, each once, in the order of their first slots (the set's order does not matter, and route
// blocks stay runs of neighbouring rows).  row_cnt is -1 for a row of no sequence.
//
// A block per row, PER neighbouring slots a thread.  Duplicates are found in a hash table in shared
// memory (linear probing) that holds slots and keeps the smallest slot of each ID, so which slot
// stays does not depend on the threads' order; the slots that stayed are compacted in order.
// Bound by instructions: few slots a thread and a table four times the row keep probes short.
constexpr int kMaxRowThreads = 1024, kMaxSlots = 16384;
template <int PER>
__global__ void __launch_bounds__(kMaxRowThreads)
paged_rows_kernel(const int32_t* __restrict__ routes, CacheView cache, int n_sel, unsigned n_entries,
                  int* __restrict__ status, int32_t* __restrict__ row_cnt, int32_t* __restrict__ row_cols) {
  extern __shared__ unsigned table[];  // n_entries slots, then the row's IDs
  __shared__ int s_warp[32];
  constexpr unsigned kEmpty = ~0u;
  int* s_id = reinterpret_cast<int*>(table + n_entries);
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t* ids = routes + t * n_sel;
  const int i0 = PER * tid;
  next_may_start();
  int id[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) id[j] = i0 + j < n_sel ? __ldg(ids + i0 + j) : -1;
  if (t == 0 && tid == 0) *status = 0;
  for (unsigned i = tid; i < n_entries; i += blockDim.x) table[i] = kEmpty;
  const int seq = cache_seq(cache, t);
  if (seq < 0) {  // uniform
    if (tid == 0) row_cnt[t] = -1;
    return;
  }
  const int len = __ldg(cache.kv_len + seq);
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    if (id[j] >= len) id[j] = -1;
    if (i0 + j < n_sel) s_id[i0 + j] = id[j];
  }
  __syncthreads();
  unsigned at[PER];  // each ID's entry
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    if (id[j] < 0) continue;
    const unsigned mine = i0 + j;
    unsigned h = __umulhi(static_cast<unsigned>(id[j]) * 2654435769u, n_entries);
    for (;;) {  // ends: more entries than IDs
      const unsigned e = atomicCAS(table + h, kEmpty, mine);
      if (e == kEmpty) break;
      if (s_id[e] == id[j]) {
        atomicMin(table + h, mine);
        break;
      }
      if (++h == n_entries) h = 0;
    }
    at[j] = h;
  }
  __syncthreads();
  int mine = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j)  // id becomes the pool row
    id[j] = id[j] >= 0 && table[at[j]] == static_cast<unsigned>(i0 + j) ? cache_row(cache, seq, id[j]) : -1;
#pragma unroll
  for (int j = 0; j < PER; ++j) mine += id[j] >= 0;
  auto scan = [&](int x) {  // inclusive, over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    return x;
  };
  const int incl = scan(mine);
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  const int sums = scan(lane < static_cast<int>(blockDim.x >> 5) ? s_warp[lane] : 0);
  int out = incl - mine + (warp > 0 ? __shfl_sync(0xffffffffu, sums, warp - 1) : 0);
  int32_t* dst = row_cols + t * n_sel;
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (id[j] >= 0) dst[out++] = id[j];
  if (tid == static_cast<int>(blockDim.x) - 1) row_cnt[t] = out;  // the last slot's thread: all of them
}

__global__ void __launch_bounds__(kThreads, kCps)
paged_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
             const __nv_bfloat16* __restrict__ v, const int32_t* row_cnt, const int32_t* row_cols,
             int n_sel, unsigned n_items, int G, int splits, float scale_log2, float* partial,
             __nv_bfloat16* __restrict__ out, float* __restrict__ lse) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gq = lane >> 2, cq = lane & 3, mi = lane >> 3;
  const int H = G * kHeadsPerGroup;
  int4* desc = reinterpret_cast<int4*>(smem + kOffDesc);
  __nv_bfloat16* sP = reinterpret_cast<__nv_bfloat16*>(smem + kOffP);
  float* sMax = reinterpret_cast<float*>(smem + kOffMax);
  float* sSum = reinterpret_cast<float*>(smem + kOffSum);
  int* sJump = reinterpret_cast<int*>(smem + kOffJump);
  if (tid < 32) reinterpret_cast<uint4*>(smem + kOffZero)[tid] = make_uint4(0, 0, 0, 0);
  next_may_start();
  after_previous();

  // The chunk to issue next: item (t, g, split), keys [key0, key_end) of its row's list.
  unsigned it = blockIdx.x;
  unsigned t = 0;
  int g = 0, key0 = 0, key_end = 0;
  bool first = true, none = false;
  int cnt_next = 0;  // row_cnt of item it + gridDim.x, read an item ahead
  auto row_of_item = [&](unsigned i) { return i / static_cast<unsigned>(splits) / static_cast<unsigned>(G); };
  auto enter = [&](int cnt) {
    if (it >= n_items) return;
    const unsigned r = it / splits;
    t = r / G;
    g = static_cast<int>(r - t * G);
    const unsigned part = it - r * splits;
    none = cnt < 0;
    // parts of whole chunks, as equal as they go
    const unsigned n = (static_cast<unsigned>(max(cnt, 0)) + kKeys - 1) / kKeys;
    key0 = static_cast<int>(n * part / splits) * kKeys;
    key_end = min(static_cast<int>(n * (part + 1) / splits) * kKeys, cnt);
    first = true;
    const unsigned nx = it + gridDim.x;
    cnt_next = nx < n_items ? row_cnt[row_of_item(nx)] : 0;
  };
  // Lane j (and j + 8, ...) holds the pool row of the warp's key j of the chunk, -1 behind the last.
  auto rows_of = [&]() {
    const int i = key0 + 8 * warp + (lane & 7);
    return it < n_items && i < key_end ? row_cols[static_cast<int64_t>(t) * n_sel + i] : -1;
  };
  enter(it < n_items ? row_cnt[row_of_item(it)] : 0);
  int row = rows_of();
  // Issues the chunk into `stage`, records its descriptor, advances.
  auto issue = [&](int stage) {
    const uint32_t st = sbase + stage * kStageBytes;
    if (it < n_items) {
      const int nk = max(min(key_end - key0, kKeys), 0);
      if (nk > 0) {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const __nv_bfloat16* base = (kv ? v : k) + lane * 8;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int rj = __shfl_sync(0xffffffffu, row, j);
            const int64_t off = (static_cast<int64_t>(max(rj, 0)) * G + g) * kHeadDim;
            cp_async16(st + kv * kTile + swz512(8 * warp + j, lane), base + off, rj >= 0);
          }
        }
        if (first) {
          const __nv_bfloat16* qs = q + (static_cast<int64_t>(t) * H + g * kHeadsPerGroup) * kHeadDim;
#pragma unroll
          for (int r = 0; r < kHeadsPerGroup; r += kNw)
            cp_async16(st + 2 * kTile + swz512(r + warp, lane), qs + (r + warp) * kHeadDim + lane * 8, true);
        }
      }
      const bool last = key0 + kKeys >= key_end;
      if (tid == 0)
        desc[stage] = make_int4(static_cast<int>(it), nk, (first ? kFirst : 0) | (last ? kLast : 0) | (none ? kNone : 0),
                                0);
      first = false;
      key0 += kKeys;
      if (last) {
        it += gridDim.x;
        enter(cnt_next);
      }
    } else if (tid == 0) {
      desc[stage] = make_int4(0, 0, kEnd, 0);
    }
    cp_async_commit();
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
    issue(stage ^ 1);
    const int nk = d.y, flags = d.z;
    if (flags & kEnd) break;
    const unsigned vi = static_cast<unsigned>(d.x);
    const int64_t qrow0 = static_cast<int64_t>(vi / splits) * kHeadsPerGroup;  // [T, H] rows of the item's heads
    float* part = partial + static_cast<int64_t>(vi) * kPartFloats;
    if (nk == 0) {  // no keys: a part of one chunk
      if (flags & kNone) continue;
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
    if (flags & kFirst) {
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
    const int col = warp * 8 + 2 * cq;
    const bool v0 = col < nk, v1 = col + 1 < nk;
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
      *reinterpret_cast<uint32_t*>(sP + gq * kPStride + col) = pack_bf16(p0, p1);
      *reinterpret_cast<uint32_t*>(sP + (gq + 8) * kPStride + col) = pack_bf16(p2, p3);
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
      *reinterpret_cast<uint32_t*>(sP + gq * kPStride + col) = pack_bf16(p0, p1);
      *reinterpret_cast<uint32_t*>(sP + (gq + 8) * kPStride + col) = pack_bf16(p2, p3);
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
    if (flags & kLast) {  // CTA-uniform
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
        const float i0 = t0 == 0.f ? 0.f : 1.f / t0, i1 = t1 == 0.f ? 0.f : 1.f / t1;  // 0: all scores -inf
        __nv_bfloat16* orow = out + qrow0 * kHeadDim;
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt) {
          const int dim = warp * (kNt * 8) + nt * 8 + 2 * cq;
          *reinterpret_cast<uint32_t*>(orow + gq * kHeadDim + dim) = pack_bf16(o[nt][0] * i0, o[nt][1] * i0);
          if (second)
            *reinterpret_cast<uint32_t*>(orow + (gq + 8) * kHeadDim + dim) = pack_bf16(o[nt][2] * i1, o[nt][3] * i1);
        }
        if (warp == 0 && cq == 0) {
          lse[qrow0 + gq] = (m0 + log2f(t0)) * kLn2;
          if (second) lse[qrow0 + gq + 8] = (m1 + log2f(t1)) * kLn2;
        }
      }
    }
  }
  cp_async_wait<0>();
}

// Joins the parts of a (token, group), 8 dims per lane.  Few parts: a block per (token, group), a warp
// per head.  Many parts (few rows): a block per head, its warps an eighth of the parts each, added in
// order (one warp over 32 parts took 11 us, eight take 5).
constexpr int kManyParts = 8;
template <bool MANY>
__global__ void __launch_bounds__(MANY ? 256 : kHeadsPerGroup * 32)
paged_join_kernel(const float* partial, const int32_t* row_cnt, int G, int splits,
                  __nv_bfloat16* __restrict__ out, float* __restrict__ lse) {
  __shared__ float sO[MANY ? 8 : 1][kHeadDim];
  __shared__ float sL[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned item = MANY ? blockIdx.x / kHeadsPerGroup : blockIdx.x;
  const int h = MANY ? blockIdx.x - item * kHeadsPerGroup : warp;
  const float* base = partial + static_cast<int64_t>(item) * splits * kPartFloats;
  const float* ml = base + kHeadsPerGroup * kPartRow + 2 * h;
  after_previous();
  const bool none = row_cnt[item / G] < 0;
  float m = -INFINITY;
  for (int i = lane; i < splits; i += 32) m = fmaxf(m, ml[static_cast<int64_t>(i) * kPartFloats]);
  if (none) return;  // a row of no sequence (uniform)
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  float l = 0.f, o[8] = {};
  const int first = MANY ? splits * warp / 8 : 0, end = MANY ? splits * (warp + 1) / 8 : splits;
#pragma unroll 8
  for (int i = first; i < end; ++i) {
    const float2 x = *reinterpret_cast<const float2*>(ml + static_cast<int64_t>(i) * kPartFloats);
    const float4* p = reinterpret_cast<const float4*>(base + static_cast<int64_t>(i) * kPartFloats + h * kPartRow) + 2 * lane;
    float4 u = p[0], y = p[1];
    float w = x.x == -INFINITY ? 1.f : exp2f(x.x - m);
    if (x.x == -INFINITY && x.y == 0.f) {  // a part without visible keys wrote no sums
      w = 0.f;
      u = y = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    l += x.y * w;
    o[0] += u.x * w, o[1] += u.y * w, o[2] += u.z * w, o[3] += u.w * w;
    o[4] += y.x * w, o[5] += y.y * w, o[6] += y.z * w, o[7] += y.w * w;
  }
  if (MANY) {
#pragma unroll
    for (int i = 0; i < 8; ++i) sO[warp][8 * lane + i] = o[i];
    if (lane == 0) sL[warp] = l;
    __syncthreads();
    if (warp > 0) return;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      l += sL[w];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] += sO[w][8 * lane + i];
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t row = static_cast<int64_t>(item) * kHeadsPerGroup + h;
  *reinterpret_cast<uint4*>(out + row * kHeadDim + 8 * lane) =
      make_uint4(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv),
                 pack_bf16(o[4] * inv, o[5] * inv), pack_bf16(o[6] * inv, o[7] * inv));
  if (lane == 0) lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace

// Parts per row.  A part costs its keys and, where parts have to be joined, about 25 keys' time
// (12 KB of sums written and read again, against 1 KB of K and V per key); the CTAs take parts in
// turn, so the call lasts as long as the CTA with the most of them.  The best number makes that
// least, never with under 64 keys a part: many parts where rows are few, one or a few where the
// last round of whole rows would leave most CTAs idle (2048 rows of 2048 keys on 592 CTAs: 738 us
// whole).
int paged_splits(int64_t T, int G, int64_t max_keys) {
  const int64_t slots = 148 * kCps, items = T * G;
  int best = 1;
  double least = 0.0;
  for (int n = 1; n <= 64 && (n == 1 || n * 64 <= max_keys); ++n) {
    if (n > 1 && items * n > 16 * slots) break;  // the last round no longer counts
    const double rounds = static_cast<double>((items * n + slots - 1) / slots);
    const double cost = rounds * (static_cast<double>(max_keys) / n + (n > 1 ? 25.0 : 0.0));
    if (n == 1 || cost < least) {
      least = cost;
      best = n;
    }
  }
  return best;
}

size_t paged_partial_bytes(int64_t T, int G, int splits) {
  return splits > 1 ? static_cast<size_t>(T) * G * splits * kPartFloats * sizeof(float) : 0;
}

cudaError_t launch_paged_rows(const int32_t* routes, const CacheView& c, int64_t T, int n_sel, int* status,
                              int32_t* row_cnt, int32_t* row_cols, cudaStream_t s) {
  const int n_entries = n_sel < 16 ? 64 : (n_sel <= 8192 ? 4 * n_sel : 2 * n_sel);
  const int smem = 4 * (n_entries + n_sel), per = n_sel <= 2048 ? 2 : (n_sel <= 4096 ? 4 : 16);
  const auto kern = per == 2 ? paged_rows_kernel<2> : (per == 4 ? paged_rows_kernel<4> : paged_rows_kernel<16>);
  if (per > 2) {  // the most that any row of this variant takes, whatever other threads launch meanwhile
    const int most = per == 4 ? 4 * (4 * 4096 + 4096) : 4 * (2 * kMaxSlots + kMaxSlots);
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
  }
  const int threads = ((n_sel + per - 1) / per + 31) / 32 * 32;
  kern<<<static_cast<unsigned>(T), threads, smem, s>>>(routes, c, n_sel, n_entries, status, row_cnt, row_cols);
  return cudaGetLastError();
}

cudaError_t launch_paged_forward(const void* q, const void* k_pages, const void* v_pages, const int32_t* row_cnt,
                                 const int32_t* row_cols, int64_t T, int G, int n_sel, float scale, int splits,
                                 void* partial, void* out, float* lse, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(paged_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const int64_t n_items = T * G * splits;
  const int64_t slots = static_cast<int64_t>(kCps) * sm_count();
  e = launch_after(paged_kernel, dim3(static_cast<unsigned>(n_items < slots ? n_items : slots)), kThreads, kSmem, s,
                   static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k_pages),
                   static_cast<const __nv_bfloat16*>(v_pages), row_cnt, row_cols, n_sel,
                   static_cast<unsigned>(n_items), G, splits, scale * kLog2e, static_cast<float*>(partial),
                   static_cast<__nv_bfloat16*>(out), lse);
  if (e != cudaSuccess || splits == 1) return e;
  const bool many = splits > kManyParts;
  return launch_after(many ? paged_join_kernel<true> : paged_join_kernel<false>,
                      dim3(static_cast<unsigned>(T * G * (many ? kHeadsPerGroup : 1))),
                      many ? 256 : kHeadsPerGroup * 32, 0, s, static_cast<const float*>(partial), row_cnt, G, splits,
                      static_cast<__nv_bfloat16*>(out), lse);
}

}  // namespace qsa
