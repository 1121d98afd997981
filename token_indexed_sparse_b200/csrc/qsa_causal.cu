// Positional attention of a packed batch's new tokens over a paged K/V cache on
// the fifth-generation tensor cores: the token at position p sees the keys j <= p
// with j > p - window or j < sinks (all j <= p without a window).
//
// The 12 heads of a KV group read the same keys, so the rows of a query tile are
// (token, head) pairs: tile i of sequence b and group g holds the flattened rows
// [128 i, 128 i + 128) of the sequence's 12 n new rows, about 11 tokens, and all of
// its keys but a few at the diagonal and at the window's edge are seen by every row.
//
// Work.  An item (b, i, g) is a run of 128-key tiles.  All tiles of all items, in
// order, are cut into equal ranges, one per CTA (one CTA per SM), so a decode step
// over a few long caches and a prompt of many tiles both fill the device; a CTA
// finds its range by scanning the lengths itself (the host knows none of them).  An
// item that falls into several ranges leaves unnormalised FP32 sums per range in the
// workspace, and causal_join_kernel adds them in range order (bit for bit
// reproducible; at most two parts per CTA).
//
// Pipeline of one CTA (12 warps):
//   warp 8      page lookups and TMA: K as two [128 keys][128 dims] units, V as two
//               [64 keys][256 dims] units, through one ring of five 32 KB units in the order
//               the tensor core consumes them: K0 K1 V0 K2 V1 K3 ...
//   warp 9      issues S(x) = Q K^T (M 128, N 128) into one of two S buffers
//   warp 10     issues O += P V (M 128, N 256, P read from tensor memory)
//   warps 0-7   softmax: row r of the tile on two threads, 64 keys each: P = exp2(S scale
//               log2e - m) as BF16 over the half's own S columns; the running maximum m may
//               lag the true one by 2^8 (P < 256), so O is rescaled only on a jump
//   warp 11     the next item's Q rows (cp.async into the 128-byte swizzle)
// Tensor memory: O 256 columns, S / P two buffers of 128.
//
// Both products cost 1024 tensor cycles per tile (4096 multiply-adds a cycle and SM), Q K^T
// 1500 in fact: with M = N = 128 its operands come through shared memory in 94 cycles an
// instruction, not 64.  A decode step is bound by the cache's bytes (48 sequences of up to
// 32768 tokens: 0.27 ms, 6.3 TB/s), a long chunk by the time from S to P and back, about
// 3200 cycles a tile, and by the power cap when kept up (2048 tokens behind 30000, 24 heads:
// 1.23 to 1.26 ms, 1.2 to 1.3 PFLOP/s in a burst, 1.40 to 1.48 ms kept up; in 1024 behind 16000,
// tensor pipe 64 % active, MUFU 32 %).  Short items (a window of 1021: 131 us for 39 us of operations,
// tensor pipe 33 %) by their starts, ends and edge tiles.
//
// P is BF16 because a product takes both operands in one 16-bit type, and V is BF16: 2.3e-3 of an output
// against 64 bits where rounding the output alone gives 1.7e-3.  Row sums are taken before it.
//
// Values that a row must not see: keys past the diagonal, outside the window, without a
// page are masked in S.  P V multiplies every V row of the tile, and 0 * NaN is NaN, so in
// a tile that some row does not see whole, V rows that no row sees are overwritten with
// zeros, and non-finite elements of rows that only some see are zeroed and added back, in
// the epilogue, to the rows that see them.
#include <cuda.h>

#include "qsa_cache.cuh"
#include "qsa_device.cuh"
#include "qsa_internal.h"
#include "qsa_launch.cuh"

namespace qsa {
namespace {

constexpr int kRows = 128;                     // query rows per tile
constexpr int kTileKeys = 128;
constexpr int kThreads = 384;
constexpr int kProducer = 8, kMmaS = 9, kMmaO = 10, kLoader = 11;  // warps
constexpr int kUnits = 5;                      // ring units
constexpr int kSubBytes = 16384;               // K: [128 keys][64 dims]; V: 32 keys of 256 dims
constexpr int kUnitBytes = 2 * kSubBytes;
constexpr int kOffRing = kRows * 512;          // Q: four [128][64] blocks, 128-byte swizzle
constexpr int kOffX = kOffRing + kUnits * kUnitBytes;  // [2][2][128] floats that a row's threads exchange
constexpr int kOffBar = kOffX + 4 * kRows * 4;
// barriers
constexpr int kBFull = 0, kBEmpty = kBFull + kUnits, kBQFull = kBEmpty + kUnits, kBQEmpty = kBQFull + 1,
              kBS = kBQEmpty + 1, kBP = kBS + 2, kBPv = kBP + 2, kBDrain = kBPv + 2,
              kBars = kBDrain + 2;
constexpr int kOffTmem = kOffBar + kBars * 8;
constexpr int kOffAbort = kOffTmem + 4;
constexpr int kOffPoison = kOffAbort + 4;      // [3]: the item saw non-finite V it had to take out
constexpr int kOffStart = kOffPoison + 12;     // the CTA's first tile: sequence, query tile, group, tile
constexpr int kOffTile = kOffStart + 16;       // tiles whose scores have been issued
constexpr int kSmem = kOffTile + 4;            // no room to align the base: checked instead
static_assert(kSmem <= 232448, "shared memory per block");
constexpr uint32_t kSpin = 1u << 22;           // polls before a wait gives up (seconds)
constexpr uint32_t kColS = 256;                // tensor-memory columns: O [0, 256), S0, S1
constexpr float kLag = 8.f;
constexpr int kMinTiles = 2;                   // fewer tiles than this are not worth a CTA of their own
constexpr int kMaxCtas = 148;
constexpr int kPartFloats = kRows * kHeadDim;  // FP32 sums of a part
// kind::f16, FP32 accumulate, BF16: S (both K-major, N 128) and O (B MN-major, N 256)
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10);
constexpr uint32_t kIdescS = kIdesc | ((128u >> 3) << 17);
constexpr uint32_t kIdescO = kIdesc | (1u << 16) | ((256u >> 3) << 17);
// M, in the instruction descriptor.  A tile of one token (12 rows) takes M 64: its first 16 rows lie in
// the same lanes, the time is the same, the power is not.
__device__ __forceinline__ uint32_t idesc_m(int rows) { return (rows <= 16 ? 64u >> 4 : 128u >> 4) << 24; }

struct Args {
  CacheView c;
  int64_t T;
  int G;
  int window, sinks;
};

// ---------------------------------------------------------------------------
// items
// ---------------------------------------------------------------------------

// Positions are 32 bits here: a first position is taken as -2^30 at least and the packed rows are below 2^28,
// so what is below zero stays there and nothing wraps.
struct Seq {          // one sequence's new tokens (clamped to the packed rows)
  int start, n;       // packed rows [start, start + n)
  int p0;             // position of the first
};
__device__ __forceinline__ Seq seq_of(const Args& a, int b) {
  Seq s;
  const int end = __ldg(a.c.cu_q + b + 1), z = min(max(end, 0), static_cast<int>(a.T));
  s.start = min(max(__ldg(a.c.cu_q + b), 0), z);
  s.n = z - s.start;
  const int64_t p0 = static_cast<int64_t>(__ldg(a.c.kv_len + b)) - (static_cast<int64_t>(end) - s.start);
  s.p0 = static_cast<int>(max(p0, static_cast<int64_t>(-(1 << 30))));
  return s;
}
__device__ __forceinline__ int query_tiles(const Seq& s) {
  return (s.n * kHeadsPerGroup - 1) / kRows + (s.n > 0 ? 1 : 0);
}
// Keys [lo, hi) and [0, first) that a token at position p sees.
__device__ __forceinline__ int row_hi(const Args& a, int p) {
  return max(0, min(p + 1, a.c.max_pages << a.c.page_shift));
}
__device__ __forceinline__ int row_lo(const Args& a, int p) {
  return a.window > 0 && p + 1 > a.window ? p + 1 - a.window : 0;
}
__device__ __forceinline__ int first_keys(const Args& a) { return a.window > 0 ? a.sinks : 0; }

struct Item {         // what query tile i of a sequence sees
  int rows;           // valid rows
  int hi0, hi1;       // row_hi of its first and last token
  int lo0, lo1;       // row_lo of them
  int n_first;        // key tiles of the first keys in front of the window's
  int w_first;        // first key tile of the window
  int n;              // key tiles, at least one
};
__device__ __forceinline__ Item item_of(const Args& a, const Seq& s, int i) {
  Item it;
  const int r0 = i * kRows;  // below n * 12 <= T * H, which fits 31 bits
  it.rows = min(kRows, s.n * kHeadsPerGroup - r0);
  const int pa = s.p0 + r0 / kHeadsPerGroup, pz = s.p0 + (r0 + it.rows - 1) / kHeadsPerGroup;
  it.hi0 = row_hi(a, pa);
  it.hi1 = row_hi(a, pz);
  it.lo0 = row_lo(a, pa);
  it.lo1 = row_lo(a, pz);
  it.w_first = it.lo0 / kTileKeys;
  const int first = (min(first_keys(a), it.hi1) + kTileKeys - 1) / kTileKeys;
  const int n_w = it.hi1 > it.lo0 ? (it.hi1 + kTileKeys - 1) / kTileKeys - it.w_first : 0;
  if (n_w == 0) it.w_first = 0;
  it.n_first = n_w > 0 ? min(first, it.w_first) : first;
  it.n = max(it.n_first + n_w, 1);
  return it;
}
// V lies in runs of neighbouring keys, [four 64-dim blocks][run][64 dims]: 32 keys, or a 16-key page.
__device__ __forceinline__ int v_run(const Args& a) { return a.c.page_shift == 4 ? 16 : 32; }
__device__ __forceinline__ int key_tile(const Item& it, int x) {
  return x < it.n_first ? x : it.w_first + x - it.n_first;
}

// Whether any row sees one of the 16 keys from `key` on (key 0's always count, so that every item has
// a product that starts its sums): the steps that P V takes.
__device__ __forceinline__ bool step_seen(const Item& it, int first, int key) {
  return key == 0 || key < first || (key < it.hi1 && key + 16 > it.lo0);
}

// The CTA's walk: pieces (item, tiles [x0, x1)) of its range.  Every role walks alone:
//   Walk w(...); while (w.take(a)) { ...; }
struct Walk {
  int b, i, g, x0, x1;
  int64_t left;   // tiles after this piece
  int k;          // piece counter
  Seq s;
  Item it;
  __device__ __forceinline__ Walk(const Args& a, const int* start, int64_t tiles)
      : b(start[0]), i(start[1]), g(start[2]), x0(0), x1(start[3]), left(tiles), k(-1), s(seq_of(a, b)) {
    it.n = 0;
  }
  __device__ __forceinline__ bool take(const Args& a) {  // the next piece (one site per role: it is much code)
    if (left <= 0) return false;
    if (++k == 0) {
      x0 = x1;
    } else {
      x0 = 0;
      if (++g == a.G) {
        g = 0;
        if (++i == query_tiles(s)) {
          i = 0;
          do s = seq_of(a, ++b);
          while (s.n == 0 && b + 1 < a.c.B);
        }
      }
    }
    it = item_of(a, s, i);
    x1 = static_cast<int>(min(static_cast<int64_t>(it.n), x0 + left));
    left -= x1 - x0;
    return true;
  }
};

template <typename V>
__device__ __forceinline__ V block_scan(V x, V* warp_sums, V& total) {  // inclusive, 384 threads
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  V before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    total += warp_sums[w];
  }
  return x + before;
}

// Walks all query tiles in batches of 384, a thread each: f(sequence or -1, query
// tile, its key tiles times G), called by every thread of the block; stops when it returns true.
template <class F>
__device__ __forceinline__ void each_batch(const Args& a, int* pre, long long* sums, F f) {
  for (int b0 = 0; b0 < a.c.B; b0 += kThreads) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    const int nq = b < a.c.B ? query_tiles(seq_of(a, b)) : 0;
    int n_all;
    const int incl = block_scan<int>(nq, reinterpret_cast<int*>(sums), n_all);
    pre[threadIdx.x] = incl - nq;
    __syncthreads();
    for (int j0 = 0; j0 < n_all; j0 += kThreads) {
      const int j = j0 + static_cast<int>(threadIdx.x);
      int seq = -1, i = 0;
      long long w = 0;
      if (j < n_all) {
        int lo = 0, hi = kThreads;  // the last sequence of the chunk with pre <= j
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (pre[mid] <= j) lo = mid;
          else hi = mid;
        }
        seq = b0 + lo;
        i = j - pre[lo];
        w = static_cast<long long>(item_of(a, seq_of(a, seq), i).n) * a.G;
      }
      if (f(seq, i, w)) return;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// tensor core, tensor memory, TMA
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint64_t desc_k_major(uint32_t addr) {  // 128-byte swizzle, 8-row groups 1024 bytes apart
  return static_cast<uint64_t>((addr >> 4) & 0x3fff) | (static_cast<uint64_t>(1) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}
// MN-major: 64-dim blocks `run` keys (of 128 bytes) apart, 8-key groups 1024 bytes
__device__ __forceinline__ uint64_t desc_v(uint32_t addr, int run) {
  return static_cast<uint64_t>((addr >> 4) & 0x3fff) | (static_cast<uint64_t>(run * 128 >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr) : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float (&v)[64]) {
  uint32_t r[64];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr) : "memory");
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      " tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr) : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
      "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]),
      "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]),
      "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int row, int chunk, int g, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];\n" ::"r"(dst),
      "l"(map), "r"(0), "r"(row), "r"(chunk), "r"(g), "r"(bar)
      : "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// Two FP32 operations an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 a, a, b, c;\n mov.b64 {%0, %1}, a;\n}\n"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}\n"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u); }

// Polls a barrier kSpin times at most, and no longer once a role has given up.
__device__ __forceinline__ bool poll_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  bool ok = mbar_try(bar, parity);
#pragma unroll 1
  for (uint32_t it = 0; !ok && it < kSpin; ++it) {
    ok = mbar_try(bar, parity);
    if ((it & 255) == 255 && *abort_flag) break;
  }
  return ok;
}
// Bounded wait that also gives up once another role has.  For what takes a few tiles' time.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  const bool ok = poll_bar(bar, parity, abort_flag);
  if (!ok) *abort_flag = 1;
  return ok;
}
// Brings a warp's lanes together without __syncwarp's memory ordering, which waits for every read
// in flight (a page of the block table: 800 cycles).
__device__ __forceinline__ void converge() {
  asm volatile("{\n .reg .pred p, q;\n setp.eq.u32 q, 0, 0;\n vote.sync.all.pred p, q, 0xffffffff;\n}\n");
}
// The same for a whole warp: every lane polls (and so has the barrier's ordering itself), all agree.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag));
}

// A whole warp's wait for the end of an item, which may have millions of key tiles: its polls start over as
// long as tiles are issued (whoever issues them waits a tile's time at most, and gives up by itself).
__device__ __forceinline__ bool warp_wait_item(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                               volatile int* tile) {
  for (;;) {
    const int seen = __shfl_sync(0xffffffffu, *tile, 0);
    if (__all_sync(0xffffffffu, poll_bar(bar, parity, abort_flag))) return true;
    const bool stuck = *abort_flag || *tile == seen;
    if (__shfl_sync(0xffffffffu, stuck, 0)) break;
  }
  *abort_flag = 1;
  return false;
}

struct Ring {  // position in the ring of units
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step(int n = 1) {  // n <= kUnits
    slot += n;
    if (slot >= kUnits) {
      slot -= kUnits;
      phase ^= 1;
    }
  }
};

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------

// Part of the workspace per CTA: where its last item goes on.
struct __align__(16) Cont {
  int row0;    // packed row of the query tile's first token
  int rows;    // 0: the CTA's last item ends in its range
  int first;   // head, within the group, of the query tile's first row
  int g;
  int c_last;  // the last CTA with a part
  int status;  // nonzero: a bounded wait gave up
  int pad[2];
};

__global__ void __launch_bounds__(kThreads, 1)
causal_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
              const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ v_pool, const Args a,
              float scale_log2, float* __restrict__ part, float2* __restrict__ part_ml, Cont* __restrict__ cont,
              __nv_bfloat16* __restrict__ out, float* __restrict__ lse) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = a.G * kHeadsPerGroup;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffAbort);
  int* start = reinterpret_cast<int*>(smem + kOffStart);
  volatile int* tile = reinterpret_cast<volatile int*>(smem + kOffTile);
  auto bar = [&](int i) { return sb + kOffBar + 8 * i; };

  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(&k_map) : "memory");
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(&v_map) : "memory");
  }
  // ---- the CTA's range of tiles (scratch in the ring, before any copy)
  int64_t t_begin = 0, t_end = 0, n_tiles = 0;
  int n_ctas = 1;
  {
    int* pre = reinterpret_cast<int*>(smem + kOffRing);
    long long* sums = reinterpret_cast<long long*>(smem + kOffRing + 4096);
    long long mine = 0, all = 0;
    int batches = 0, seq0 = -1, tile0 = 0;  // the last batch's query tile of this thread
    long long w0 = 0;
    each_batch(a, pre, sums, [&](int seq, int i, long long w) {
      mine += w;
      ++batches;
      seq0 = seq, tile0 = i, w0 = w;
      return false;
    });
    const long long incl0 = block_scan<long long>(mine, sums, all);
    n_tiles = all;
    n_ctas = static_cast<int>(min(static_cast<int64_t>(gridDim.x), max(n_tiles / kMinTiles, static_cast<int64_t>(1))));
    const int c = static_cast<int>(blockIdx.x);
    const bool aligned = (sb & 1023) == 0;  // what the 128-byte swizzle needs
    if (tid == 0) {
      Cont ct{};
      ct.status = aligned ? 0 : 2;
      cont[c] = ct;
    }
    if (n_tiles == 0 || c >= n_ctas || !aligned) return;  // uniform
    t_begin = n_tiles * c / n_ctas;
    t_end = n_tiles * (c + 1) / n_ctas;
    auto locate = [&](int seq, int i, long long w, long long at) {  // if the range begins in this query tile
      if (t_begin < at || t_begin >= at + w) return;
      const int n = static_cast<int>(w / a.G);
      const long long off = t_begin - at;  // of the key tiles of all groups, which may pass 31 bits
      const int g = off <= 0x7fffffff ? static_cast<int>(off) / n : static_cast<int>(off / n);
      start[0] = seq;
      start[1] = i;
      start[2] = g;
      start[3] = static_cast<int>(off - static_cast<long long>(g) * n);
    };
    if (batches == 1) {  // what the scan above has in hand
      locate(seq0, tile0, w0, incl0 - w0);
    } else {
      long long base = 0;
      each_batch(a, pre, sums, [&](int seq, int i, long long w) {
        long long batch;
        const long long incl = block_scan<long long>(w, sums, batch);
        locate(seq, i, w, base + incl - w);
        base += batch;
        return base > t_begin;
      });
    }
  }
  if (tid == 0) {
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(bar(kBFull + i), 1);
      mbar_init(bar(kBEmpty + i), 1);
    }
    mbar_init(bar(kBQFull), 32);
    mbar_init(bar(kBQEmpty), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBS + i), 1);
      mbar_init(bar(kBP + i), 8);
      mbar_init(bar(kBPv + i), 1);
    }
    mbar_init(bar(kBDrain), 1);
    mbar_init(bar(kBDrain + 1), 1);
    *abort_flag = 0;
    *tile = 0;
    for (int i = 0; i < 3; ++i) reinterpret_cast<int*>(smem + kOffPoison)[i] = 0;
    mbar_fence_init();
  }
  if (warp == kMmaS) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(sb + kOffTmem), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  fence_before();
  fence_proxy_async();  // the scan's scratch lies where TMA writes next
  __syncthreads();
  fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + kOffTmem);
  const int64_t tiles = t_end - t_begin;


  if (warp == kProducer) {
    // ------------------------------------------------------------ K / V units
    const int page_shift = a.c.page_shift, page = 1 << page_shift;
    const int n_pg = page < kTileKeys ? kTileKeys >> page_shift : 1;  // pages per tile
    const int no_row = a.c.n_pages << page_shift;                      // past the pool: TMA fills zeros
    const int k_box = min(page, kTileKeys), run = v_run(a);
    Ring ring;
    uint32_t issued = 0;
    bool ok = true;
    Walk w(a, start, tiles);
    // lane l holds the pool row of the first key of page l of a tile
    auto rows_of = [&](int x) {
      const int64_t j = static_cast<int64_t>(key_tile(w.it, x)) * kTileKeys + static_cast<int64_t>(lane) * page;
      const int r = lane < n_pg ? cache_row(a.c, w.b, j) : -1;
      return r < 0 ? no_row : r;
    };
    auto claim = [&]() {  // the next unit, free and expecting its bytes
      ok = warp_wait(bar(kBEmpty + ring.slot), ring.phase ^ 1, abort_flag);
      if (!ok) return;
      if (lane == 0) mbar_arrive_tx(bar(kBFull + ring.slot), kUnitBytes);
      __syncwarp();
      ++issued;
    };
    auto load_k = [&](int rows) {
#pragma unroll 1
      for (int u = 0; u < 2; ++u) {
        claim();
        if (!ok) return;
        // lane = block of 64 dims * pages + page
        const int blk = lane >= n_pg ? 1 : 0, pg = lane - blk * n_pg;
        const int r = __shfl_sync(0xffffffffu, rows, pg & 31);
        if (lane < 2 * n_pg)
          tma_load(sb + kOffRing + ring.slot * kUnitBytes + blk * kSubBytes + pg * k_box * 128, &k_map, r, 2 * u + blk,
                   w.g, bar(kBFull + ring.slot));
        ring.step();
      }
    };
    auto load_v = [&](int rows) {
#pragma unroll 1
      for (int u = 0; u < 2; ++u) {
        claim();
        if (!ok) return;
        const uint32_t dst = sb + kOffRing + ring.slot * kUnitBytes;
        // lane = run of keys
        const int key = 64 * u + run * (lane & 3), from = page < kTileKeys ? (key & 127) >> page_shift : 0;
        const int r = __shfl_sync(0xffffffffu, rows, from);
        if (lane < 64 / run)
          tma_load(dst + lane * run * 512, &v_map, r == no_row ? no_row : r + key - (from << page_shift), 0, w.g,
                   bar(kBFull + ring.slot));
        ring.step();
      }
    };
    while (ok && w.take(a)) {
      int cur = rows_of(w.x0), prev = 0;
      for (int x = w.x0; x < w.x1 && ok; ++x) {
        const int ahead = x + 1 < w.x1 ? rows_of(x + 1) : 0;  // table reads a tile ahead of their use
        load_k(cur);
        if (x > w.x0 && ok) load_v(prev);
        prev = cur;
        cur = ahead;
      }
      if (ok) load_v(prev);
    }
    if (lane == 0) {  // copies in flight end before the block does, whoever has given up meanwhile (bounded)
      Ring r = ring;
      for (uint32_t i = 0; i < min(issued, static_cast<uint32_t>(kUnits)); ++i) {
        if (--r.slot < 0) {
          r.slot = kUnits - 1;
          r.phase ^= 1;
        }
        mbar_wait(bar(kBFull + r.slot), r.phase);
      }
    }
    __syncwarp();
  } else if (warp == kMmaS || warp == kMmaO) {
    // ------------------------------------------------------------ tensor core
    // One thread per product: each wait and commit stalls its thread for longer than the few
    // instructions that queue at the tensor core last, so one thread alone left it idle for
    // half of the time; two keep it fed.
    if (lane == 0) {
      Ring ring;
      bool ok = true;
      uint32_t tau = 0;  // tiles so far
      Walk w(a, start, tiles);
      auto wait = [&](int i, uint32_t parity) { return wait_bar(bar(i), parity, abort_flag); };
      if (warp == kMmaS) {
        const uint64_t q_desc = desc_k_major(sb), k_desc = desc_k_major(sb + kOffRing);
        while (ok && w.take(a)) {
          ok = wait(kBQFull, w.k & 1);
          const int n = w.x1 - w.x0;
          const uint32_t idesc = kIdescS | idesc_m(w.it.rows);
#pragma unroll 1
          for (int y = 0; y < n && ok; ++y, ++tau) {
            const uint32_t s = tmem + kColS + 128 * (tau & 1);
            // P of tile tau - 2 has been read (S of this tile goes over it); K's two units are there.
            // A wait costs its thread 150 cycles even when it is over, so K's, which came long ago,
            // come first.  They may not in an item's first two tiles: a parity tells a unit's use from
            // the one before it only, so the slot's previous use (5 units earlier) must be known to have
            // landed.  From the third tile on that is V of tile tau - 3, whose product the wait
            // of the tile before saw end, and K of tile tau - 1; in the first two it is V of the item
            // before, whose product the wait for tile tau - 2 sees end.
            Ring second = ring;
            second.step();
            auto landed = [&]() {
              return wait(kBFull + ring.slot, ring.phase) && wait(kBFull + second.slot, second.phase);
            };
            if (y >= 2) ok = landed();
            if (ok && tau >= 2) ok = wait(kBPv + (tau & 1), ((tau - 2) >> 1) & 1);
            if (ok && y < 2) ok = landed();
            if (!ok) break;
            fence_after();
            *tile = static_cast<int>(tau + 1);
#pragma unroll 1
            for (int u = 0; u < 2; ++u) {
              const uint64_t kd = k_desc + ring.slot * (kUnitBytes >> 4), qd = q_desc + u * (2 * kRows * 128 >> 4);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                mma_ss(s, qd + (i >> 2) * (kRows * 128 >> 4) + 2 * (i & 3), kd + (i >> 2) * (kSubBytes >> 4) + 2 * (i & 3),
                       idesc, i > 0 || u > 0);
              commit(bar(kBEmpty + ring.slot));
              ring.step();
            }
            commit(bar(kBS + (tau & 1)));
            if (y > 0) ring.step(2);  // V of tile y - 1
          }
          if (ok) commit(bar(kBQEmpty));
          ring.step(2);               // V of the last tile
        }
      } else {
        const int run = v_run(a), first = first_keys(a);
        const uint64_t v_desc = desc_v(sb + kOffRing, run);
        while (ok && w.take(a)) {
          const int n = w.x1 - w.x0;
          bool summing = false;       // the item's first product starts its sums
          const uint32_t idesc = kIdescO | idesc_m(w.it.rows);
          ring.step(n > 1 ? 4 : 2);   // K of the first two tiles
#pragma unroll 1
          for (int y = 0; y < n && ok; ++y, ++tau) {
            const uint32_t p = tmem + kColS + 128 * (tau & 1);
            const int k0 = key_tile(w.it, w.x0 + y) * kTileKeys;
            uint32_t steps = 0;  // of 16 keys, those that some row sees
#pragma unroll
            for (int i = 0; i < 8; ++i) steps |= step_seen(w.it, first, k0 + 16 * i) ? 1u << i : 0u;
            // What is over early first, P last.  S of this tile before V's units: their slots' previous
            // uses are K of this tile and V of the tiles before it (see the parity note above).  An item's
            // first P also says that the sums before have been read: the same threads do both.
            Ring second = ring;
            second.step();
            ok = wait(kBS + (tau & 1), (tau >> 1) & 1) && wait(kBFull + ring.slot, ring.phase) &&
                 wait(kBFull + second.slot, second.phase) && wait(kBP + (tau & 1), (tau >> 1) & 1);
            if (!ok) break;
            fence_after();
#pragma unroll 1
            for (int u = 0; u < 2; ++u) {
              const uint64_t vd = v_desc + ring.slot * (kUnitBytes >> 4);
#pragma unroll
              for (int i = 0; i < 4; ++i) {  // 16 keys: a run, or half of one
                if (!(steps >> (4 * u + i) & 1)) continue;
                mma_ts(tmem, p + 64 * u + 8 * i,
                       vd + (run == 16 ? i * (8192 >> 4) : (i >> 1) * (kSubBytes >> 4) + (i & 1) * (2048 >> 4)), idesc, summing);
                summing = true;
              }
              commit(bar(kBEmpty + ring.slot));
              ring.step();
            }
            commit(bar(kBPv + (tau & 1)));
            if (y + 2 < n) ring.step(2);  // K of tile y + 2
          }
        }
      }
      // The products in flight end before tensor memory is freed, whoever has given up meanwhile (bounded).
      const int i = kBDrain + (warp == kMmaO ? 1 : 0);
      commit(bar(i));
      mbar_wait(bar(i), 0);
    }
    __syncwarp();
  } else if (warp >= kLoader) {
    // ------------------------------------------------------------ Q rows
    Walk w(a, start, tiles);
    bool ok = true;
    while (w.take(a)) {
      if (w.k > 0) ok = warp_wait_item(bar(kBQEmpty), (w.k - 1) & 1, abort_flag, tile);
      if (!ok) break;
      // a 512-byte row an instruction; rows past the last are zeros, whose products draw less power than
      // leftovers (a decode step of 12 rows kept up for a second: 315 us against 327)
      const int r0 = w.i * kRows;
      int h = r0 % kHeadsPerGroup;
      const __nv_bfloat16* src = q + ((static_cast<int64_t>(w.s.start) + r0 / kHeadsPerGroup) * H +
                                      w.g * kHeadsPerGroup + h) * kHeadDim + lane * 8;
      const int64_t to_next_token = static_cast<int64_t>(H - kHeadsPerGroup + 1) * kHeadDim;
      const uint32_t dst = sb + (lane >> 3) * (kRows * 128);
#pragma unroll 4
      for (int r = 0; r < kRows; ++r) {
        cp_async16(dst + r * 128 + (((lane & 7) ^ (r & 7)) << 4), src, r < w.it.rows);
        if (++h == kHeadsPerGroup) {
          h = 0;
          src += to_next_token;
        } else {
          src += kHeadDim;
        }
      }
      cp_async_commit();
      cp_async_wait<0>();
      fence_proxy_async();
      mbar_arrive(bar(kBQFull));
    }
  } else {
    // ------------------------------------------------------------ softmax
    // Thread (half, row): keys 64 half .. 64 half + 63 of every tile.  Both halves of a tile at once
    // (against a tile per warpgroup, two at a time) halve the time between S and P, which is
    // what keeps the tensor core waiting.  A wait that gives up does not end the walk: no wait after it
    // polls, so the hardware barriers below always meet.
    const int half = warp >> 2, wq = warp & 3, row = 32 * wq + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * wq) << 16);
    volatile float* sX = reinterpret_cast<volatile float*>(smem + kOffX);
    volatile int* poison = reinterpret_cast<volatile int*>(smem + kOffPoison);
    const int page_shift = a.c.page_shift;
    const int n_pg = (1 << page_shift) < kTileKeys ? kTileKeys >> page_shift : 1;
    const int first = first_keys(a);
    uint32_t tau = 0, units = 0;  // tiles so far, ring units before the piece
    uint32_t ex = 0;              // exchanges so far
    bool given_up = false;
    auto wait = [&](int i, uint32_t parity) {
      if (!given_up) given_up = !wait_bar(bar(i), parity, abort_flag);
      converge();
    };
    // the other thread's value of the row (two buffers in turn: a buffer is written again only after
    // the exchange behind it, which both have reached)
    auto give = [&](float x) { sX[((ex & 1) * 2 + half) * kRows + row] = x; };
    auto other = [&]() {
      bar_sync(1 + wq, 64);
      return sX[((ex++ & 1) * 2 + (half ^ 1)) * kRows + row];
    };
    Walk w(a, start, tiles);
    while (w.take(a)) {
      const bool live = 32 * wq < w.it.rows;
      const int r0 = w.i * kRows;
      const int p = w.s.p0 + (r0 + row) / kHeadsPerGroup;
      const int hi = row < w.it.rows ? row_hi(a, p) : 0, lo = row < w.it.rows ? row_lo(a, p) : 0;
      const int n = w.x1 - w.x0;
      // Lane l's page of the l-th page of tile y, read a tile ahead of its use
      // (volatile: sunk to its use, the read's latency stood between S and P of every tile).
      auto page_of = [&](int y) {
        if (y >= n || lane >= n_pg) return -1;
        const int64_t pg = (static_cast<int64_t>(key_tile(w.it, w.x0 + y)) * kTileKeys >> page_shift) + lane;
        if (pg >= a.c.max_pages) return -1;
        int v;
        asm volatile("ld.global.nc.b32 %0, [%1];\n"
                     : "=r"(v) : "l"(a.c.table + static_cast<int64_t>(w.b) * a.c.max_pages + pg));
        return v;
      };
      int page = page_of(0);
      float m = -INFINITY, l = 0.f;  // the row's running maximum; this half's part of its sum
      for (int y = 0; y < n; ++y, ++tau) {
        const int k0 = key_tile(w.it, w.x0 + y) * kTileKeys;
        // pages of the tile without a row
        const uint32_t bad = __ballot_sync(0xffffffffu, lane < n_pg && (page < 0 || page >= a.c.n_pages));
        page = page_of(y + 1);
        const bool edge = bad != 0 || k0 + kTileKeys > w.it.hi0 || (k0 < w.it.lo1 && k0 + kTileKeys > first);
        // the row's visible keys among 32 i .. 32 i + 31 of the tile
        auto vis = [&](int i) {
          const int c0 = k0 + 32 * i;
          uint32_t v = low_bits(hi - c0) & (~low_bits(lo - c0) | low_bits(first - c0));
          if (bad != 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (bad >> (n_pg > 1 ? (32 * i + 16 * h) >> page_shift : 0) & 1) v &= h ? 0x0000ffffu : 0xffff0000u;
          }
          return v;
        };
        const uint32_t s_addr = lanes + kColS + 128 * (tau & 1) + 64 * half;
        wait(kBS + (tau & 1), (tau >> 1) & 1);
        fence_after();
        if (live) {
          // P against the maximum before this tile; once more only if that has to move
          float sum, top = -INFINITY;
          uint32_t pk[32];
          const float m_old = m;
          for (bool again = false;; again = true) {
            float s[64];
            float2 ls = make_float2(0.f, 0.f);
            tmem_ld64(s_addr, s);
            if (edge) {
              const uint32_t v0 = vis(2 * half), v1 = vis(2 * half + 1);
#pragma unroll
              for (int c = 0; c < 32; ++c) {
                s[c] = v0 >> c & 1 ? s[c] : -INFINITY;
                s[32 + c] = v1 >> c & 1 ? s[32 + c] : -INFINITY;
              }
            }
            if (!again) {
#pragma unroll
              for (int c = 0; c < 64; c += 2) top = fmaxf(top, fmaxf(s[c], s[c + 1]));
              top *= scale_log2;
              give(top);                            // the other half's maximum comes while P is computed,
              if (y == 0) m = fmaxf(top, other());  // or is waited for: nothing is known yet
            }
            const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int c = 0; c < 64; c += 2) {
              const float2 x = fma2(make_float2(s[c], s[c + 1]), make_float2(scale_log2, scale_log2), make_float2(-base, -base));
              const float2 p = make_float2(exp2_fast(x.x), exp2_fast(x.y));
              ls = add2(ls, p);
              pk[c >> 1] = pack_bf16(p.x, p.y);
            }
            sum = ls.x + ls.y;
            if (again || y == 0) break;
            top = fmaxf(top, other());
            if (top > m + kLag) m = top;
            if (!__any_sync(0xffffffffu, m != m_old)) break;
          }
          // O holds sums against m_old: this half of the dims, where the maximum moved
          const bool jump = y > 0 && m != m_old && m_old != -INFINITY;
          if (__any_sync(0xffffffffu, jump)) {
            wait(kBPv + ((tau - 1) & 1), ((tau - 1) >> 1) & 1);
            fence_after();
            const float f = jump ? exp2_fast(m_old - m) : 1.f;
#pragma unroll 1
            for (int i = 4 * half; i < 4 * half + 4; ++i) {
              float o[32];
              tmem_ld32(lanes + 32 * i, o);
#pragma unroll
              for (int c = 0; c < 32; ++c) o[c] *= f;
              tmem_st32(lanes + 32 * i, o);
            }
          }
          if (m != m_old) l *= exp2_fast(m_old - m);
          l += sum;
          tmem_st32(s_addr, pk);
          tmem_st_wait();
        }
        if (edge) {
          // this thread's key of the tile and half of its dims: V rows that not every query row sees, in
          // the steps that P V takes
          const int j = k0 + row;
          const bool page_ok = !(bad >> (n_pg > 1 ? row >> page_shift : 0) & 1);
          const bool any = page_ok && j < w.it.hi1 && (j >= w.it.lo0 || j < first);
          const bool all = page_ok && j < w.it.hi0 && (j >= w.it.lo1 || j < first);
          // V of tile y follows K of tile y + 1: its two units are 4 y + 4 on, the last tile's 4 y + 2
          const uint32_t u = units + (y + 1 < n ? 4 * y + 4 : 4 * y + 2) + (row >> 6);
          // the slot may have held V of the tile before: only once that has been used does the unit's
          // parity tell this use from that one
          if (y > 0) wait(kBPv + ((tau - 1) & 1), ((tau - 1) >> 1) & 1);
          wait(kBFull + u % kUnits, (u / kUnits) & 1);
          const int run = v_run(a), in_unit = row & 63;
          uint8_t* vr = smem + kOffRing + (u % kUnits) * kUnitBytes + in_unit / run * run * 512 + in_unit % run * 128;
          if (!all && step_seen(w.it, first, j & ~15)) {
            for (int i = 16 * half; i < 16 * half + 16; ++i) {
              uint4* x = reinterpret_cast<uint4*>(vr + (i >> 3) * run * 128 + (((i & 7) ^ (lane & 7)) << 4));
              if (!any) {
                *x = make_uint4(0, 0, 0, 0);
                continue;
              }
              uint4 val = *x;
              uint32_t* e = reinterpret_cast<uint32_t*>(&val);
              bool changed = false;
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const uint32_t z = e[c];
                if ((z & 0x7f80u) == 0x7f80u) e[c] &= 0xffff0000u;
                if ((z & 0x7f800000u) == 0x7f800000u) e[c] &= 0x0000ffffu;
                changed |= e[c] != z;
              }
              if (changed) {
                *x = val;
                poison[w.k % 3] = 1;
              }
            }
          }
          fence_proxy_async();
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBP + (tau & 1)));
      }
      units += 4 * n;
      // ---- epilogue: the row's sum, then half of the dims each
      if (tid == 0) poison[(w.k + 1) % 3] = 0;  // last read two items ago
      bar_sync(5, 256);                          // every thread's part of poison[k % 3] is in
      const bool poisoned = poison[w.k % 3] != 0;
      give(l);
      const float total = l + other();  // the same in both
      wait(kBPv + ((tau - 1) & 1), ((tau - 1) >> 1) & 1);
      fence_after();
      if (live) {
        const bool whole = w.x0 == 0 && w.x1 == w.it.n;
        // [T, H] row of a row of the tile
        auto out_row = [&](int r) {
          const int f = w.i * kRows + r, t = f / kHeadsPerGroup;
          return (static_cast<int64_t>(w.s.start) + t) * H + w.g * kHeadsPerGroup + f - t * kHeadsPerGroup;
        };
        const int slot = 2 * static_cast<int>(blockIdx.x) + (w.x0 == 0 ? 1 : 0);
        const float inv = total == 0.f ? 0.f : 1.f / total;
        // Stores of whole rows by their threads would touch 32 lines each; so four lanes exchange the
        // 16-byte pieces of their rows and store 64 bytes of a row together.
        // (One site for outputs and parts, rolled: this code runs once an item, out of a cold
        // instruction cache.)
        uint8_t* to[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int r = (row & ~3) + x;
          to[x] = whole ? reinterpret_cast<uint8_t*>(out + out_row(r) * kHeadDim)
                        : reinterpret_cast<uint8_t*>(part + static_cast<int64_t>(slot) * kPartFloats + r * kHeadDim);
          to[x] += 16 * (lane & 3);
        }
        const int pieces = whole ? 4 : 8;  // of 64 bytes, in this half's 128 dims
#pragma unroll 1
        for (int i = 0; i < pieces; ++i) {
          // v[4 x ..] goes in as 16-byte piece x of this lane's row and comes out as this lane's piece of row x
          uint32_t v[16];
          if (whole) {
            float o[32];
            tmem_ld32(lanes + 128 * half + 32 * i, o);
#pragma unroll
            for (int c = 0; c < 16; ++c) v[c] = pack_bf16(o[2 * c] * inv, o[2 * c + 1] * inv);
          } else {
            tmem_ld16(lanes + 128 * half + 16 * i, v);
          }
#pragma unroll
          for (int bit = 1; bit <= 2; bit *= 2) {
            const bool up = (lane & bit) != 0;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              if (x & bit) continue;
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? v[4 * x + c] : v[4 * (x + bit) + c], bit);
                if (up) v[4 * x + c] = got;
                else v[4 * (x + bit) + c] = got;
              }
            }
          }
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if ((row & ~3) + x < w.it.rows)
              *reinterpret_cast<uint4*>(to[x] + 64 * (pieces * half + i)) =
                  make_uint4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
        }
        if (poisoned) {  // non-finite V elements taken out of the product, back where they are seen
          __syncwarp();  // the row as its four lanes stored it
          const int64_t at = out_row(row) * kHeadDim;
          float* sums = part + static_cast<int64_t>(slot) * kPartFloats + row * kHeadDim;
#pragma unroll 1
          for (int j = w.it.lo0; row < w.it.rows && j < hi; ++j) {
            if (j >= w.it.lo1 && j < w.it.hi0) j = w.it.hi0;  // (seen by all: left in the product)
            if (j >= hi || (j < lo && j >= first) || (j < first && j < w.it.hi0)) continue;
            const int r = cache_row(a.c, w.b, j);
            if (r < 0) continue;
            const __nv_bfloat16* vr = v_pool + (static_cast<int64_t>(r) * a.G + w.g) * kHeadDim;
#pragma unroll 1
            for (int d = 128 * half; d < 128 * half + 128; ++d) {
              const float x = __bfloat162float(vr[d]);
              if (isfinite(x)) continue;
              if (whole) out[at + d] = __float2bfloat16_rn(__bfloat162float(out[at + d]) + x);
              else sums[d] += x;
            }
          }
        }
        if (half == 0 && row < w.it.rows) {
          if (whole) lse[out_row(row)] = total == 0.f ? -INFINITY : (m + log2f(total)) * kLn2;
          else part_ml[slot * kRows + row] = make_float2(m, total);
        }
      }
      if (tid == 0 && w.x0 == 0 && w.x1 < w.it.n) {  // the item goes on in the ranges behind this one
        Cont ct{};
        ct.row0 = w.s.start + r0 / kHeadsPerGroup;
        ct.first = r0 % kHeadsPerGroup;
        ct.rows = w.it.rows;
        ct.g = w.g;
        const int64_t item_end = t_end - (w.x1 - w.x0) + w.it.n;  // this piece is the range's last
        ct.c_last = static_cast<int>((item_end * n_ctas - 1) / n_tiles);
        cont[blockIdx.x] = ct;
      }
      fence_before();
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kMmaS) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(512));
  if (tid == 0 && *abort_flag) cont[blockIdx.x].status = 2;
}

// Joins the parts of the items that were cut, in part order.  The blocks take units of work in turn:
// 16 rows of an item with few parts (a warp a row), one row of an item with many (few rows, a
// long cache: a sixteenth of the parts a warp).  Every block finds the units in the ranges' Conts (a grid
// of a block per possible unit took 7 us to find that there is nothing to do).  Block 0 also gathers
// the ranges' status into the call's.
constexpr int kJoinWarps = 16, kBatch = 5;
__global__ void __launch_bounds__(kJoinWarps * 32)
causal_join_kernel(const float* part, const float2* part_ml, const Cont* cont, int n_ranges, int G,
                   int* __restrict__ status, __nv_bfloat16* __restrict__ out, float* __restrict__ lse) {
  __shared__ float sO[kJoinWarps][kHeadDim];
  __shared__ float2 sMl[kJoinWarps];
  __shared__ int s_units[kMaxCtas + 1];  // units before range c's
  __shared__ int s_warp[kJoinWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  static_assert(kMaxCtas <= kJoinWarps * 32, "a thread per range");
  after_previous();
  {
    int mine = 0, bad = 0;
    if (tid < n_ranges) {
      const Cont ct = cont[tid];
      bad = ct.status;
      if (ct.rows > 0) mine = ct.c_last - tid + 1 <= kJoinWarps ? (ct.rows + kJoinWarps - 1) / kJoinWarps : ct.rows;
    }
    int up_to = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, up_to, o);
      if (lane >= o) up_to += y;
    }
    if (lane == 31) s_warp[warp] = up_to;
    bad = __syncthreads_or(bad);
    for (int w = 0; w < warp; ++w) up_to += s_warp[w];
    if (tid <= kMaxCtas) s_units[tid] = up_to - mine;
    if (blockIdx.x == 0 && tid == 0) *status = bad ? 2 : 0;
    __syncthreads();
  }
  for (int unit = blockIdx.x; unit < s_units[n_ranges]; unit += gridDim.x) {
    int c0 = 0;
    for (int o = 128; o > 0; o >>= 1)
      if (c0 + o < n_ranges && s_units[c0 + o] <= unit) c0 += o;  // the last range with units at or before it
    const Cont ct = cont[c0];
    const int n = ct.c_last - c0 + 1;  // part 0: slot (c0, 1), part i: slot (c0 + i, 0)
    auto slot = [&](int i) { return i == 0 ? 2 * c0 + 1 : 2 * (c0 + i); };
    const bool few = n <= kJoinWarps;
    const int r = few ? kJoinWarps * (unit - s_units[c0]) + warp : unit - s_units[c0];
    // this warp's sums (dims 8 lane on) of parts [a, z) of row r, against their largest maximum m
    float o[8] = {}, l = 0.f, m = -INFINITY;
    const int z = r >= ct.rows ? 0 : (few ? n : n * (warp + 1) / kJoinWarps);
    for (int a = few ? 0 : n * warp / kJoinWarps; a < z; a += kBatch) {  // a batch's reads in flight together
      float2 ml[kBatch];
      float4 u[kBatch], v[kBatch];
      float top = m;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (a + i >= z) continue;
        ml[i] = part_ml[slot(a + i) * kRows + r];
        const float4* p =
            reinterpret_cast<const float4*>(part + static_cast<int64_t>(slot(a + i)) * kPartFloats + r * kHeadDim) + 2 * lane;
        u[i] = p[0];
        v[i] = p[1];
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (a + i < z) top = fmaxf(top, ml[i].x);
      const float g = m == top ? 1.f : exp2f(m - top);
      m = top;
      l *= g;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] *= g;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (a + i >= z) continue;
        const float f = ml[i].x == -INFINITY ? 1.f : exp2f(ml[i].x - m);  // sums without a maximum are zeros or NaN
        l += ml[i].y * f;
        o[0] += u[i].x * f, o[1] += u[i].y * f, o[2] += u[i].z * f, o[3] += u[i].w * f;
        o[4] += v[i].x * f, o[5] += v[i].y * f, o[6] += v[i].z * f, o[7] += v[i].w * f;
      }
    }
    const int f = ct.first + r;
    const int64_t row = (static_cast<int64_t>(ct.row0) + f / kHeadsPerGroup) * G * kHeadsPerGroup +
                        ct.g * kHeadsPerGroup + f % kHeadsPerGroup;
    if (few) {
      if (r >= ct.rows) continue;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      *reinterpret_cast<uint4*>(out + row * kHeadDim + 8 * lane) =
          make_uint4(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv),
                     pack_bf16(o[4] * inv, o[5] * inv), pack_bf16(o[6] * inv, o[7] * inv));
      if (lane == 0) lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      continue;
    }
    __syncthreads();  // (few is the block's)
#pragma unroll
    for (int i = 0; i < 8; ++i) sO[warp][8 * lane + i] = o[i];
    if (lane == 0) sMl[warp] = make_float2(m, l);
    __syncthreads();
    if (tid >= kHeadDim) continue;
    float top = -INFINITY, total = 0.f, y = 0.f;
#pragma unroll
    for (int x = 0; x < kJoinWarps; ++x) top = fmaxf(top, sMl[x].x);
#pragma unroll
    for (int x = 0; x < kJoinWarps; ++x) {
      const float g = sMl[x].x == -INFINITY ? 1.f : exp2f(sMl[x].x - top);
      total += sMl[x].y * g;
      y += sO[x][tid] * g;
    }
    out[row * kHeadDim + tid] = __float2bfloat16_rn(total == 0.f ? 0.f : y / total);
    if (tid == 0) lse[row] = total == 0.f ? -INFINITY : (top + log2f(total)) * kLn2;
  }
}

// The pool as {64 dims, rows, four 64-dim blocks, G}: a box is rows of one page, swizzled.
bool encode_pool(CUtensorMap* map, const void* pool, uint64_t rows, int G, uint32_t box_rows, uint32_t box_blocks) {
  const auto fn = reinterpret_cast<CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                                CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                                CUtensorMapFloatOOBfill)>(tensor_map_encoder());
  if (!fn) return false;
  cuuint64_t dims[4] = {64, rows, 4, static_cast<cuuint64_t>(G)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(G) * 512, 128, 512};
  cuuint32_t box[4] = {64, box_rows, box_blocks, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(pool), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr size_t kContBytes = (kMaxCtas * sizeof(Cont) + 255) / 256 * 256;
constexpr size_t kMlBytes = 2 * kMaxCtas * kRows * sizeof(float2);

}  // namespace

size_t causal_scratch_bytes() { return kContBytes + kMlBytes + 2 * kMaxCtas * static_cast<size_t>(kPartFloats) * 4; }

cudaError_t launch_paged_causal(const void* q, const void* k_pages, const void* v_pages, const CacheView& c, int64_t T,
                                int G, int window, int sinks, float scale, int* status, void* scratch, void* out,
                                float* lse, cudaStream_t s) {
  CUtensorMap k_map, v_map;
  const uint32_t page = 1u << c.page_shift;
  const uint64_t rows = static_cast<uint64_t>(c.n_pages) << c.page_shift;
  if (!encode_pool(&k_map, k_pages, rows, G, page < kTileKeys ? page : kTileKeys, 1) ||
      !encode_pool(&v_map, v_pages, rows, G, page < 32 ? page : 32, 4))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(causal_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  uint8_t* ws = static_cast<uint8_t*>(scratch);
  Cont* cont = reinterpret_cast<Cont*>(ws);
  float2* ml = reinterpret_cast<float2*>(ws + kContBytes);
  float* part = reinterpret_cast<float*>(ws + kContBytes + kMlBytes);
  const int grid = sm_count() < kMaxCtas ? sm_count() : kMaxCtas;
  causal_kernel<<<grid, kThreads, kSmem, s>>>(k_map, v_map, static_cast<const __nv_bfloat16*>(q),
                                              static_cast<const __nv_bfloat16*>(v_pages), Args{c, T, G, window, sinks},
                                              scale * kLog2e, part, ml, cont, static_cast<__nv_bfloat16*>(out), lse);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_after(causal_join_kernel, dim3(2 * grid), kJoinWarps * 32, 0, s, static_cast<const float*>(part),
                      static_cast<const float2*>(ml), static_cast<const Cont*>(cont), grid, G, status,
                      static_cast<__nv_bfloat16*>(out), lse);
}

}  // namespace qsa
