// Attention of one new token per request over a paged key-value cache, for
// sm_100a, split over the cache's length and joined.
//
// Mathematics.  For a unit (cell, request, KV head) with g query heads:
//   s_t = scale <q, k_t>,  m = max s_t,  l = sum exp(s_t - m),
//   out = sum exp(s_t - m) v_t / l,  lse = m + ln l,
// one pass over the tokens: every warp keeps its own running (m, l, out) over
// the tiles of 16 or 32 tokens it takes and rescales when its maximum rises by
// more than weights may grow (kSlack); the warps of a CTA are joined through
// shared memory, the CTAs of a unit through a workspace and a second kernel.
//
// What bounds it: the pages' bytes.  One new token does 4 g D flops on the
// 4 D bytes (bf16) of a token, g flops a byte where the tensor pipe could
// take 250.  So every warp keeps its own ring of tiles in shared memory, filled
// by cp.async two or three tiles ahead (an SM has 100 KB and more in flight, and
// one latency of HBM at its share of the bandwidth is 50 KB), without a barrier
// between warps; keys and values are separate groups, so a tile's keys are
// replaced while its values are still used.  Rows behind a request's length
// and rows of bad pages are filled with zeros and not read.  Direct loads into
// registers, 12 warps to an SM as here, waited for a tile at a time: 781 us
// instead of 615 for 32 requests of 16384 tokens, 200 instead of 82 for 67 ragged ones
// (short runs, in turn).
//
// Measured (bytes of the pages over the time, both kernels).  Seconds long, under
// the power cap: 32 requests of 16384 tokens, 16 heads of 128 in bf16 631 us, 6.8
// TB/s; 67 ragged requests of 120000 tokens in 2 cells, 8 heads of 64 with 4
// queries in fp16 84 us, 5.9 TB/s; one request of 4113 tokens, 33.7 MB, 11 us, of
// which the join's launch and round trips are 3.  Short runs on 1 GB: pages of 1
// token 6.5 TB/s, of 24 tokens 6.2, 8 bits a value 5.9 to 6.1 with 1 and 8 queries and
// 5.4 to 5.6 with 16, where the conversion of codes (a byte permute per two) takes
// the issue slots.
// mma.sync and not tcgen05: a tile of 128 rows would be seven eighths padding and
// its results a trip to tensor memory away, and the tensor pipe is 5 to 20 % busy.
//
// Fragments (lane = 4 r + c).  Scores: m16n8k16 with the queries as A and 8
// tokens as B (ldmatrix).  The accumulator holds queries r (and r + 8) x
// tokens 2c, 2c + 1, which is the layout of the B operand of the second
// product out^T = V^T p^T: p needs no exchange.  Its A operand comes from
// ldmatrix.trans.  Weights p are used as a sum of two 16-bit floats
// (p = hi + lo up to 2^-16 p), so their rounding stays below that of a bf16
// output: with up to 4 query rows the rows r + 4 of A repeat the queries and
// their lanes take the lo part (no instruction more), otherwise a second
// product adds it.
// hi is cut towards zero, and lo is the type's smallest step at least where hi is
// not zero (weight_lo), so that an infinite value times a weight stays infinite
// (0 times infinity is NaN) while a weight of zero adds nothing.  fp16 weights are
// scaled by 2^14 so that small ones keep their bits.  A weight is so kept to 2^-16
// of itself or, if that is more, to the smallest step relative to the largest
// weight of the warp: 2^-133 in bf16, 2^-24 / 2^14 = 2^-38 in fp16.
//
// Cells that share.  Listed cells that read the same pool cell are one unit
// with all their query rows (Sets), so their pages are read once.
//
// Q8 pages.  A byte code c moved into the low half of a bf16 pattern is the
// (subnormal) bf16 c 2^-133, exactly; queries carry 2^64 and weights 2^64, so
// products are normal floats and the powers of two leave at the end.
// Scales and zero points enter per token: s = ks <q, c> + kz sum(q), and
// out = sum (p vs) c + sum p vz.
//
// Split.  The tiles of all units, in order, are dealt to the workers (one CTA
// each) in equal contiguous shares, a unit's start and end counted as the tiles
// that they cost, found by every CTA from a prefix sum of the device lengths:
// ragged lengths, few long requests and many short ones all give every SM the
// same bytes, and nothing depends on lengths the host may not know.  A worker
// meets at most one unit that began before it and one that ends behind it: two
// workspace slots each.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "loopkv_internal.cuh"

namespace loopkv {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kSms = 148;
constexpr int kMaxWorkers = kSms * 3;
constexpr int kPage = 16;             // pages of a multiple of this are FLAT (below)
constexpr int kMinTokens = 128;       // what a worker takes at least
constexpr int kUnitTokens = 384;      // tokens that a unit's start and end are worth (the largest tried)
constexpr int kEmptyTokens = 32;      // and a unit without tokens, which is only written
constexpr int kMaxRows = LOOPKV_MAX_PAGED_GROUP;  // query rows of a set
constexpr int kJoinThreads = 256;
constexpr int kFewParts = 16;         // a warp joins fewer continuations than this
constexpr int kJoinOwners = (kMaxWorkers + kFewParts - 1) / kFewParts;
constexpr int kJoinSpread = 32;       // blocks at most that share an owner's rows and channels
constexpr int kCurrentBit = 1 << 30;  // in a set's cell: the last token is in cur_k / cur_v

struct RowView {
  const uint16_t* data;
  int64_t cell, row, head;
  __device__ const uint16_t* at(int c, int r, int h) const {
    return data + c * cell + r * row + h * head;
  }
};

struct PagedDecodeParams {
  const uint8_t* k;
  const uint8_t* v;
  const float4* meta;
  const int32_t* table;
  const int32_t* len;
  RowView q, cur_k, cur_v;
  uint16_t* out;
  float* lse;
  float* part;        // [2 * workers][rows][D] partial results
  float2* stat;       // [2 * workers][rows] their maxima and sums
  int32_t* split;     // [workers][2]: a unit begun but not ended here, workers that continue it
  uint32_t* status;
  int32_t n_sets, batch, heads, group, max_pages, n_pages, workers;
  int32_t rows;       // query rows of the largest set
  uint32_t cell_rows; // token rows of a pool cell
  float scale2;       // sm_scale * log2(e)
  float unit2;        // the same for a score as the products give it (Q8: times 2^69)
  float slack;        // kSlack in those units
  PageDiv div, by_heads, by_group, by_batch;
};

// Listed cells that read the same pool cell in the same way, in sets of at
// most kMaxRows query rows: members first[s] .. first[s + 1] - 1, row i of the
// set being query row i % group of member i / group.
struct Sets {
  int32_t cell[LOOPKV_MAX_CELLS_PER_CALL];
  uint16_t first[LOOPKV_MAX_CELLS_PER_CALL + 1];
  uint16_t member[LOOPKV_MAX_CELLS_PER_CALL];  // index in the caller's list
};

template <int FMT>
struct Mma;
template <>
struct Mma<LOOPKV_PAGE_BF16> {
  static __device__ __forceinline__ void run(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
  // (lo, hi) halves of a word
  static __device__ __forceinline__ uint32_t pack(float x, float y) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ uint32_t pack_down(float x, float y) {  // towards zero
    return __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
  }
  // the lo part of weights beside their hi part
  static __device__ __forceinline__ uint32_t weight_lo(uint32_t hi, float lo0, float lo1) {
    uint32_t least, w;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(least) : "r"(hi), "r"(0x00010001u));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(w) : "r"(pack(lo0, lo1)), "r"(least));
    return w;
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
  static constexpr float kShift = 0.f;
  static constexpr float kSlack = 8.f;  // weights reach 2^8 before sums are rescaled
};
template <>
struct Mma<LOOPKV_PAGE_Q8> : Mma<LOOPKV_PAGE_BF16> {};
template <>
struct Mma<LOOPKV_PAGE_F16> {
  static __device__ __forceinline__ void run(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ uint32_t pack(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ uint32_t pack_down(float x, float y) {
    uint32_t w;
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(y), "f"(x));
    return w;
  }
  static __device__ __forceinline__ uint32_t weight_lo(uint32_t hi, float lo0, float lo1) {
    uint32_t least, w;
    asm("min.f16x2 %0, %1, %2;" : "=r"(least) : "r"(hi), "r"(0x00010001u));
    asm("max.f16x2 %0, %1, %2;" : "=r"(w) : "r"(pack(lo0, lo1)), "r"(least));
    return w;
  }
  static __device__ __forceinline__ float lo(uint32_t w) {
    return __half2float(__ushort_as_half((unsigned short)(w & 0xffffu)));
  }
  static __device__ __forceinline__ float hi(uint32_t w) {
    return __half2float(__ushort_as_half((unsigned short)(w >> 16)));
  }
  // weights are exp2(s - m + 14): 2^14 at most, and only those below 2^-28
  // of the largest lose bits to fp16's smallest step
  static constexpr float kShift = 14.f;
  static constexpr float kSlack = 0.f;  // 2^16 would be infinite
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float lse_of(float top, float sum) {
  return sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

// n / d, in 32 bits where they do (a 64-bit division is a hundred instructions)
__device__ __forceinline__ uint64_t quotient(uint64_t n, uint32_t d) {
  return (n >> 32) == 0 ? (uint32_t)n / d : n / d;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t s) {
  return __byte_perm(a, b, s);
}

__device__ __forceinline__ uint32_t shared_at(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
// 16 bytes to shared memory; `on` false: zeros, and nothing is read
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
  __syncwarp();
}
__device__ __forceinline__ void ldsm(uint32_t (&w)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldsm_trans(uint32_t (&w)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
}

// A warp's tile in shared memory: key rows, value rows, Q8: meta.  16-byte
// piece x of row t lies at piece x ^ swizzle(t), so that the 8 rows of an
// ldmatrix read 8 different banks' worth.
template <int D, int FMT, int MODE>
struct Shape {
  static constexpr bool kQ8 = FMT == LOOPKV_PAGE_Q8;
  static constexpr int kRowBytes = kQ8 ? D : 2 * D;
  static constexpr int kPieces = kRowBytes / 16;
  static constexpr int kRowsPerCopy = 32 / kPieces;    // rows one instruction of a warp copies
  // Tokens of a tile, a warp's step.  What a step costs besides its products
  // (waits, rows, maxima: some 100 instructions) is halved by 32, which took 8-bit
  // pages of 1024 ragged requests from 266 to 186 us; two such tiles of 16 bits x 128
  // channels do not fit shared memory, and the registers of 8 bits x 128
  // channels x 16 rows do not hold them (187 us with 16 tokens, 266 with 32).
  static constexpr int kTok = kRowBytes == 256 || (kQ8 && D == 128 && MODE == 2) ? 16 : 32;
  static constexpr int kCopies = kTok / kRowsPerCopy;
  static constexpr int kGroups = kTok / 8;
  static constexpr uint32_t kAll = kTok == 32 ? 0xffffffffu : 0xffffu;
  static constexpr int kSteps = D / 16;        // contraction steps of the scores
  static constexpr int kMTiles = D / 16;       // 16-channel tiles of the output
  static constexpr int kRowsBytes = kTok * kRowBytes;
  static constexpr int kTileBytes = 2 * kRowsBytes + (kQ8 ? 16 * kTok : 0);
  static constexpr int kStages = kTileBytes > 8000 ? 2 : 3;
  static constexpr int kWarpBytes = kStages * kTileBytes;
  static constexpr int kCtasPerSm = 3;
  // costs in tiles
  static constexpr int kUnitCost = kUnitTokens / kTok, kEmptyCost = kEmptyTokens / kTok, kMinCost = kMinTokens / kTok;
  static constexpr int kWorkers = kSms * kCtasPerSm;
  static __device__ __forceinline__ int swizzle(int t) { return kPieces == 4 ? (t >> 1) & 3 : t & 7; }
};

// MODE 0: up to 4 query rows, 1: 8, 2: 16.  FLAT: pages of whole runs of 16 tokens,
// so that the rows of a tile, or of each half of one of 32, follow one another.
template <int D, int FMT, int MODE, bool FLAT>
__global__ void __launch_bounds__(kThreads, Shape<D, FMT, MODE>::kCtasPerSm)
paged_decode_kernel(const __grid_constant__ PagedDecodeParams p, const __grid_constant__ Sets sets) {
  require_ieee_subnormals();
  using S = Shape<D, FMT, MODE>;
  using M = Mma<FMT>;
  constexpr bool Q8 = S::kQ8;
  constexpr int NT = MODE == 2 ? 2 : 1;      // query halves (8 columns of out^T each)
  constexpr int ROWS = 8 * NT;               // query rows a warp keeps
  constexpr int OS = D + 4;                  // floats of a row in shared memory (banks)
  static_assert(ROWS * OS * 4 <= S::kWarpBytes, "a warp's results take the place of its tiles");
  extern __shared__ __align__(256) uint8_t smem[];
  float* const sm = reinterpret_cast<float*>(smem + kWarps * S::kWarpBytes);  // [kWarps + 1][kMaxRows] maxima, factors
  float* const sl = sm + (kWarps + 1) * kMaxRows;                // sums, one over the joint one
  float* const sz = sl + (kWarps + 1) * kMaxRows;                // [kWarps][kMaxRows] zero-point sums (Q8)
  int* const prefix = reinterpret_cast<int*>(sz + kWarps * kMaxRows);  // [batch + 1] cost before a request
  __shared__ int warp_sums[kWarps];
  __shared__ int64_t out_at[kMaxRows];
  __shared__ const uint16_t* cur_at[kMaxRows];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
  uint8_t* const ring = smem + warp * S::kWarpBytes;
  const uint32_t ring_at = shared_at(ring);
  // where this lane copies to and reads from, within a row and a tile
  const int piece = lane % S::kPieces, copy_row = lane / S::kPieces;
  const int k_row = (lane & 7) + ((lane >> 4) << 3), k_piece = (lane >> 3) & 1;  // tokens 0-7 | 8-15 x 2 pieces
  const int v_row = (lane & 7) + (Q8 ? ((lane >> 3) & 1) << 3 : (lane >> 4) << 3);
  const int v_piece = Q8 ? lane >> 4 : (lane >> 3) & 1;
  // (rows begin on multiples of their size, so a later piece is an exclusive or away)
  const uint32_t k_at = k_row * S::kRowBytes + ((k_piece ^ S::swizzle(k_row)) << 4);
  const uint32_t v_at = v_row * S::kRowBytes + ((v_piece ^ S::swizzle(v_row)) << 4);
  const uint32_t page_rows = (uint32_t)p.heads * (uint32_t)p.div.size;  // (a pool's rows are numbered in 32 bits)
  uint32_t status = 0;

  {  // the constants' first lines, while the kernel before this one ends
    const int warm = sets.cell[0] + sets.first[1] + sets.member[0] + p.n_sets + p.group;
    asm volatile("" ::"r"(warm));
  }
  wait_for_previous();
  // Cost of a unit of every request: its tiles and its start and end.
  {
    const int per = (p.batch + kThreads - 1) / kThreads;
    int sum = 0;
    for (int k = 0; k < per; ++k) {
      const int b = tid * per + k;
      if (b >= p.batch) break;
      int n = p.len[b];
      if (n < 0 || n > p.max_pages * p.div.size) {
        status |= LOOPKV_PAGE_BAD_LENGTH;
        n = 0;
      }
      const int t = n == 0 ? S::kEmptyCost : S::kUnitCost + (n + S::kTok - 1) / S::kTok;
      prefix[b + 1] = t;
      sum += t;
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    int before = inc - sum;
    for (int w = 0; w < warp; ++w) before += warp_sums[w];
    if (tid == 0) prefix[0] = 0;
    for (int k = 0; k < per; ++k) {
      const int b = tid * per + k;
      if (b >= p.batch) break;
      before += prefix[b + 1];
      prefix[b + 1] = before;
    }
    __syncthreads();
  }
  const int per_request = p.n_sets * p.heads;
  const int64_t all = (int64_t)prefix[p.batch] * per_request;
  const int64_t want = (all + S::kMinCost - 1) / S::kMinCost;
  const int workers = (int)(want < p.workers ? want : p.workers);
  const int me = blockIdx.x;
  if (tid == 0) p.split[2 * me + 1] = 0;
  if (me >= workers) return;
  // shares of all / workers, the first ones one longer
  const uint64_t share = quotient((uint64_t)all, (uint32_t)workers), longer = (uint64_t)all - share * workers;
  int64_t x = (int64_t)(share * me + min((uint64_t)me, longer));
  const int64_t x1 = x + (int64_t)share + ((uint64_t)me < longer ? 1 : 0);
  int b = 0;
  {
    int lo = 0, hi = p.batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((int64_t)prefix[mid] * per_request <= x) lo = mid; else hi = mid - 1;
    }
    b = lo;
  }

  while (x < x1) {
    const int cost = prefix[b + 1] - prefix[b];
    const int64_t rem = x - (int64_t)prefix[b] * per_request;
    const int u = (int)quotient((uint64_t)rem, (uint32_t)cost), from = (int)(rem - (int64_t)u * cost);
    const int set = p.by_heads.page(u), h = u - set * p.heads;
    const int upto = (int)min((int64_t)cost, from + (x1 - x));
    const int first = sets.first[set], rows = (sets.first[set + 1] - first) * p.group;
    int n = p.len[b];
    if (n < 0 || n > p.max_pages * p.div.size) n = 0;
    x += upto - from;
    if (n == 0) {
      // written by the worker whose share has its first position
      for (int i = from == 0 ? tid : rows * (D / 8); i < rows * (D / 8); i += kThreads) {
        const int row = i / (D / 8), mem = p.by_group.page(row), li = sets.member[first + mem];
        const int64_t at = (((int64_t)li * p.batch + b) * p.heads + h) * p.group + row - mem * p.group;
        reinterpret_cast<uint4*>(p.out + at * D)[i - row * (D / 8)] = make_uint4(0, 0, 0, 0);
        if (i == row * (D / 8) && p.lse) p.lse[at] = -INFINITY;
      }
      if (x == (int64_t)prefix[b + 1] * per_request) ++b;
      continue;
    }
    // position i of a unit's cost is its tile i - S::kUnitCost
    const int tiles = cost - S::kUnitCost, t0 = max(0, from - S::kUnitCost), t1 = upto - S::kUnitCost;
    if (t1 <= 0) break;  // the share ends before the unit's first tile
    const bool current = (sets.cell[set] & kCurrentBit) != 0 && n > 0;
    const uint32_t cell_row = (uint32_t)(sets.cell[set] & ~kCurrentBit) * p.cell_rows + (uint32_t)(h * p.div.size);
    const int np = current ? n - 1 : n;  // tokens read from pages

    // The page of the lane's token of a tile (FLAT: of the first token of the
    // lane's half of it), loaded a step before the tile is copied.  A tile is then
    // a row of every lane's token (FLAT: of every half's first one) and a bit per
    // token to be read.
    const int32_t* const entry = p.table + (int64_t)b * p.max_pages;
    struct Next {
      int page, off;  // off < 0: no token of the pages
    };
    auto page_of = [&](int tile) -> Next {
      const int pos = tile * S::kTok + (lane & (FLAT ? S::kTok - 16 : S::kTok - 1));
      if (tile >= t1 || pos >= np) return {-1, -1};
      const int j = p.div.page(pos);
      return {entry[j], pos - j * p.div.size};
    };
    auto rows_of = [&](int tile, Next at, uint32_t* row) -> uint32_t {
      const bool good = at.page >= 0 && at.page < p.n_pages;
      if (!good && at.off >= 0) status |= LOOPKV_PAGE_BAD_PAGE;
      *row = good ? cell_row + (uint32_t)at.page * page_rows + (uint32_t)at.off : 0u;
      const uint32_t found = __ballot_sync(0xffffffffu, good) & S::kAll;
      const int left = np - tile * S::kTok;
      return FLAT && left < S::kTok ? found & ((1u << max(left, 0)) - 1u) : found;
    };
    auto copy_rows = [&](uint32_t at, const uint8_t* src, uint32_t row, uint32_t bits) {
      at += copy_row * S::kRowBytes;
      src += 16 * piece;
      auto dst = [&](int t) { return at + t * S::kRowBytes + ((piece ^ S::swizzle(t + copy_row)) << 4); };
      if constexpr (FLAT) {
        const uint8_t* half[S::kTok / 16];
#pragma unroll
        for (int h = 0; h < S::kTok / 16; ++h)
          half[h] = src + ((uint64_t)(S::kTok == 16 ? row : __shfl_sync(0xffffffffu, row, 16 * h)) + copy_row) * S::kRowBytes;
        auto from = [&](int t) { return half[t / 16] + t % 16 * S::kRowBytes; };
        if (bits == S::kAll) {
#pragma unroll
          for (int i = 0; i < S::kCopies; ++i) copy16(dst(i * S::kRowsPerCopy), from(i * S::kRowsPerCopy));
        } else {
          bits >>= copy_row;
#pragma unroll
          for (int i = 0; i < S::kCopies; ++i)
            copy16(dst(i * S::kRowsPerCopy), from(i * S::kRowsPerCopy), (bits >> (i * S::kRowsPerCopy) & 1) != 0);
        }
      } else {
        bits >>= copy_row;
#pragma unroll
        for (int i = 0; i < S::kCopies; ++i) {
          const uint32_t from = __shfl_sync(0xffffffffu, row, i * S::kRowsPerCopy + copy_row);
          copy16(dst(i * S::kRowsPerCopy), src + (uint64_t)from * S::kRowBytes, (bits >> (i * S::kRowsPerCopy) & 1) != 0);
        }
      }
    };
    auto copy_keys = [&](int stage, uint32_t row, uint32_t bits) {
      const uint32_t at = ring_at + stage * S::kTileBytes;
      copy_rows(at, p.k, row, bits);
      if (Q8 && lane < S::kTok)
        copy16(at + 2 * S::kRowsBytes + 16 * lane,
               reinterpret_cast<const uint8_t*>(p.meta + (row + (FLAT ? (uint64_t)(lane & 15) : 0))),
               (bits >> lane & 1) != 0);
      copy_commit();
    };
    auto copy_values = [&](int stage, uint32_t row, uint32_t bits) {
      copy_rows(ring_at + stage * S::kTileBytes + S::kRowsBytes, p.v, row, bits);
      copy_commit();
    };

    // The first tiles' pages, the query fragments (asked for before the tiles: at
    // the start of a call every SM's copies are in the way of what comes behind
    // them), and the tiles' copies; valid[0] is this step's.
    uint32_t qa[S::kSteps][MODE == 2 ? 4 : 2], valid[S::kStages];
    Next next;
    {
      Next pages[S::kStages];
#pragma unroll
      for (int s = 0; s < S::kStages; ++s) pages[s] = page_of(t0 + warp + s * kWarps);
      next = page_of(t0 + warp + S::kStages * kWarps);
#pragma unroll
      for (int half = 0; half < NT; ++half) {
        const int row = MODE == 0 ? (r & 3) : r + 8 * half;
        const bool on = row < rows;
        const int mem = on ? p.by_group.page(row) : 0;
        const uint16_t* src = p.q.at(sets.member[first + mem], b, h * p.group + (on ? row - mem * p.group : 0));
#pragma unroll
        for (int i = 0; i < S::kSteps; ++i) {
          uint2 w = make_uint2(0, 0);
          if (on) {
            if constexpr (!Q8)
              w = make_uint2(*reinterpret_cast<const uint32_t*>(src + 16 * i + 2 * c),
                             *reinterpret_cast<const uint32_t*>(src + 16 * i + 8 + 2 * c));
            else  // a lane's 4 codes of a 16-byte piece are channels 4 c ..
              w = *reinterpret_cast<const uint2*>(src + 16 * i + 4 * c);
          }
          qa[i][MODE == 2 ? half : 0] = w.x;
          qa[i][MODE == 2 ? 2 + half : 1] = w.y;
        }
      }
#pragma unroll
      for (int s = 0; s < S::kStages; ++s) {
        uint32_t row;
        const uint32_t bits = rows_of(t0 + warp + s * kWarps, pages[s], &row);
        copy_keys(s, row, bits);
        copy_values(s, row, bits);
        valid[s] = bits;
      }
    }

    float qsum[NT];
#pragma unroll
    for (int half = 0; half < NT; ++half) {
      qsum[half] = 0.f;
      if constexpr (Q8) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < S::kSteps; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t& w = qa[i][MODE == 2 ? 2 * k + half : k];
            sum += M::lo(w) + M::hi(w);
            w = M::pack(M::lo(w) * 0x1p64f, M::hi(w) * 0x1p64f);
          }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        qsum[half] = sum * 0x1p-69f;
      }
    }

    float o[NT][S::kMTiles][4];
    // running maximum in units of the products, minus it in log2 units, sums
    float m[NT], low[NT], l[NT], z[NT];
#pragma unroll
    for (int half = 0; half < NT; ++half) {
      m[half] = -INFINITY;
      low[half] = l[half] = z[half] = 0.f;
#pragma unroll
      for (int j = 0; j < S::kMTiles; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[half][j][k] = 0.f;
    }

    int stage = 0;
    for (int tile = t0 + warp; tile < t1; tile += kWarps) {
      const uint32_t keys = ring_at + stage * S::kTileBytes, values = keys + S::kRowsBytes;
      copy_wait<2 * S::kStages - 1>();

      // Scores.
      float s[S::kGroups][4];
#pragma unroll
      for (int g = 0; g < S::kGroups; ++g) s[g][0] = s[g][1] = s[g][2] = s[g][3] = 0.f;
      auto score = [&](int g, int ks, uint32_t b0, uint32_t b1) {
        if constexpr (MODE == 2) M::run(s[g], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], b0, b1);
        else M::run(s[g], qa[ks][0], 0u, qa[ks][1], 0u, b0, b1);
      };
#pragma unroll
      for (int i = 0; i < S::kPieces / 2; ++i)
#pragma unroll
        for (int h = 0; h < S::kGroups; h += 2) {
          uint32_t w[4];  // tokens 0-7 of the half: pieces 2 i, 2 i + 1; tokens 8-15: the same
          ldsm(w, ((keys + k_at) ^ (i << 5)) + 8 * h * S::kRowBytes);
          if constexpr (Q8) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              score(h + (k >> 1), 2 * i + (k & 1), prmt(w[k], 0, 0x4140), prmt(w[k], 0, 0x4342));
          } else {
            score(h, i, w[0], w[1]);
            score(h + 1, i, w[2], w[3]);
          }
        }
      float4 meta[S::kGroups][2];
      if constexpr (Q8) {
        const float4* src = reinterpret_cast<const float4*>(ring + stage * S::kTileBytes + 2 * S::kRowsBytes);
#pragma unroll
        for (int g = 0; g < S::kGroups; ++g)
#pragma unroll
          for (int k = 0; k < 2; ++k) meta[g][k] = src[2 * c + k + 8 * g];
      }
      const uint32_t bits = valid[0];
      __syncwarp();
      const int ahead = tile + S::kStages * kWarps;
      uint32_t row;
      const uint32_t ahead_bits = rows_of(ahead, next, &row);
      next = page_of(ahead + kWarps);
      copy_keys(stage, row, ahead_bits);
#pragma unroll
      for (int i = 0; i + 1 < S::kStages; ++i) valid[i] = valid[i + 1];
      valid[S::kStages - 1] = ahead_bits;

      // Weights, two tokens of every 8 of a query row per lane.
      uint32_t ph[NT][S::kGroups], pl[NT][S::kGroups];
#pragma unroll
      for (int half = 0; half < NT; ++half) {
        float e[S::kGroups][2], top = -INFINITY;
#pragma unroll
        for (int g = 0; g < S::kGroups; ++g)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            e[g][k] = s[g][2 * half + k];
            if constexpr (Q8) e[g][k] = fmaf(e[g][k], meta[g][k].x, meta[g][k].y * qsum[half]);
          }
        if (bits != S::kAll) {
#pragma unroll
          for (int g = 0; g < S::kGroups; ++g)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              if ((bits >> (2 * c + k + 8 * g) & 1) == 0) e[g][k] = -INFINITY;
        }
#pragma unroll
        for (int g = 0; g < S::kGroups; ++g) top = fmaxf(top, fmaxf(e[g][0], e[g][1]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float high = fmaxf(m[half], top);
        if (__any_sync(0xffffffffu, high > m[half] + p.slack)) {
          // a first maximum scales sums that are still zero
          const float next_low = high == -INFINITY ? 0.f : fmaf(-high, p.unit2, M::kShift);
          const float a = m[half] == -INFINITY ? 0.f : exp2_fast(next_low - low[half]);
          m[half] = high;
          low[half] = next_low;
          l[half] *= a;
          if constexpr (Q8) z[half] *= a;
          const float a0 = __shfl_sync(0xffffffffu, a, 8 * c), a1 = __shfl_sync(0xffffffffu, a, 8 * c + 4);
#pragma unroll
          for (int j = 0; j < S::kMTiles; ++j) {
            o[half][j][0] *= a0;
            o[half][j][1] *= a1;
            o[half][j][2] *= a0;
            o[half][j][3] *= a1;
          }
        }
#pragma unroll
        for (int g = 0; g < S::kGroups; ++g)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            e[g][k] = exp2_fast(fmaf(e[g][k], p.unit2, low[half]));
            l[half] += e[g][k];
            if constexpr (Q8) {
              z[half] = fmaf(e[g][k], meta[g][k].w, z[half]);
              e[g][k] *= meta[g][k].z * 0x1p64f;
            }
          }
#pragma unroll
        for (int g = 0; g < S::kGroups; ++g) {
          ph[half][g] = M::pack_down(e[g][0], e[g][1]);
          const float lo0 = e[g][0] - M::lo(ph[half][g]), lo1 = e[g][1] - M::hi(ph[half][g]);
          pl[half][g] = Q8 ? M::pack(lo0, lo1) : M::weight_lo(ph[half][g], lo0, lo1);  // (codes are finite)
          if (MODE == 0 && r >= 4) ph[half][g] = pl[half][g];
        }
      }

      // out^T += V^T p^T
      copy_wait<2 * S::kStages - 1>();
#pragma unroll
      for (int i = 0; i < S::kPieces / 2; ++i)
#pragma unroll
        for (int h = 0; h < S::kGroups; h += 2) {
          uint32_t w[4];
          ldsm_trans(w, ((values + v_at) ^ (i << 5)) + 8 * h * S::kRowBytes);
          if constexpr (!Q8) {
            // tile i: rows r, r + 8 are channels 16 i + r, 16 i + 8 + r
#pragma unroll
            for (int half = 0; half < NT; ++half) {
              M::run(o[half][i], w[0], w[1], w[2], w[3], ph[half][h], ph[half][h + 1]);
              if constexpr (MODE != 0) M::run(o[half][i], w[0], w[1], w[2], w[3], pl[half][h], pl[half][h + 1]);
            }
          } else {
            // tile j: rows r, r + 8 are channels 16 j + 2 r, 16 j + 2 r + 1, the
            // low and the high bytes of a pair
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int j = 2 * i + k;
              const uint32_t a0 = prmt(w[2 * k], 0, 0x4240), a1 = prmt(w[2 * k], 0, 0x4341);
              const uint32_t a2 = prmt(w[2 * k + 1], 0, 0x4240), a3 = prmt(w[2 * k + 1], 0, 0x4341);
#pragma unroll
              for (int half = 0; half < NT; ++half) {
                M::run(o[half][j], a0, a1, a2, a3, ph[half][h], ph[half][h + 1]);
                if constexpr (MODE != 0) M::run(o[half][j], a0, a1, a2, a3, pl[half][h], pl[half][h + 1]);
              }
            }
          }
        }
      __syncwarp();
      copy_values(stage, row, ahead_bits);
      stage = stage + 1 == S::kStages ? 0 : stage + 1;
    }
    copy_wait<0>();  // empty groups only

    // Join the warps.
    float* const so = reinterpret_cast<float*>(ring);
    auto so_of = [&](int w) { return reinterpret_cast<const float*>(smem + w * S::kWarpBytes); };
#pragma unroll
    for (int half = 0; half < NT; ++half) {
      l[half] += __shfl_xor_sync(0xffffffffu, l[half], 1);
      l[half] += __shfl_xor_sync(0xffffffffu, l[half], 2);
      if constexpr (Q8) {
        z[half] += __shfl_xor_sync(0xffffffffu, z[half], 1);
        z[half] += __shfl_xor_sync(0xffffffffu, z[half], 2);
      }
      if (c == 0) {
        sm[warp * kMaxRows + r + 8 * half] = m[half] == -INFINITY ? -INFINITY : -low[half];
        sl[warp * kMaxRows + r + 8 * half] = l[half];
        if constexpr (Q8) sz[warp * kMaxRows + r + 8 * half] = z[half];
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float* dst = so + (2 * c + k + 8 * half) * OS;
#pragma unroll
        for (int j = 0; j < S::kMTiles; ++j) {
          if constexpr (!Q8) {
            dst[16 * j + r] = o[half][j][k];
            dst[16 * j + 8 + r] = o[half][j][2 + k];
          } else {
            *reinterpret_cast<float2*>(dst + 16 * j + 2 * r) =
                make_float2(o[half][j][k] * 0x1p69f, o[half][j][2 + k] * 0x1p69f);
          }
        }
      }
    }
    const bool with_current = current && t1 == tiles;
    if (with_current) {
      for (int i = warp; i < rows; i += kWarps) {
        const int mem = p.by_group.page(i), li = sets.member[first + mem];
        const uint16_t* q = p.q.at(li, b, h * p.group + i - mem * p.group);
        const uint16_t* k = p.cur_k.at(li, b, h);
        float dot = 0.f;
        for (int d = 2 * lane; d < D; d += 64) {
          const uint32_t a = *reinterpret_cast<const uint32_t*>(q + d);
          const uint32_t w = *reinterpret_cast<const uint32_t*>(k + d);
          dot = fmaf(M::lo(a), M::lo(w), dot);
          dot = fmaf(M::hi(a), M::hi(w), dot);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
        if (lane == 0) sm[kWarps * kMaxRows + i] = dot * p.scale2;
      }
    }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == tiles;
    const int slot = 2 * me + (t0 == 0 ? 1 : 0);
    if (tid < rows) {
      // factors of the warps' sums in the place of their maxima, one over the
      // joint sum in sl[i]
      float top = with_current ? sm[kWarps * kMaxRows + tid] : -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w * kMaxRows + tid]);
      const float base = top == -INFINITY ? 0.f : top;
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2_fast(sm[w * kMaxRows + tid] - base);
        sum = fmaf(f, sl[w * kMaxRows + tid], sum);
        sm[w * kMaxRows + tid] = f;
      }
      if (with_current) {
        const float f = exp2_fast(sm[kWarps * kMaxRows + tid] - base);
        sum += f;
        sm[kWarps * kMaxRows + tid] = f;
      }
      const int mem = p.by_group.page(tid), li = sets.member[first + mem];
      const int64_t to = (((int64_t)li * p.batch + b) * p.heads + h) * p.group + tid - mem * p.group;
      out_at[tid] = whole ? to * D : ((int64_t)slot * p.rows + tid) * D;
      cur_at[tid] = with_current ? p.cur_v.at(li, b, h) : nullptr;
      sl[tid] = sum == 0.f ? 0.f : 1.f / sum;
      if (!whole) p.stat[slot * p.rows + tid] = make_float2(top, sum);
      else if (p.lse) p.lse[to] = lse_of(top, sum);
    }
    __syncthreads();
    for (int idx = tid; idx < rows * (D / 4); idx += kThreads) {
      const int i = idx / (D / 4), d = 4 * (idx - i * (D / 4));
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = sm[w * kMaxRows + i];
        float4 y = *reinterpret_cast<const float4*>(so_of(w) + i * OS + d);
        if constexpr (MODE == 0) {
          const float4 lo = *reinterpret_cast<const float4*>(so_of(w) + (i + 4) * OS + d);
          y = make_float4(y.x + lo.x, y.y + lo.y, y.z + lo.z, y.w + lo.w);
        }
        if constexpr (Q8) {
          const float zero = sz[w * kMaxRows + i];
          y = make_float4(y.x + zero, y.y + zero, y.z + zero, y.w + zero);
        }
        acc = make_float4(fmaf(f, y.x, acc.x), fmaf(f, y.y, acc.y), fmaf(f, y.z, acc.z), fmaf(f, y.w, acc.w));
      }
      if (with_current) {
        const float f = sm[kWarps * kMaxRows + i];
        const uint2 w = *reinterpret_cast<const uint2*>(cur_at[i] + d);
        acc = make_float4(fmaf(f, M::lo(w.x), acc.x), fmaf(f, M::hi(w.x), acc.y), fmaf(f, M::lo(w.y), acc.z), fmaf(f, M::hi(w.y), acc.w));
      }
      if (whole) {
        const float f = sl[i];
        const bool none = f == 0.f;
        *reinterpret_cast<uint2*>(p.out + out_at[i] + d) =
            make_uint2(none ? 0u : M::pack(acc.x * f, acc.y * f), none ? 0u : M::pack(acc.z * f, acc.w * f));
      } else {
        *reinterpret_cast<float4*>(p.part + out_at[i] + d) = acc;
      }
    }
    if (!whole && t0 == 0 && tid == 0) {
      // the workers behind this one that hold the rest of the unit
      const int64_t last = x - upto + cost - 1;
      p.split[2 * me] = (set * p.batch + b) * p.heads + h;
      const uint64_t at = (uint64_t)last, head = longer * (share + 1);
      p.split[2 * me + 1] = (int)(at < head ? at / (share + 1) : longer + (at - head) / share) - me;
    }
    __syncthreads();  // shared memory is free for the next unit
    if (x == (int64_t)prefix[b + 1] * per_request) ++b;
  }
  if (status && p.status) atomicOr(p.status, status);
}

// Where a row of a unit goes.
__device__ __forceinline__ int64_t out_row(const PagedDecodeParams& p, const Sets& sets, int unit, int row) {
  const int sb = p.by_heads.page(unit), h = unit - sb * p.heads, set = p.by_batch.page(sb), b = sb - set * p.batch;
  const int first = sets.first[set], mem = p.by_group.page(row);
  if (first + mem >= sets.first[set + 1]) return -1;  // a smaller set
  return (((int64_t)sets.member[first + mem] * p.batch + b) * p.heads + h) * p.group + row - mem * p.group;
}

// Join the parts of the units that a worker i began and did not end: its own
// (slot 2 i + 1) and those of the workers behind it (slots 2 (i + k)).  What is
// joined is one query row of such a unit; with up to kFewParts parts it is a
// warp's work.  More are a block's, 32 channels at a time: all parts' maxima and
// sums and four channels of up to four parts to a thread at once, then the
// rest.  Owners of units of that many parts are kFewParts workers apart and more,
// so every kFewParts workers have one at most, found by a look at their
// entries.  What bounds it: two dependent round trips to L2 and, as in any
// short kernel, its start.  With a running maximum over the parts and one thread a
// channel 2 units of 300 parts took 17 us, with a block per worker and row 2000
// rows of 2 parts took 8.
template <int D, int FMT>
__global__ void __launch_bounds__(kJoinThreads)
paged_join_kernel(const __grid_constant__ PagedDecodeParams p, const __grid_constant__ Sets sets) {
  require_ieee_subnormals();
  using M = Mma<FMT>;
  constexpr int WARPS = kJoinThreads / 32, LANES = D / 4, CHUNKS = D / 32, GROUPS = kJoinThreads / 8;
  constexpr int PER = (kMaxWorkers + kJoinThreads - 1) / kJoinThreads, FIRST = 4;
  static_assert(GROUPS == 32, "a group a lane");
  __shared__ float factor[kMaxWorkers], wm[WARPS], wl[WARPS];
  __shared__ float4 sa[GROUPS][8 + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  wait_for_previous();
  const int2* const split = reinterpret_cast<const int2*>(p.split);
  auto slot = [&](int i, int k) { return k == 0 ? 2 * i + 1 : 2 * (i + k); };
  auto part = [&](int i, int k, int row) {
    return reinterpret_cast<const float4*>(p.part + ((int64_t)slot(i, k) * p.rows + row) * D);
  };
  auto add = [](float4& acc, float f, const float4& a) {
    acc = make_float4(fmaf(f, a.x, acc.x), fmaf(f, a.y, acc.y), fmaf(f, a.z, acc.z), fmaf(f, a.w, acc.w));
  };
  auto store = [&](int64_t at, const float4& acc, float sum) {
    const bool none = sum == 0.f;
    *reinterpret_cast<uint2*>(p.out + at) = make_uint2(none ? 0u : M::pack(acc.x / sum, acc.y / sum),
                                                       none ? 0u : M::pack(acc.z / sum, acc.w / sum));
  };

  const int few = blockIdx.x % kJoinOwners, w0 = few * kFewParts + lane;
  const int2 seen = lane < kFewParts && w0 < p.workers ? split[w0] : make_int2(0, 0);
  const uint32_t many = __ballot_sync(0xffffffffu, seen.y >= kFewParts);
  if (many != 0) {
    const int from = __ffs(many) - 1, i = few * kFewParts + from;
    const int unit = __shfl_sync(0xffffffffu, seen.x, from), more = __shfl_sync(0xffffffffu, seen.y, from);
    for (int it = blockIdx.x / kJoinOwners; it < p.rows * CHUNKS; it += gridDim.x / kJoinOwners) {
      const int row = it / CHUNKS, chunk = it % CHUNKS;
      const int64_t to = out_row(p, sets, unit, row);
      if (to < 0) continue;
      const int lane4 = tid % 8, group = tid / 8;
      float2 mine[PER];
      float4 a[FIRST];
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int k = tid + j * kJoinThreads;
        mine[j] = k <= more ? p.stat[slot(i, k) * p.rows + row] : make_float2(-INFINITY, 0.f);
      }
#pragma unroll
      for (int j = 0; j < FIRST; ++j) {
        const int k = group + j * GROUPS;
        a[j] = k <= more ? part(i, k, row)[8 * chunk + lane4] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int j = 0; j < PER; ++j) top = fmaxf(top, mine[j].x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (lane == 0) wm[warp] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < WARPS; ++w) top = fmaxf(top, wm[w]);
      const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int k = tid + j * kJoinThreads;
        const float f = exp2_fast(mine[j].x - base);
        if (k <= more) factor[k] = f;
        sum = fmaf(f, mine[j].y, sum);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) wl[warp] = sum;
      __syncthreads();
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int j = 0; j < FIRST; ++j)
        if (group + j * GROUPS <= more) add(acc, factor[group + j * GROUPS], a[j]);
#pragma unroll 4
      for (int k = group + FIRST * GROUPS; k <= more; k += GROUPS) add(acc, factor[k], part(i, k, row)[8 * chunk + lane4]);
      sa[group][lane4] = acc;
      __syncthreads();
      acc = sa[lane][warp];  // four channels of a group: a warp sums them over the groups
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        acc.x += __shfl_xor_sync(0xffffffffu, acc.x, o);
        acc.y += __shfl_xor_sync(0xffffffffu, acc.y, o);
        acc.z += __shfl_xor_sync(0xffffffffu, acc.z, o);
        acc.w += __shfl_xor_sync(0xffffffffu, acc.w, o);
      }
      sum = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) sum += wl[w];
      if (lane == 0) store(to * D + 32 * chunk + 4 * warp, acc, sum);
      if (tid == 0 && chunk == 0 && p.lse) p.lse[to] = lse_of(top, sum);
      __syncthreads();  // shared memory is free for the next row
    }
  }

  for (int it = blockIdx.x * WARPS + warp; it < p.workers * p.rows; it += gridDim.x * WARPS) {
    const int i = it / p.rows, row = it - i * p.rows;
    const int2 own = split[i];
    const int more = own.y;
    if (more == 0 || more >= kFewParts) continue;
    const int64_t to = out_row(p, sets, own.x, row);
    if (to < 0) continue;
    // 32 / LANES parts at a time, the first ones before the factors are known
    const int lane4 = lane % LANES, k1 = lane / LANES;
    float4 a[FIRST];
    const float2 mine = lane <= more ? p.stat[slot(i, lane) * p.rows + row] : make_float2(-INFINITY, 0.f);
#pragma unroll
    for (int j = 0; j < FIRST; ++j) {
      const int k = k1 + j * (32 / LANES);
      a[j] = k <= more ? part(i, k, row)[lane4] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float top = mine.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float f = exp2_fast(mine.x - (top == -INFINITY ? 0.f : top));
    float sum = f * mine.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < FIRST; ++j) {
      const int k = k1 + j * (32 / LANES);
      const float g = __shfl_sync(0xffffffffu, f, k);
      if (k <= more) add(acc, g, a[j]);
    }
    for (int k0 = FIRST * (32 / LANES); k0 <= more; k0 += 32 / LANES) {
      const int k = k0 + k1;
      const float g = __shfl_sync(0xffffffffu, f, k);
      if (k <= more) add(acc, g, part(i, k, row)[lane4]);
    }
#pragma unroll
    for (int o = 16; o >= LANES; o >>= 1) {
      acc.x += __shfl_xor_sync(0xffffffffu, acc.x, o);
      acc.y += __shfl_xor_sync(0xffffffffu, acc.y, o);
      acc.z += __shfl_xor_sync(0xffffffffu, acc.z, o);
      acc.w += __shfl_xor_sync(0xffffffffu, acc.w, o);
    }
    if (lane < LANES) store(to * D + 4 * lane, acc, sum);
    if (lane == 0 && p.lse) p.lse[to] = lse_of(top, sum);
  }
}

size_t work_bytes_of(int D) {
  return sizeof(float) * 2 * (size_t)kMaxWorkers * kMaxRows * (D + 2) + sizeof(int32_t) * 2 * kMaxWorkers;  // part, stat, split
}

template <int D, int FMT, int MODE, bool FLAT>
loopkv_status launch_decode_kernel(PagedDecodeParams p, const Sets& sets, cudaStream_t stream) {
  using S = Shape<D, FMT, MODE>;
  p.workers = S::kWorkers;
  auto smem = [](int batch) {
    return kWarps * S::kWarpBytes + sizeof(float) * (3 * kWarps + 2) * kMaxRows + sizeof(int) * ((size_t)batch + 1);
  };
  const auto kernel = paged_decode_kernel<D, FMT, MODE, FLAT>;
  if (!allow_shared(kernel, smem(LOOPKV_MAX_PAGED_BATCH))) return LOOPKV_ERR_CUDA;
  const loopkv_status rc = launch_early(kernel, dim3((unsigned)p.workers), kThreads, smem(p.batch), stream, p, sets);
  if (rc != LOOPKV_OK) return rc;
  const int blocks = kJoinOwners * std::min(kJoinSpread, p.rows * (D / 32));
  return launch_early(paged_join_kernel<D, FMT>, dim3((unsigned)blocks), kJoinThreads, 0, stream, p, sets);
}

template <int D, int FMT, int MODE>
loopkv_status launch_decode_mode(const PagedDecodeParams& p, const Sets& sets, cudaStream_t stream) {
  return p.div.size % kPage == 0 ? launch_decode_kernel<D, FMT, MODE, true>(p, sets, stream)
                                 : launch_decode_kernel<D, FMT, MODE, false>(p, sets, stream);
}

template <int D, int FMT>
loopkv_status launch_decode_format(const PagedDecodeParams& p, const Sets& sets, cudaStream_t stream) {
  if (p.rows <= 4) return launch_decode_mode<D, FMT, 0>(p, sets, stream);
  if (p.rows <= 8) return launch_decode_mode<D, FMT, 1>(p, sets, stream);
  return launch_decode_mode<D, FMT, 2>(p, sets, stream);
}

template <int D>
loopkv_status launch_decode_dim(int format, const PagedDecodeParams& p, const Sets& sets,
                                cudaStream_t stream) {
  switch (format) {
    case LOOPKV_PAGE_BF16: return launch_decode_format<D, LOOPKV_PAGE_BF16>(p, sets, stream);
    case LOOPKV_PAGE_F16: return launch_decode_format<D, LOOPKV_PAGE_F16>(p, sets, stream);
    default: return launch_decode_format<D, LOOPKV_PAGE_Q8>(p, sets, stream);
  }
}

bool desc_ok(const loopkv_page_pool* pool, const loopkv_paged_desc* d) {
  return d != nullptr && d->batch >= 1 && d->batch <= LOOPKV_MAX_PAGED_BATCH && d->max_pages >= 1 &&
         (int64_t)d->max_pages * pool->page_size <= LOOPKV_MAX_PAGED_TOKENS && d->q_per_kv >= 1 &&
         d->q_per_kv <= LOOPKV_MAX_PAGED_GROUP && std::isfinite(d->sm_scale);
}

RowView view(const loopkv_rows* r) {
  return {static_cast<const uint16_t*>(r->data), r->cell_stride, r->row_stride, r->head_stride};
}

}  // namespace
}  // namespace loopkv

using namespace loopkv;

extern "C" loopkv_status loopkv_paged_workspace(const loopkv_page_pool* pool,
                                                const loopkv_paged_desc* desc, size_t* bytes) {
  if (bytes == nullptr || !pool_ok(pool) || !desc_ok(pool, desc)) return LOOPKV_ERR_INVALID_ARG;
  *bytes = work_bytes_of(pool->head_dim);
  return LOOPKV_OK;
}

extern "C" loopkv_status loopkv_paged_decode(const loopkv_page_pool* pool, const loopkv_paged_desc* desc,
                                             const int32_t* h_cells, const uint8_t* h_current,
                                             int32_t n_cells, const int32_t* d_table,
                                             const int32_t* d_len, const loopkv_rows* q,
                                             const loopkv_rows* cur_k, const loopkv_rows* cur_v,
                                             void* d_out, float* d_lse, void* d_work,
                                             size_t work_bytes, uint32_t* d_status, void* stream) {
  if (!pool_ok(pool) || !desc_ok(pool, desc) || h_cells == nullptr) return LOOPKV_ERR_INVALID_ARG;
  if (n_cells < 1 || n_cells > LOOPKV_MAX_CELLS_PER_CALL) return LOOPKV_ERR_INVALID_ARG;
  auto aligned4 = [](const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 3u) == 0; };
  if (d_table == nullptr || d_len == nullptr || d_out == nullptr || d_work == nullptr || !rows_ok(q))
    return LOOPKV_ERR_INVALID_ARG;
  if (!aligned4(d_table) || !aligned4(d_len) || !aligned16(d_out) || !aligned4(d_lse) ||
      !aligned16(d_work) || !aligned4(d_status))
    return LOOPKV_ERR_INVALID_ARG;
  if (work_bytes < work_bytes_of(pool->head_dim)) return LOOPKV_ERR_INVALID_ARG;
  // Listed cells that read the same tokens are sets: their pages are read once.
  if (pool->n_cells >= kCurrentBit) return LOOPKV_ERR_INVALID_ARG;
  Sets sets{};
  const int most = kMaxRows / desc->q_per_kv;  // members of a set
  int n_sets = 0, largest = 0, place = 0;
  bool any_current = false, taken[LOOPKV_MAX_CELLS_PER_CALL] = {};
  auto key = [&](int i) { return h_cells[i] | (h_current != nullptr && h_current[i] != 0 ? kCurrentBit : 0); };
  for (int i = 0; i < n_cells; ++i)
    if (h_cells[i] < 0 || h_cells[i] >= pool->n_cells) return LOOPKV_ERR_INVALID_ARG;
  for (int i = 0; i < n_cells; ++i) {
    if (taken[i]) continue;
    const int cell = key(i);
    int size = 0;
    sets.cell[n_sets] = cell;
    sets.first[n_sets] = (uint16_t)place;
    for (int j = i; j < n_cells && size < most; ++j) {
      if (taken[j] || key(j) != cell) continue;
      taken[j] = true;
      sets.member[place++] = (uint16_t)j;
      ++size;
    }
    ++n_sets;
    largest = std::max(largest, size);
    any_current = any_current || (cell & kCurrentBit) != 0;
  }
  sets.first[n_sets] = (uint16_t)place;
  if (any_current && (!rows_ok(cur_k) || !rows_ok(cur_v))) return LOOPKV_ERR_INVALID_ARG;
  // units are numbered in 32 bits
  if ((int64_t)n_cells * desc->batch * pool->n_kv_heads >= (1LL << 31)) return LOOPKV_ERR_INVALID_ARG;
  PagedDecodeParams p{};
  p.k = static_cast<const uint8_t*>(pool->k);
  p.v = static_cast<const uint8_t*>(pool->v);
  p.meta = reinterpret_cast<const float4*>(pool->meta);
  p.table = d_table;
  p.len = d_len;
  p.q = view(q);
  if (any_current) {
    p.cur_k = view(cur_k);
    p.cur_v = view(cur_v);
  }
  p.out = static_cast<uint16_t*>(d_out);
  p.lse = d_lse;
  p.part = static_cast<float*>(d_work);
  p.stat = reinterpret_cast<float2*>(p.part + 2 * (size_t)kMaxWorkers * kMaxRows * pool->head_dim);
  p.split = reinterpret_cast<int32_t*>(p.stat + 2 * (size_t)kMaxWorkers * kMaxRows);
  p.status = d_status;
  p.n_sets = n_sets;
  p.rows = largest * desc->q_per_kv;
  p.batch = desc->batch;
  p.heads = pool->n_kv_heads;
  p.group = desc->q_per_kv;
  p.max_pages = desc->max_pages;
  p.n_pages = pool->n_pages;
  p.cell_rows = (uint32_t)((int64_t)pool->n_pages * pool->n_kv_heads * pool->page_size);
  const float sm_scale = desc->sm_scale > 0.f ? desc->sm_scale : 1.0f / std::sqrt((float)pool->head_dim);
  p.scale2 = sm_scale * 1.4426950408889634f;
  const bool q8 = pool->format == LOOPKV_PAGE_Q8;
  p.unit2 = q8 ? p.scale2 * 0x1p69f : p.scale2;
  if (!std::isfinite(p.unit2)) return LOOPKV_ERR_INVALID_ARG;
  // (finite: the first maximum is -infinity)
  const bool f16 = pool->format == LOOPKV_PAGE_F16;
  p.slack = std::min((f16 ? Mma<LOOPKV_PAGE_F16>::kSlack : Mma<LOOPKV_PAGE_BF16>::kSlack) / p.unit2, 1e30f);
  p.div = PageDiv(pool->page_size);
  p.by_heads = PageDiv(p.heads);
  p.by_group = PageDiv(p.group);
  p.by_batch = PageDiv(p.batch);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return pool->head_dim == 64 ? launch_decode_dim<64>(pool->format, p, sets, s)
                              : launch_decode_dim<128>(pool->format, p, sets, s);
}
