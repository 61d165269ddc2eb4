// Attention of one new token per request over a paged key-value cache, for
// sm_100a, split over the cache's length and joined.
//
// Mathematics.  For a unit (cell, request, KV head) with g query heads:
//   s_t = scale <q, k_t>,  m = max s_t,  l = sum exp(s_t - m),
//   out = sum exp(s_t - m) v_t / l,  lse = m + ln l,
// one pass over the tokens: every warp keeps its own running (m, l, out) over
// the 16-token tiles it takes and rescales when its maximum rises; the
// warps of a CTA are joined through shared memory, the CTAs of a unit through
// a workspace and a second kernel.  Scores are kept in log2 units.
//
// What bounds it: the pages' bytes.  One new token does 4 g D flops on the
// 4 D bytes (bf16) of a token, g flops a byte where the tensor pipe could
// take 250, so the tokens are streamed from HBM straight into the registers
// that mma.sync reads - no shared memory, no barrier in the loop, every warp
// on its own - and the contraction costs a fraction of the issue slots.
//
// Fragments (lane = 4 r + c).  Scores: m16n8k16 with the queries as A and 8
// tokens as B; token r of an 8-token group is column r, and since the order of
// the contraction is free, lane (r, c) reads 16 contiguous bytes of its
// token, chunk c of 4, as the B operands of two steps.  The accumulator holds
// queries r (and r + 8) x tokens 2c, 2c + 1, which is the layout of the B
// operand of the second product out^T = V^T p^T: p needs no exchange.  Its A
// operand pairs two tokens of one channel: lane (r, c) reads 16 bytes of
// its tokens 2c, 2c + 1, 2c + 8, 2c + 9 (the row chunk r) and pairs
// them with byte permutes.  Weights p are used as a sum of two 16-bit floats
// (p = hi + lo up to 2^-16 p), so their rounding stays below that of a bf16
// output: with g <= 4 the rows r + 4 of A repeat the queries and their lanes
// take the lo part (no instruction more), otherwise a second product adds it.
// hi is cut towards zero and lo kept above zero (kTiny, far below any weight's
// rounding), so that an infinite value stays infinite and is no NaN.
// fp16 weights are scaled by 2^14 so that small ones keep their bits.
//
// Q8 pages.  A byte code c moved into the low half of a bf16 pattern is the
// (subnormal) bf16 c 2^-133, exactly; queries carry 2^64 and weights 2^64, so
// products are normal floats and the powers of two leave at the end.
// Scales and zero points enter per token: s = ks <q, c> + kz sum(q), and
// out = sum (p vs) c + sum p vz.
//
// Split.  The tiles of all units, in order, are dealt to the workers (one CTA
// each) in equal contiguous shares, found by every CTA from a prefix sum of
// the device lengths: ragged lengths, few long requests and many short ones
// all give every SM the same bytes, and nothing depends on lengths the
// host may not know.  A worker meets at most one unit that began before it
// and one that ends behind it: two workspace slots each.

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
constexpr int kCtasPerSm = 3;
constexpr int kSms = 148;
constexpr int kWorkers = kSms * kCtasPerSm;
constexpr int kTile = 16;            // tokens of a warp's step
constexpr int kMinTiles = 2 * kWarps;  // tiles a worker takes at least
constexpr int kMaxGroup = LOOPKV_MAX_PAGED_GROUP;
constexpr uint32_t kNoRow = 0xffffffffu;
constexpr int kCurrentBit = 1 << 30;  // in a cell list entry: the last token is in cur_k / cur_v

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
  float* part;        // [2 * workers][g][D + 2] partial results: out, m, l
  int32_t* split;     // [workers][2]: a unit begun but not ended here, workers that continue it
  uint32_t* status;
  int32_t n_cells, batch, heads, group, max_pages, n_pages, workers;
  int64_t cell_rows;  // token rows of a pool cell
  float scale2;       // sm_scale * log2(e)
  PageDiv div;
};

struct Cells {
  int32_t cell[LOOPKV_MAX_CELLS_PER_CALL];
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
  static constexpr float kTiny = 0x1p-100f;
  static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
  static constexpr float kShift = 0.f;
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
  static constexpr float kTiny = 0x1p-24f;
  static __device__ __forceinline__ float lo(uint32_t w) {
    return __half2float(__ushort_as_half((unsigned short)(w & 0xffffu)));
  }
  static __device__ __forceinline__ float hi(uint32_t w) {
    return __half2float(__ushort_as_half((unsigned short)(w >> 16)));
  }
  // weights are exp2(s - m + 14): 2^14 at most, and only those below 2^-28
  // of the largest lose bits to fp16's smallest step
  static constexpr float kShift = 14.f;
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t s) {
  return __byte_perm(a, b, s);
}

__device__ __forceinline__ uint4 load16(const uint8_t* p, bool on) {
  uint4 x = make_uint4(0, 0, 0, 0);
  if (on)
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
        : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(p));
  return x;
}
__device__ __forceinline__ uint2 load8(const uint8_t* p, bool on) {
  uint2 x = make_uint2(0, 0);
  if (on)
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(x.x), "=r"(x.y) : "l"(p));
  return x;
}

// The words a lane holds of one token row (16 bytes of every 64, Q8: the
// same channels as bytes) and of one value row (its 16-byte pieces).
template <int D, int FMT>
struct Shape {
  static constexpr bool kQ8 = FMT == LOOPKV_PAGE_Q8;
  static constexpr int kRowBytes = kQ8 ? D : 2 * D;
  static constexpr int kSteps = D / 16;        // contraction steps of the scores
  static constexpr int kMTiles = D / 16;       // 16-channel tiles of the output
  static constexpr int kKeyWords = kRowBytes / 16;    // 32-bit words a lane holds of a key token
  static constexpr int kValueWords = kRowBytes / 32;  // and of a value token
};

template <int D, int FMT, int MODE>  // MODE 0: g <= 4, 1: g <= 8, 2: g <= 16
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
paged_decode_kernel(const __grid_constant__ PagedDecodeParams p, const __grid_constant__ Cells cells) {
  require_ieee_subnormals();
  using S = Shape<D, FMT>;
  using M = Mma<FMT>;
  constexpr bool Q8 = S::kQ8;
  constexpr int NT = MODE == 2 ? 2 : 1;      // query halves (8 columns of out^T each)
  constexpr int ROWS = 8 * NT;               // query rows a warp keeps
  constexpr int OS = D + 4;                  // floats of a row in shared memory (banks)
  extern __shared__ __align__(16) uint8_t smem[];
  float* const so = reinterpret_cast<float*>(smem);               // [kWarps][ROWS][OS]
  float* const sm = so + kWarps * ROWS * OS;                      // [kWarps + 1][ROWS] maxima
  float* const sl = sm + (kWarps + 1) * kMaxGroup;                // [kWarps + 1][ROWS] sums
  float* const sz = sl + (kWarps + 1) * kMaxGroup;                // [kWarps][ROWS] zero-point sums (Q8)
  int* const prefix = reinterpret_cast<int*>(sz + kWarps * kMaxGroup);  // [batch + 1] tiles before a request
  __shared__ int warp_sums[kWarps];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
  uint32_t status = 0;

  // Tiles of every request (at least one: a unit without tokens is written too).
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
      const int t = max(1, (n + kTile - 1) / kTile);
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
  const int per_request = p.n_cells * p.heads;
  const int64_t all = (int64_t)prefix[p.batch] * per_request;
  const int64_t want = (all + kMinTiles - 1) / kMinTiles;
  const int workers = (int)(want < p.workers ? want : p.workers);
  const int me = blockIdx.x;
  if (tid == 0) p.split[2 * me + 1] = 0;
  if (me >= workers) return;
  const int64_t x1 = all * (me + 1) / workers;
  int64_t x = all * me / workers;
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
    const int tiles = prefix[b + 1] - prefix[b];
    const int64_t rem = x - (int64_t)prefix[b] * per_request;
    const int u = (int)(rem / tiles), t0 = (int)(rem - (int64_t)u * tiles);
    const int ci = u / p.heads, h = u - ci * p.heads;
    const int t1 = (int)min((int64_t)tiles, t0 + (x1 - x));
    int n = p.len[b];
    if (n < 0 || n > p.max_pages * p.div.size) n = 0;
    const bool current = (cells.cell[ci] & kCurrentBit) != 0 && n > 0;
    const int cell = cells.cell[ci] & ~kCurrentBit;
    const int np = current ? n - 1 : n;  // tokens read from pages

    // Query fragments.
    uint32_t qa[S::kSteps][MODE == 2 ? 4 : 2];
    float qsum[NT];
#pragma unroll
    for (int half = 0; half < NT; ++half) {
      const int row = MODE == 0 ? (r & 3) : r + 8 * half;
      const bool on = row < p.group;
      const uint16_t* src = p.q.at(ci, b, h * p.group + (on ? row : 0));
      float sum = 0.f;
      if constexpr (!Q8) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint4 w = load16(reinterpret_cast<const uint8_t*>(src + 32 * i + 8 * c), on);
          if constexpr (MODE == 2) {
            qa[2 * i][half] = w.x;
            qa[2 * i][2 + half] = w.y;
            qa[2 * i + 1][half] = w.z;
            qa[2 * i + 1][2 + half] = w.w;
          } else {
            qa[2 * i][0] = w.x;
            qa[2 * i][1] = w.y;
            qa[2 * i + 1][0] = w.z;
            qa[2 * i + 1][1] = w.w;
          }
        }
      } else {
        // a 16-byte piece of codes holds 16 channels: 16 c + 64 i ..
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          const uint4 w0 = load16(reinterpret_cast<const uint8_t*>(src + 64 * i + 16 * c), on);
          const uint4 w1 = load16(reinterpret_cast<const uint8_t*>(src + 64 * i + 16 * c + 8), on);
          const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float a = M::lo(w[k]), z = M::hi(w[k]);
            sum += a + z;
            const uint32_t scaled = M::pack(a * 0x1p64f, z * 0x1p64f);
            if constexpr (MODE == 2) qa[4 * i + k / 2][2 * (k & 1) + half] = scaled;
            else qa[4 * i + k / 2][k & 1] = scaled;
          }
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      }
      qsum[half] = sum * p.scale2;
    }

    float o[NT][S::kMTiles][4];
    float m[NT], l[NT], z[NT];
#pragma unroll
    for (int half = 0; half < NT; ++half) {
      m[half] = -INFINITY;
      l[half] = z[half] = 0.f;
#pragma unroll
      for (int j = 0; j < S::kMTiles; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[half][j][k] = 0.f;
    }

    // Token row of the tile's token (lane & 15), or kNoRow.
    auto row_of = [&](int tile) -> uint32_t {
      const int pos = tile * kTile + (lane & 15);
      if (tile >= t1 || pos >= np) return kNoRow;
      const int j = p.div.page(pos);
      const int page = p.table[(int64_t)b * p.max_pages + j];
      if (page < 0 || page >= p.n_pages) {
        status |= LOOPKV_PAGE_BAD_PAGE;
        return kNoRow;
      }
      return (uint32_t)((int64_t)cell * p.cell_rows + ((int64_t)page * p.heads + h) * p.div.size +
                        (pos - j * p.div.size));
    };

    uint32_t row = row_of(t0 + warp);
    for (int tile = t0 + warp; tile < t1; tile += kWarps) {
      // Loads: keys of tokens r and r + 8, values of tokens 2c, 2c + 1, 2c + 8, 2c + 9.
      uint32_t kw[2][S::kKeyWords], vw[4][S::kValueWords];
      bool on[2][2];
      float4 meta[2][2];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const uint32_t kr = __shfl_sync(0xffffffffu, row, r + 8 * g);
        const uint8_t* src = p.k + (uint64_t)kr * S::kRowBytes + 16 * c;
#pragma unroll
        for (int i = 0; i < S::kKeyWords / 4; ++i) {
          const uint4 w = load16(src + 64 * i, kr != kNoRow);
          kw[g][4 * i] = w.x;
          kw[g][4 * i + 1] = w.y;
          kw[g][4 * i + 2] = w.z;
          kw[g][4 * i + 3] = w.w;
        }
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint32_t vr = __shfl_sync(0xffffffffu, row, 2 * c + (g & 1) + 8 * (g >> 1));
        on[g >> 1][g & 1] = vr != kNoRow;
        if constexpr (Q8) {
          meta[g >> 1][g & 1] = vr != kNoRow ? __ldg(p.meta + vr) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if constexpr (S::kValueWords == 2) {
          const uint2 w = load8(p.v + (uint64_t)vr * S::kRowBytes + 8 * r, vr != kNoRow);
          vw[g][0] = w.x;
          vw[g][1] = w.y;
        } else {
          const uint8_t* src = p.v + (uint64_t)vr * S::kRowBytes + 16 * r;
#pragma unroll
          for (int i = 0; i < S::kValueWords / 4; ++i) {
            const uint4 w = load16(src + 128 * i, vr != kNoRow);
            vw[g][4 * i] = w.x;
            vw[g][4 * i + 1] = w.y;
            vw[g][4 * i + 2] = w.z;
            vw[g][4 * i + 3] = w.w;
          }
        }
      }
      row = row_of(tile + kWarps);

      // Scores.
      float s[2][4];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        s[g][0] = s[g][1] = s[g][2] = s[g][3] = 0.f;
#pragma unroll
        for (int ks = 0; ks < S::kSteps; ++ks) {
          uint32_t b0, b1;
          if constexpr (Q8) {
            const uint32_t w = kw[g][ks];
            b0 = prmt(w, 0, 0x4140);
            b1 = prmt(w, 0, 0x4342);
          } else {
            b0 = kw[g][2 * ks];
            b1 = kw[g][2 * ks + 1];
          }
          if constexpr (MODE == 2) M::run(s[g], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], b0, b1);
          else M::run(s[g], qa[ks][0], 0u, qa[ks][1], 0u, b0, b1);
        }
      }

      // Weights, 4 tokens of a query row per lane.
#pragma unroll
      for (int half = 0; half < NT; ++half) {
        float e[2][2];
        float top = -INFINITY;
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float y = s[g][2 * half + k];
            if constexpr (Q8)
              y = fmaf(y, meta[g][k].x * (p.scale2 * 0x1p69f), meta[g][k].y * qsum[half]);
            else
              y *= p.scale2;
            e[g][k] = on[g][k] ? y : -INFINITY;
            top = fmaxf(top, e[g][k]);
          }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float high = fmaxf(m[half], top - M::kShift);
        if (__any_sync(0xffffffffu, high > m[half])) {
          // a first maximum scales sums that are still zero
          const float a = m[half] == -INFINITY ? 0.f : exp2_fast(m[half] - high);
          m[half] = high;
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
        const float base = m[half] == -INFINITY ? 0.f : m[half];
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            e[g][k] = exp2_fast(e[g][k] - base);
            l[half] += e[g][k];
            if constexpr (Q8) {
              z[half] = fmaf(e[g][k], meta[g][k].w, z[half]);
              e[g][k] *= meta[g][k].z * 0x1p64f;
            }
          }
        uint32_t ph[2], pl[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          ph[g] = M::pack_down(e[g][0], e[g][1]);
          pl[g] = M::pack(fmaxf(e[g][0] - M::lo(ph[g]), M::kTiny), fmaxf(e[g][1] - M::hi(ph[g]), M::kTiny));
          if (MODE == 0 && r >= 4) ph[g] = pl[g];
        }

        // out^T += V^T p^T
        if constexpr (!Q8) {
          // tile j: rows r <-> channel 8 r + j of the first piece, rows r + 8
          // <-> of the second (D = 64: channels 4 higher of the only one)
#pragma unroll
          for (int j = 0; j < S::kMTiles; ++j) {
            const uint32_t sel = (j & 1) ? 0x7632 : 0x5410;
            const int w0 = j / 2, w1 = D == 128 ? 4 + j / 2 : 2 + j / 2;
            const uint32_t a0 = prmt(vw[0][w0], vw[1][w0], sel), a1 = prmt(vw[0][w1], vw[1][w1], sel);
            const uint32_t a2 = prmt(vw[2][w0], vw[3][w0], sel), a3 = prmt(vw[2][w1], vw[3][w1], sel);
            M::run(o[half][j], a0, a1, a2, a3, ph[0], ph[1]);
            if constexpr (MODE != 0) M::run(o[half][j], a0, a1, a2, a3, pl[0], pl[1]);
          }
        } else {
          // D = 128: 16 codes of the row, channels 16 r + j and 16 r + 8 + j;
          // D = 64: 8 codes, channels 8 r + j and 8 r + 4 + j
#pragma unroll
          for (int j = 0; j < S::kMTiles; ++j) {
            const int w0 = j / 4, w1 = S::kMTiles / 4 + j / 4;
            const uint32_t k = j & 3, sel = k | (4 + k) << 4;  // byte k of each token's word
            const uint32_t x0 = prmt(vw[0][w0], vw[1][w0], sel), x1 = prmt(vw[0][w1], vw[1][w1], sel);
            const uint32_t x2 = prmt(vw[2][w0], vw[3][w0], sel), x3 = prmt(vw[2][w1], vw[3][w1], sel);
            const uint32_t a0 = prmt(x0, 0, 0x4140), a1 = prmt(x1, 0, 0x4140);
            const uint32_t a2 = prmt(x2, 0, 0x4140), a3 = prmt(x3, 0, 0x4140);
            M::run(o[half][j], a0, a1, a2, a3, ph[0], ph[1]);
            if constexpr (MODE != 0) M::run(o[half][j], a0, a1, a2, a3, pl[0], pl[1]);
          }
        }
      }
    }

    // Join the warps.
#pragma unroll
    for (int half = 0; half < NT; ++half) {
      l[half] += __shfl_xor_sync(0xffffffffu, l[half], 1);
      l[half] += __shfl_xor_sync(0xffffffffu, l[half], 2);
      if constexpr (Q8) {
        z[half] += __shfl_xor_sync(0xffffffffu, z[half], 1);
        z[half] += __shfl_xor_sync(0xffffffffu, z[half], 2);
      }
      if (c == 0) {
        sm[warp * kMaxGroup + r + 8 * half] = m[half];
        sl[warp * kMaxGroup + r + 8 * half] = l[half];
        if constexpr (Q8) sz[warp * kMaxGroup + r + 8 * half] = z[half];
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float* dst = so + (warp * ROWS + 2 * c + k + 8 * half) * OS;
#pragma unroll
        for (int j = 0; j < S::kMTiles; ++j) {
          const float f = Q8 ? 0x1p69f : 1.f;
          if constexpr (!Q8) {
            dst[8 * r + j] = o[half][j][k] * f;
            dst[D == 128 ? 64 + 8 * r + j : 8 * r + 4 + j] = o[half][j][2 + k] * f;
          } else {
            dst[(D / 8) * r + j] = o[half][j][k] * f;
            dst[(D / 8) * r + D / 16 + j] = o[half][j][2 + k] * f;
          }
        }
      }
    }
    const bool with_current = current && t1 == tiles;
    if (with_current) {
      for (int g = warp; g < p.group; g += kWarps) {
        const uint16_t* q = p.q.at(ci, b, h * p.group + g);
        const uint16_t* k = p.cur_k.at(ci, b, h);
        float dot = 0.f;
        for (int d = 2 * lane; d < D; d += 64) {
          const uint32_t a = *reinterpret_cast<const uint32_t*>(q + d);
          const uint32_t w = *reinterpret_cast<const uint32_t*>(k + d);
          dot = fmaf(M::lo(a), M::lo(w), dot);
          dot = fmaf(M::hi(a), M::hi(w), dot);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
        if (lane == 0) {
          sm[kWarps * kMaxGroup + g] = dot * p.scale2;
          sl[kWarps * kMaxGroup + g] = 1.f;
        }
      }
    }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == tiles;
    const int64_t unit = ((int64_t)ci * p.batch + b) * p.heads + h;
    float* const part = p.part + (int64_t)(2 * me + (t0 == 0 ? 1 : 0)) * p.group * (D + 2);
    for (int idx = tid; idx < p.group * D; idx += kThreads) {
      const int g = idx / D, d = idx - g * D;
      float top = with_current ? sm[kWarps * kMaxGroup + g] : -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w * kMaxGroup + g]);
      const float base = top == -INFINITY ? 0.f : top;
      float sum = 0.f, acc = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2_fast(sm[w * kMaxGroup + g] - base);
        sum = fmaf(f, sl[w * kMaxGroup + g], sum);
        float y = so[(w * ROWS + g) * OS + d];
        if constexpr (MODE == 0) y += so[(w * ROWS + g + 4) * OS + d];
        if constexpr (Q8) y += sz[w * kMaxGroup + g];
        acc = fmaf(f, y, acc);
      }
      if (with_current) {
        const float f = exp2_fast(sm[kWarps * kMaxGroup + g] - base);
        sum += f;
        acc = fmaf(f, M::lo(p.cur_v.at(ci, b, h)[d]), acc);
      }
      if (whole) {
        const float y = sum == 0.f ? 0.f : acc / sum;
        p.out[(unit * p.group + g) * D + d] = (uint16_t)(M::pack(y, y) & 0xffffu);
        if (d == 0 && p.lse)
          p.lse[unit * p.group + g] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
      } else {
        part[g * D + d] = acc;
        if (d == 0) {
          part[p.group * D + g] = top;
          part[p.group * (D + 1) + g] = sum;
        }
      }
    }
    if (!whole && t0 == 0 && tid == 0) {
      // the workers behind this one that hold the rest of the unit
      const int64_t last = x + tiles - 1;
      p.split[2 * me] = (int)(unit);
      p.split[2 * me + 1] = (int)(((last + 1) * workers - 1) / all) - me;
    }
    __syncthreads();  // shared memory is free for the next unit
    x += t1 - t0;
    if (x == (int64_t)prefix[b + 1] * per_request) ++b;
  }
  if (status && p.status) atomicOr(p.status, status);
}

// Join the parts of a unit that worker blockIdx.x began and did not end:
// its own (slot 2 i + 1) and those of the workers behind it (slots 2 (i + k)).
template <int D, int FMT>
__global__ void __launch_bounds__(D)
paged_join_kernel(const __grid_constant__ PagedDecodeParams p) {
  using M = Mma<FMT>;
  const int i = blockIdx.x, g = blockIdx.y, d = threadIdx.x;
  const int more = p.split[2 * i + 1];
  if (more == 0) return;
  const int64_t unit = (uint32_t)p.split[2 * i];
  const int64_t stride = (int64_t)p.group * (D + 2);
  auto slot = [&](int k) { return p.part + (k == 0 ? 2 * i + 1 : 2 * (i + k)) * stride; };
  float top = -INFINITY;
  for (int k = 0; k <= more; ++k) top = fmaxf(top, slot(k)[p.group * D + g]);
  const float base = top == -INFINITY ? 0.f : top;
  float sum = 0.f, acc = 0.f;
  for (int k = 0; k <= more; ++k) {
    const float* s = slot(k);
    const float f = exp2_fast(s[p.group * D + g] - base);
    sum = fmaf(f, s[p.group * (D + 1) + g], sum);
    acc = fmaf(f, s[g * D + d], acc);
  }
  const float y = sum == 0.f ? 0.f : acc / sum;
  p.out[(unit * p.group + g) * D + d] = (uint16_t)(M::pack(y, y) & 0xffffu);
  if (d == 0 && p.lse)
    p.lse[unit * p.group + g] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

size_t work_bytes_of(int group, int D) {
  return sizeof(float) * 2 * (size_t)kWorkers * group * (D + 2) + sizeof(int32_t) * 2 * kWorkers;
}

template <int D, int FMT, int MODE>
loopkv_status launch_decode_mode(const PagedDecodeParams& p, const Cells& cells, cudaStream_t stream) {
  constexpr int rows = MODE == 2 ? 16 : 8;
  const size_t smem = sizeof(float) * ((size_t)kWarps * rows * (D + 4) + (3 * kWarps + 2) * kMaxGroup) +
                      sizeof(int) * ((size_t)p.batch + 1);
  const auto kernel = paged_decode_kernel<D, FMT, MODE>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return LOOPKV_ERR_CUDA;
  kernel<<<p.workers, kThreads, smem, stream>>>(p, cells);
  if (cudaGetLastError() != cudaSuccess) return LOOPKV_ERR_CUDA;
  paged_join_kernel<D, FMT><<<dim3(p.workers, p.group), D, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? LOOPKV_OK : LOOPKV_ERR_CUDA;
}

template <int D, int FMT>
loopkv_status launch_decode_format(const PagedDecodeParams& p, const Cells& cells, cudaStream_t stream) {
  if (p.group <= 4) return launch_decode_mode<D, FMT, 0>(p, cells, stream);
  if (p.group <= 8) return launch_decode_mode<D, FMT, 1>(p, cells, stream);
  return launch_decode_mode<D, FMT, 2>(p, cells, stream);
}

template <int D>
loopkv_status launch_decode_dim(int format, const PagedDecodeParams& p, const Cells& cells,
                                cudaStream_t stream) {
  switch (format) {
    case LOOPKV_PAGE_BF16: return launch_decode_format<D, LOOPKV_PAGE_BF16>(p, cells, stream);
    case LOOPKV_PAGE_F16: return launch_decode_format<D, LOOPKV_PAGE_F16>(p, cells, stream);
    default: return launch_decode_format<D, LOOPKV_PAGE_Q8>(p, cells, stream);
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
  *bytes = work_bytes_of(desc->q_per_kv, pool->head_dim);
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
  if (work_bytes < work_bytes_of(desc->q_per_kv, pool->head_dim)) return LOOPKV_ERR_INVALID_ARG;
  Cells cl{};
  bool any_current = false;
  for (int i = 0; i < n_cells; ++i) {
    if (h_cells[i] < 0 || h_cells[i] >= pool->n_cells) return LOOPKV_ERR_INVALID_ARG;
    const bool cur = h_current != nullptr && h_current[i] != 0;
    cl.cell[i] = h_cells[i] | (cur ? kCurrentBit : 0);
    any_current = any_current || cur;
  }
  if (pool->n_cells >= kCurrentBit) return LOOPKV_ERR_INVALID_ARG;
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
  p.split = reinterpret_cast<int32_t*>(p.part + 2 * (size_t)kWorkers * desc->q_per_kv * (pool->head_dim + 2));
  p.status = d_status;
  p.n_cells = n_cells;
  p.batch = desc->batch;
  p.heads = pool->n_kv_heads;
  p.group = desc->q_per_kv;
  p.max_pages = desc->max_pages;
  p.n_pages = pool->n_pages;
  p.workers = kWorkers;
  p.cell_rows = (int64_t)pool->n_pages * pool->n_kv_heads * pool->page_size;
  const float sm_scale = desc->sm_scale > 0.f ? desc->sm_scale : 1.0f / std::sqrt((float)pool->head_dim);
  p.scale2 = sm_scale * 1.4426950408889634f;
  p.div = PageDiv(pool->page_size);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return pool->head_dim == 64 ? launch_decode_dim<64>(pool->format, p, cl, s)
                              : launch_decode_dim<128>(pool->format, p, cl, s);
}
