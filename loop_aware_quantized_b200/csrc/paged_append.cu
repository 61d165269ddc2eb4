// New tokens into the pages of their requests, for sm_100a: a scatter of
// head vectors through the slot map, as they are (bf16, fp16) or quantized to
// 8 bits per token and head on the way (asymmetric min/max, the steps of the
// 4-bit cells' quantizer with 255 steps, in explicitly rounded fp32, so that
// any IEEE implementation of the same steps gives the same codes).
//
// A thread moves 16 bytes of a key vector and the same 16 of the value vector
// (Q8: four such pieces of each, a quarter vector apart); a vector's threads sit
// in one warp, so its minimum and maximum are a few shuffles.  What bounds it:
// memory.  Each byte is read once and written once; a vector is 128 or 256
// contiguous bytes on both sides.  36000 rows of 16 heads of 128 in fp16: 96 us, 6.1
// TB/s.  With a division per value Q8 took more than twice as long as its bytes
// (2 cells of 16384 rows: 175 us, 68 now; 75 where the runs are seconds long and the
// power cap lowers the clock): see codes8.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <vector>

#include "loopkv_internal.cuh"

namespace loopkv {
namespace {

constexpr int kThreads = 128;
// 16-byte pieces of a key vector and of a value vector that a Q8 thread does:
// what is done once per vector (scale, reciprocal, addresses) is shared by so
// many more values (2: 78 us, 4: 65 us of 63 that the bytes take, short runs; 2 cells of
// 16384 rows, 16 heads of 128).
constexpr int kPieces = 4;

struct PagedAppendParams {
  const uint16_t* k;
  const uint16_t* v;
  int64_t k_cell, k_row, k_head, v_cell, v_row, v_head;  // strides in elements
  const int32_t* slots;
  uint8_t* kp;
  uint8_t* vp;
  float4* meta;
  uint32_t* status;
  uint32_t vectors;     // rows * heads
  uint32_t heads;
  int32_t n_slots;      // n_pages * page_size
  int64_t cell_rows;    // token rows of a pool cell
  PageDiv div, by_heads;
};

__device__ __forceinline__ void unpack_bf16(const uint4& x, float (&f)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {  // low bytes
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// By the definition, one value after another.  Where the scale is not finite, the
// quotients are 0 or NaN, which converts to 0.
__device__ __noinline__ uint2 codes8_exact(uint4 x, float scale, float low) {
  float f[8];
  unpack_bf16(x, f);
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int q = scale == 0.f ? 0 : __float2int_rn(__fdiv_rn(__fsub_rn(f[i], low), scale));
    c[i] = (uint32_t)(q < 0 ? 0 : (q > 255 ? 255 : q));
  }
  return make_uint2(pack4(c[0], c[1], c[2], c[3]), pack4(c[4], c[5], c[6], c[7]));
}

__device__ __forceinline__ uint64_t pair(float x, float y) {
  return (uint64_t)__float_as_uint(x) | (uint64_t)__float_as_uint(y) << 32;
}

// A vector's scale and minimum, and the reciprocal of the scale.
struct Quantizer {
  float scale, low, inverse;
  __device__ __forceinline__ Quantizer(float mn, float mx) : low(mn) {
    const float range = __fsub_rn(mx, mn);
    scale = range == 0.f ? 0.f : __fdiv_rn(range, 255.f);
    inverse = __frcp_rn(scale);
  }
  // What codes8 does not cover: scales so small or large that its steps could
  // underflow or overflow, and those whose last 16 bits are within 8 of 0.
  __device__ __forceinline__ bool ordinary() const {
    return scale > 0x1p-100f && scale < 0x1p100f && ((__float_as_uint(scale) + 8u) & 0xffffu) > 16u;
  }
  __device__ __forceinline__ float zero() const { return low == 0.f ? 0.f : low; }  // a zero minimum is stored as +0
};

// The codes of 8 values: rne(fl(t / s)), t = fl(x - low), two values to an
// instruction.  Quotients on a half step are common (bf16 values are few bits
// apart), so the rounded quotient itself is needed, and a division takes 10
// instructions and more per value.  With y the rounded reciprocal of s and q0 =
// fl(t y), q1 = fl(q0 + y (t - q0 s)), fused: one Newton step, whose argument of
// the last rounding is within 2^-46 of t / s, relatively (y and q0 are off by 2^-24
// and 2^-23, the residual is rounded by 2^-24 at most, and the products of these
// remain).  So q1 is fl(t / s) unless t / s is that close to the middle of
// two floats, and the code can differ only where one of the two is a half step h
// in [2^e, 2^(e+1)): t = s (h +- 2^(e-24)) (1 + 2^-46).  With s = S 2^a, S of 24
// bits, t is a multiple of 2^(a+e), so S 2^(e-23) would have to be within 2^(e-20)
// of an integer: S within 8 of a multiple of 2^(23-e), hence of 2^16, e being 7
// at most (and for e = -1 no t below s / 2 meets the condition).  Those scales
// are left to the definition.  rne is the sum with 2^23; the code is then the
// low byte.
__device__ __forceinline__ uint2 codes8(const uint4& x, const Quantizer& z) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  const uint64_t low = pair(-z.low, -z.low), y = pair(z.inverse, z.inverse), s = pair(-z.scale, -z.scale);
  const uint64_t magic = pair(0x1p23f, 0x1p23f);
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint64_t t = (uint64_t)(w[i] << 16) | (uint64_t)(w[i] & 0xffff0000u) << 32, q, r;
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(t) : "l"(low));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(t), "l"(y));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(q), "l"(s), "l"(t));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(q) : "l"(r), "l"(y));
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(q) : "l"(magic));
    c[2 * i] = (uint32_t)q;
    c[2 * i + 1] = (uint32_t)(q >> 32);
  }
  return make_uint2(pack4(c[0], c[1], c[2], c[3]), pack4(c[4], c[5], c[6], c[7]));
}

// The smallest and the negated largest of a thread's bf16 values, as a pair; NaN
// if there is one, so that it reaches scale and zero point.
__device__ __forceinline__ __nv_bfloat162 extremes(const uint4 (&x)[kPieces]) {
  __nv_bfloat162 mn = *reinterpret_cast<const __nv_bfloat162*>(&x[0].x), mx = mn;
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&w[i]);
      mn = __hmin2_nan(mn, v);
      mx = __hmax2_nan(mx, v);
    }
  }
  return __halves2bfloat162(__hmin_nan(__low2bfloat16(mn), __high2bfloat16(mn)),
                            __hneg(__hmax_nan(__low2bfloat16(mx), __high2bfloat16(mx))));
}

template <int LANES>
__device__ __forceinline__ Quantizer quantizer(__nv_bfloat162 e) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) e = __hmin2_nan(e, __shfl_xor_sync(0xffffffffu, e, o));
  return Quantizer(__low2float(e), -__high2float(e));
}

template <int D, bool Q8>
__global__ void __launch_bounds__(kThreads)
paged_append_kernel(const __grid_constant__ PagedAppendParams p, const __grid_constant__ CellList cells) {
  require_ieee_subnormals();
  wait_for_previous();
  constexpr int LANES = Q8 ? D / (8 * kPieces) : D / 8;
  const uint32_t i = blockIdx.x * (uint32_t)(kThreads / LANES) + threadIdx.x / LANES;
  const int part = threadIdx.x % LANES;
  const bool in = i < p.vectors;
  const uint32_t row = in ? (uint32_t)p.by_heads.page((int)i) : 0u, head = in ? i - row * p.heads : 0u;
  int slot = in ? p.slots[row] : -1;
  if (slot < -1 || slot >= p.n_slots) {
    if (p.status && part == 0) atomicOr(p.status, LOOPKV_PAGE_BAD_SLOT);
    slot = -1;
  }
  const int64_t ci = cells.out[blockIdx.y];
  const uint16_t* const ks = p.k + ci * p.k_cell + row * p.k_row + head * p.k_head + part * 8;
  const uint16_t* const vs = p.v + ci * p.v_cell + row * p.v_row + head * p.v_head + part * 8;
  const int page = p.div.page(slot < 0 ? 0 : slot), off = slot - page * p.div.size;
  const int64_t at = cells.cell[blockIdx.y] * p.cell_rows +
                     ((int64_t)page * p.heads + head) * p.div.size + off;
  if constexpr (Q8) {
    uint4 k[kPieces], v[kPieces];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      k[j] = v[j] = make_uint4(0, 0, 0, 0);
      if (slot >= 0) {
        k[j] = *reinterpret_cast<const uint4*>(ks + j * (D / kPieces));
        v[j] = *reinterpret_cast<const uint4*>(vs + j * (D / kPieces));
      }
    }
    const Quantizer kz = quantizer<LANES>(extremes(k)), vz = quantizer<LANES>(extremes(v));
    if (slot < 0) return;
    uint8_t* const kd = p.kp + at * D + part * 8;
    uint8_t* const vd = p.vp + at * D + part * 8;
    if (kz.ordinary() && vz.ordinary()) {
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        *reinterpret_cast<uint2*>(kd + j * (D / kPieces)) = codes8(k[j], kz);
        *reinterpret_cast<uint2*>(vd + j * (D / kPieces)) = codes8(v[j], vz);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        *reinterpret_cast<uint2*>(kd + j * (D / kPieces)) = codes8_exact(k[j], kz.scale, kz.low);
        *reinterpret_cast<uint2*>(vd + j * (D / kPieces)) = codes8_exact(v[j], vz.scale, vz.low);
      }
    }
    if (part == 0) {
      p.meta[at] = make_float4(kz.scale, kz.zero(), vz.scale, vz.zero());
      // (also for NaN; decode carries value scales times 2^64 and weights up to 2^8 in bf16)
      if (p.status && !(kz.scale < INFINITY && vz.scale < 0x1p56f)) atomicOr(p.status, LOOPKV_PAGE_BAD_VALUE);
    }
  } else {
    if (slot < 0) return;
    const uint4 k = *reinterpret_cast<const uint4*>(ks), v = *reinterpret_cast<const uint4*>(vs);
    *reinterpret_cast<uint4*>(p.kp + (at * D + part * 8) * 2) = k;
    *reinterpret_cast<uint4*>(p.vp + (at * D + part * 8) * 2) = v;
  }
}

}  // namespace

bool pool_ok(const loopkv_page_pool* p) {
  if (p == nullptr || p->n_cells < 1 || p->n_pages < 1) return false;
  if (p->page_size < 1 || p->page_size > kMaxPageSize) return false;
  if (p->n_kv_heads < 1 || p->n_kv_heads > (1 << 16)) return false;
  if (p->head_dim != 64 && p->head_dim != 128) return false;
  if (p->format < LOOPKV_PAGE_BF16 || p->format > LOOPKV_PAGE_Q8) return false;
  if ((int64_t)p->n_pages * p->page_size >= (1LL << 31)) return false;
  const uint64_t rows = (uint64_t)p->n_pages * (uint64_t)p->page_size * (uint64_t)p->n_kv_heads;
  if (rows >= (1ULL << 32) || rows * (uint64_t)p->n_cells >= 0xffffffffULL) return false;
  if (p->k == nullptr || p->v == nullptr || !aligned16(p->k) || !aligned16(p->v)) return false;
  const bool q8 = p->format == LOOPKV_PAGE_Q8;
  return q8 == (p->meta != nullptr) && aligned16(p->meta);
}

bool rows_ok(const loopkv_rows* r) {
  return r != nullptr && r->data != nullptr && aligned16(r->data) && r->cell_stride >= 0 &&
         r->row_stride >= 0 && r->head_stride >= 0 &&
         ((r->cell_stride | r->row_stride | r->head_stride) & 7) == 0;
}

}  // namespace loopkv

using namespace loopkv;

extern "C" loopkv_status loopkv_paged_append(const loopkv_page_pool* pool, const int32_t* h_cells,
                                             int32_t n_cells, int32_t n_rows, const int32_t* d_slots,
                                             const loopkv_rows* k, const loopkv_rows* v,
                                             uint32_t* d_status, void* stream) {
  if (!pool_ok(pool) || h_cells == nullptr || n_cells < 1 || n_cells > LOOPKV_MAX_CELLS_PER_CALL)
    return LOOPKV_ERR_INVALID_ARG;
  if (n_rows < 0 || (reinterpret_cast<uintptr_t>(d_status) & 3u) != 0) return LOOPKV_ERR_INVALID_ARG;
  CellList cl{};
  int stored = 0;
  for (int i = 0; i < n_cells; ++i) {
    const int c = h_cells[i];
    if (c < -1 || c >= pool->n_cells) return LOOPKV_ERR_INVALID_ARG;
    if (c < 0) continue;
    for (int j = 0; j < stored; ++j)
      if (cl.cell[j] == c) return LOOPKV_ERR_INVALID_ARG;
    cl.cell[stored] = c;
    cl.out[stored++] = i;
  }
  if (n_rows == 0) return LOOPKV_OK;
  if (d_slots == nullptr || (reinterpret_cast<uintptr_t>(d_slots) & 3u) != 0 || !rows_ok(k) || !rows_ok(v))
    return LOOPKV_ERR_INVALID_ARG;
  if (stored == 0) return LOOPKV_OK;
  const int64_t vectors = (int64_t)n_rows * pool->n_kv_heads;
  const bool q8 = pool->format == LOOPKV_PAGE_Q8;
  const int64_t blocks = (vectors * (pool->head_dim / (q8 ? 8 * kPieces : 8)) + kThreads - 1) / kThreads;
  if (vectors >= (1LL << 31) - kThreads) return LOOPKV_ERR_UNSUPPORTED;
  PagedAppendParams p{};
  p.k = static_cast<const uint16_t*>(k->data);
  p.v = static_cast<const uint16_t*>(v->data);
  p.k_cell = k->cell_stride;
  p.k_row = k->row_stride;
  p.k_head = k->head_stride;
  p.v_cell = v->cell_stride;
  p.v_row = v->row_stride;
  p.v_head = v->head_stride;
  p.slots = d_slots;
  p.kp = static_cast<uint8_t*>(pool->k);
  p.vp = static_cast<uint8_t*>(pool->v);
  p.meta = reinterpret_cast<float4*>(pool->meta);
  p.status = d_status;
  p.vectors = (uint32_t)vectors;
  p.heads = (uint32_t)pool->n_kv_heads;
  p.n_slots = pool->n_pages * pool->page_size;
  p.cell_rows = (int64_t)pool->n_pages * pool->n_kv_heads * pool->page_size;
  p.div = PageDiv(pool->page_size);
  p.by_heads = PageDiv(pool->n_kv_heads);
  const dim3 grid((unsigned)blocks, (unsigned)stored);
  if (pool->head_dim == 64)
    return q8 ? launch_early(paged_append_kernel<64, true>, grid, kThreads, 0, stream, p, cl)
              : launch_early(paged_append_kernel<64, false>, grid, kThreads, 0, stream, p, cl);
  return q8 ? launch_early(paged_append_kernel<128, true>, grid, kThreads, 0, stream, p, cl)
            : launch_early(paged_append_kernel<128, false>, grid, kThreads, 0, stream, p, cl);
}
