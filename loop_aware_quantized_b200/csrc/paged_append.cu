// New tokens into the pages of their requests, for sm_100a: a scatter of
// head vectors through the slot map, as they are (bf16, fp16) or quantized to
// 8 bits per token and head on the way (asymmetric min/max, the steps of the
// 4-bit cells' quantizer with 255 steps, in explicitly rounded fp32, so that
// any IEEE implementation of the same steps gives the same codes).
//
// A thread moves 16 bytes of a key vector and the same 16 of the value
// vector; the D / 8 threads of one (row, head) sit in one warp, so a Q8
// vector's minimum and maximum are a few shuffles.  What bounds it: memory.
// Each byte is read once and written once; a vector is 128 or 256
// contiguous bytes on both sides.

#include <cuda_runtime.h>

#include <cstdint>
#include <vector>

#include "loopkv_internal.cuh"

namespace loopkv {
namespace {

constexpr int kThreads = 256;

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
  PageDiv div;
};

__device__ __forceinline__ void unpack_bf16(const uint4& x, float (&f)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// The 8 codes of a thread's 8 values, given its vector's scale and minimum.
__device__ __forceinline__ uint2 codes8(const float (&f)[8], float scale, float low) {
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int q = scale == 0.f ? 0 : __float2int_rn(__fdiv_rn(__fsub_rn(f[i], low), scale));
    c[i] = (uint32_t)(q < 0 ? 0 : (q > 255 ? 255 : q));
  }
  return make_uint2(c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24,
                    c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24);
}

template <int LANES>
__device__ __forceinline__ void scale_zero(const float (&f)[8], float* scale, float* zero, float* low) {
  float mn = f[0], mx = f[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    mn = fminf(mn, f[i]);
    mx = fmaxf(mx, f[i]);
  }
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  const float range = __fsub_rn(mx, mn);
  *scale = range == 0.f ? 0.f : __fdiv_rn(range, 255.f);
  *low = mn;
  *zero = mn == 0.f ? 0.f : mn;  // a zero minimum is stored as +0
}

template <int D, bool Q8>
__global__ void __launch_bounds__(kThreads)
paged_append_kernel(const __grid_constant__ PagedAppendParams p, const __grid_constant__ CellList cells) {
  require_ieee_subnormals();
  constexpr int LANES = D / 8;
  const uint32_t i = blockIdx.x * (uint32_t)(kThreads / LANES) + threadIdx.x / LANES;
  const int part = threadIdx.x % LANES;
  const bool in = i < p.vectors;
  const uint32_t row = in ? i / p.heads : 0u, head = in ? i - row * p.heads : 0u;
  int slot = in ? p.slots[row] : -1;
  if (slot < -1 || slot >= p.n_slots) {
    if (p.status && part == 0) atomicOr(p.status, LOOPKV_PAGE_BAD_SLOT);
    slot = -1;
  }
  uint4 k = make_uint4(0, 0, 0, 0), v = k;
  const int64_t ci = cells.out[blockIdx.y];
  if (slot >= 0) {
    k = *reinterpret_cast<const uint4*>(p.k + ci * p.k_cell + row * p.k_row + head * p.k_head + part * 8);
    v = *reinterpret_cast<const uint4*>(p.v + ci * p.v_cell + row * p.v_row + head * p.v_head + part * 8);
  }
  const int page = p.div.page(slot < 0 ? 0 : slot), off = slot - page * p.div.size;
  const int64_t at = cells.cell[blockIdx.y] * p.cell_rows +
                     ((int64_t)page * p.heads + head) * p.div.size + off;
  if constexpr (Q8) {
    float kf[8], vf[8];
    unpack_bf16(k, kf);
    unpack_bf16(v, vf);
    float4 m;
    float kl, vl;
    scale_zero<LANES>(kf, &m.x, &m.y, &kl);
    scale_zero<LANES>(vf, &m.z, &m.w, &vl);
    if (slot < 0) return;
    *reinterpret_cast<uint2*>(p.kp + at * D + part * 8) = codes8(kf, m.x, kl);
    *reinterpret_cast<uint2*>(p.vp + at * D + part * 8) = codes8(vf, m.z, vl);
    if (part == 0) p.meta[at] = m;
  } else {
    if (slot < 0) return;
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
  const int64_t blocks = (vectors * (pool->head_dim / 8) + kThreads - 1) / kThreads;
  if (vectors >= (1LL << 32) - kThreads || blocks >= (1LL << 31)) return LOOPKV_ERR_UNSUPPORTED;
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
  const dim3 grid((unsigned)blocks, (unsigned)stored);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool q8 = pool->format == LOOPKV_PAGE_Q8;
  if (pool->head_dim == 64 && q8) paged_append_kernel<64, true><<<grid, kThreads, 0, s>>>(p, cl);
  else if (pool->head_dim == 64) paged_append_kernel<64, false><<<grid, kThreads, 0, s>>>(p, cl);
  else if (q8) paged_append_kernel<128, true><<<grid, kThreads, 0, s>>>(p, cl);
  else paged_append_kernel<128, false><<<grid, kThreads, 0, s>>>(p, cl);
  return cudaGetLastError() == cudaSuccess ? LOOPKV_OK : LOOPKV_ERR_CUDA;
}
