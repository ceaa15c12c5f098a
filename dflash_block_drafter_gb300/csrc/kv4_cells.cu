// Writing and reading the cells of the 4-bit paged K/V cache (kv4.cuh).
//
// Quantisation of 32 consecutive channels x: m = the x of largest magnitude
// (the first of equals), d = fp16(m / -8), code = clamp(rint(x / d), -8, 7) + 8
// (rint: halves to even; every code 8 where d is 0); a cell's value is
// d * (code - 8), so m itself is met to d's rounding.  x / d is a quotient of
// two 11-bit significands at most: the 32-bit quotient lies on a half only
// where the exact one does, so rounding it is rounding the exact quotient.
//
// Both kernels are bound by memory: a thread holds the 8 channels of one code
// word (a 16-byte load of K or V, one 4-byte store), the quad of a block
// finds m by shuffles, and a warp covers 256 consecutive channels of a row.
#include <cstddef>

#include "internal.h"
#include "kv4.cuh"
#include "kernels.h"
#include "common.cuh"

namespace dflash {
namespace {

struct CellArgs {
  uint8_t* data;
  int n_pages, page_shift, n_kv;
  const int32_t* slots;
  int n_rows;
  const uint16_t* k;
  const uint16_t* v;
  long long k_stride, v_stride;  // elements between rows
  float* k_out;
  float* v_out;
  int32_t* status;
};

// Address of the group of (slot, head); the cell in the group is slot % 16.
template <int D>
__device__ __forceinline__ uint8_t* group_of(const CellArgs& a, int slot, int head) {
  const int groups = 1 << (a.page_shift - 4);
  const size_t page = static_cast<size_t>(slot >> a.page_shift);
  const int grp = (slot & ((1 << a.page_shift) - 1)) >> 4;
  return a.data + ((page * a.n_kv + head) * groups + grp) * Kv4<D>::GROUP_BYTES;
}

template <bool BF16>
__device__ __forceinline__ float widen(uint32_t pair, int half) {
  if (BF16) return __uint_as_float(half ? pair & 0xffff0000u : pair << 16);
  const __half2 h = *reinterpret_cast<const __half2*>(&pair);
  return half ? __high2float(h) : __low2float(h);
}

// Thread = (row, side, head, word): words of a head fastest, then heads, then
// K / V, then rows.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) kv4_write_kernel(const CellArgs a) {
  using F = Kv4<D>;
  const int per_row = 2 * a.n_kv * F::WORDS;
  const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  const long long row = i / per_row;
  if (row >= a.n_rows) return;  // whole quads leave: per_row is a multiple of 16
  const int in_row = static_cast<int>(i - row * per_row);
  const int w = in_row % F::WORDS, hs = in_row / F::WORDS;
  const int side = hs >= a.n_kv, head = hs - side * a.n_kv;
  const int slot = a.slots[row];
  const long long cells = static_cast<long long>(a.n_pages) << a.page_shift;
  if (slot < 0 || slot >= cells) {  // the same for the whole quad
    if (slot >= cells && in_row == 0) set_status(a.status, DFLASH_DEV_CAPACITY);
    return;
  }
  const unsigned quad = 0xfu << (threadIdx.x & 28);
  const uint16_t* src = side ? a.v + row * a.v_stride : a.k + row * a.k_stride;
  const uint4 raw = *reinterpret_cast<const uint4*>(src + head * D + w * 8);
  const uint32_t pr[4] = {raw.x, raw.y, raw.z, raw.w};
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = widen<BF16>(pr[e >> 1], e & 1);
  float top = 0.f;
  bool bad = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    top = fmaxf(top, fabsf(x[e]));
    bad |= !(fabsf(x[e]) <= 65504.f);  // beyond FP16's range, infinite or NaN
  }
  top = fmaxf(top, __shfl_xor_sync(quad, top, 1));
  top = fmaxf(top, __shfl_xor_sync(quad, top, 2));
  bad = __any_sync(quad, bad);
  // sign of the first element of that magnitude: smallest (index, sign)
  int first = 1 << 10;
#pragma unroll
  for (int e = 7; e >= 0; --e)
    if (fabsf(x[e]) == top) first = ((w & 3) * 8 + e) * 2 + (x[e] < 0.f ? 1 : 0);
  first = min(first, __shfl_xor_sync(quad, first, 1));
  first = min(first, __shfl_xor_sync(quad, first, 2));
  const __half dh = __float2half_rn((first & 1) ? top * 0.125f : top * -0.125f);
  const float d = __half2float(dh);
  uint32_t code = 0x88888888u;
  __half store = dh;
  if (bad) {
    store = __ushort_as_half(0);
    if ((w & 3) == 0) set_status(a.status, DFLASH_DEV_NONFINITE);
  } else if (d != 0.f) {
    code = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int q = static_cast<int>(fminf(fmaxf(rintf(x[e] / d), -8.f), 7.f)) + 8;
      code |= static_cast<uint32_t>(q) << (4 * e);
    }
  }
  uint8_t* g = group_of<D>(a, slot, head);
  const int cell = slot & 15;
  *reinterpret_cast<uint32_t*>(g + (side ? F::v_word(cell, w) : F::k_word(cell, w))) = code;
  if ((w & 3) == 0) *reinterpret_cast<__half*>(g + (side ? F::v_scale(cell, w >> 2) : F::k_scale(cell, w >> 2))) = store;
}

template <int D>
__global__ void __launch_bounds__(256) kv4_read_kernel(const CellArgs a) {
  using F = Kv4<D>;
  const int per_row = 2 * a.n_kv * F::WORDS;
  const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  const long long row = i / per_row;
  if (row >= a.n_rows) return;
  const int in_row = static_cast<int>(i - row * per_row);
  const int w = in_row % F::WORDS, hs = in_row / F::WORDS;
  const int side = hs >= a.n_kv, head = hs - side * a.n_kv;
  float* base = side ? a.v_out : a.k_out;
  if (!base) return;
  const int slot = a.slots[row];
  const long long cells = static_cast<long long>(a.n_pages) << a.page_shift;
  float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (slot >= 0 && slot < cells) {
    const uint8_t* g = group_of<D>(a, slot, head);
    const int cell = slot & 15;
    const uint32_t code = *reinterpret_cast<const uint32_t*>(g + (side ? F::v_word(cell, w) : F::k_word(cell, w)));
    const float d = __half2float(
        *reinterpret_cast<const __half*>(g + (side ? F::v_scale(cell, w >> 2) : F::k_scale(cell, w >> 2))));
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = d * static_cast<float>(static_cast<int>((code >> (4 * e)) & 15u) - 8);
  } else if (slot >= cells && in_row == 0) {
    set_status(a.status, DFLASH_DEV_CAPACITY);
  }
  float4* out = reinterpret_cast<float4*>(base + (row * a.n_kv + head) * D + w * 8);
  out[0] = make_float4(y[0], y[1], y[2], y[3]);
  out[1] = make_float4(y[4], y[5], y[6], y[7]);
}

template <int D>
cudaError_t launch(const CellArgs& a, int type, bool write, cudaStream_t st) {
  const long long total = static_cast<long long>(a.n_rows) * 2 * a.n_kv * Kv4<D>::WORDS;
  const long long blocks = (total + 255) / 256;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  const unsigned grid = static_cast<unsigned>(blocks);
  if (!write) kv4_read_kernel<D><<<grid, 256, 0, st>>>(a);
  else if (type == DFLASH_T_BF16) kv4_write_kernel<D, true><<<grid, 256, 0, st>>>(a);
  else kv4_write_kernel<D, false><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cells(const dflash_kv4_cache* c, const CellArgs& a, int type, bool write, cudaStream_t st) {
  switch (c->head_dim) {
    case 64: return launch<64>(a, type, write, st);
    case 128: return launch<128>(a, type, write, st);
    default: return launch<256>(a, type, write, st);
  }
}

}  // namespace

int log2_page(const dflash_kv4_cache* c) {
  int s = 4;
  while ((1 << s) < c->page_size) ++s;
  return s;
}

}  // namespace dflash

using namespace dflash;

extern "C" {

int dflash_kv4_check(const dflash_kv4_cache* c) {
  if (!c || !c->data || reinterpret_cast<uintptr_t>(c->data) % 16) return DFLASH_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return DFLASH_ERR_UNSUPPORTED;
  const int p = c->page_size;
  if (p < 16 || p > 256 || (p & (p - 1))) return DFLASH_ERR_UNSUPPORTED;
  if (c->n_kv_heads < 1 || c->n_kv_heads > 256 || c->n_pages < 1) return DFLASH_ERR_INVALID_ARG;
  if (static_cast<long long>(c->n_pages) * p > 0x7fffffffll) return DFLASH_ERR_CAPACITY;
  return DFLASH_OK;
}

size_t dflash_kv4_bytes(int32_t n_pages, int32_t page_size, int32_t n_kv_heads, int32_t head_dim) {
  dflash_kv4_cache c{reinterpret_cast<void*>(16), n_pages, page_size, n_kv_heads, head_dim};
  if (dflash_kv4_check(&c) != DFLASH_OK) return 0;
  return static_cast<size_t>(n_pages) * n_kv_heads * (page_size / 16) * 18 * head_dim;
}

int dflash_kv4_write(const dflash_kv4_cache* c, const void* k, const void* v, int32_t type, int64_t k_stride,
                     int64_t v_stride, const int32_t* slots, int32_t n_rows, int32_t* dev_status,
                     dflash_stream_t stream) {
  if (const int e = dflash_kv4_check(c)) return e;
  if (type != DFLASH_T_BF16 && type != DFLASH_T_FP16) return DFLASH_ERR_UNSUPPORTED;
  if (n_rows < 0) return DFLASH_ERR_INVALID_ARG;
  if (n_rows == 0) return DFLASH_OK;
  const int64_t width = static_cast<int64_t>(c->n_kv_heads) * c->head_dim;
  if (!k || !v || !slots || reinterpret_cast<uintptr_t>(k) % 16 || reinterpret_cast<uintptr_t>(v) % 16 ||
      k_stride < width || v_stride < width || k_stride % 8 || v_stride % 8)
    return DFLASH_ERR_INVALID_ARG;
  CellArgs a{};
  a.data = static_cast<uint8_t*>(c->data);
  a.n_pages = c->n_pages;
  a.page_shift = log2_page(c);
  a.n_kv = c->n_kv_heads;
  a.slots = slots;
  a.n_rows = n_rows;
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.status = dev_status;
  return cuda_status(launch_cells(c, a, type, true, reinterpret_cast<cudaStream_t>(stream)), "kv4 write");
}

int dflash_kv4_read(const dflash_kv4_cache* c, const int32_t* slots, int32_t n_rows, float* k_out, float* v_out,
                    int32_t* dev_status, dflash_stream_t stream) {
  if (const int e = dflash_kv4_check(c)) return e;
  if (n_rows < 0) return DFLASH_ERR_INVALID_ARG;
  if (n_rows == 0 || (!k_out && !v_out)) return DFLASH_OK;
  if (!slots || reinterpret_cast<uintptr_t>(k_out) % 16 || reinterpret_cast<uintptr_t>(v_out) % 16)
    return DFLASH_ERR_INVALID_ARG;
  CellArgs a{};
  a.data = static_cast<uint8_t*>(c->data);
  a.n_pages = c->n_pages;
  a.page_shift = log2_page(c);
  a.n_kv = c->n_kv_heads;
  a.slots = slots;
  a.n_rows = n_rows;
  a.k_out = k_out;
  a.v_out = v_out;
  a.status = dev_status;
  return cuda_status(launch_cells(c, a, 0, false, reinterpret_cast<cudaStream_t>(stream)), "kv4 read");
}

}  // extern "C"
