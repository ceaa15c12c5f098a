// Writing and reading the cells of the 4-bit paged K/V cache (kv4.cuh).
//
// Quantisation of 32 consecutive channels x: m = the x of largest magnitude
// (the first of equals), d = fp16(m / -8), code = clamp(rint(x / d), -8, 7) + 8
// (rint: halves to even; every code 8 where d is 0); a cell's value is
// d * (code - 8), so m itself is met to d's rounding.  x / d is a quotient of
// two 11-bit significands at most: near 0.5 .. 8.5 it lies on a half or more
// than 2^-13 away from one.  x times the approximate 1 / d is off by less than
// 2^-19; rounded to a multiple of 2^-17 (one FMA onto 96) it is on a half exactly
// where x / d is, and on the same side elsewhere, so that one more addition rounds
// it as the definition says.  Where d is so small (FP16's subnormals) that |x / d|
// passes 8.4, each value is divided.
//
// A thread holds the 8 channels of one code word of K and of V (two 16-byte
// loads, two 4-byte stores; reading: two codes in, 64 bytes out), the quad of a
// block finds m by shuffles, and a warp covers 256 consecutive channels of a row.
// Measured on 30001 rows of 8 heads of 128 in random slots: written in 41 us (bound
// by the extremes, roundings and packing; the bytes alone take 23; a division per
// value took 88), read in 44 us (the bytes: 41).
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
  int rows_of_block;
  uint32_t magic;  // ceil(2^32 / words of a row)
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

// A block takes the words of `rows` rows (a multiple of 4 words each, so
// that quads stay whole): item = row * words + word of the row's heads.
// Dividing by `words` is a multiplication: both are far below 2^16.
struct Item {
  int row, head, w;  // row in the block; head; word of the head
  bool in;
};
template <int D>
__device__ __forceinline__ Item item_of(const CellArgs& a, int i) {
  Item t;
  const int words = a.n_kv * Kv4<D>::WORDS;
  t.row = static_cast<int>(__umulhi(static_cast<uint32_t>(i), a.magic));
  const int word = i - t.row * words;
  t.head = word / Kv4<D>::WORDS;
  t.w = word % Kv4<D>::WORDS;
  t.in = t.row < a.rows_of_block;
  return t;
}

// max and min that return NaN if either is one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
  uint32_t r;
  if (BF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t min_pair(uint32_t a, uint32_t b) {
  uint32_t r;
  if (BF16) asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Whether the block's first value of magnitude `top` is negative.
template <bool BF16>
__device__ __noinline__ bool first_is_negative(uint4 raw, int w, unsigned quad, float top) {
  const uint32_t pr[4] = {raw.x, raw.y, raw.z, raw.w};
  int first = 1 << 10;  // smallest (index, sign)
#pragma unroll
  for (int e = 7; e >= 0; --e) {
    const float x = widen<BF16>(pr[e >> 1], e & 1);
    if (fabsf(x) == top) first = ((w & 3) * 8 + e) * 2 + (x < 0.f ? 1 : 0);
  }
  first = min(first, __shfl_xor_sync(quad, first, 1));
  first = min(first, __shfl_xor_sync(quad, first, 2));
  return first & 1;
}

// The codes by a division per value (d may be 0).
template <bool BF16>
__device__ __noinline__ uint32_t divide_all(uint4 raw, float d) {
  if (d == 0.f) return 0x88888888u;
  const uint32_t pr[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t code = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int q = static_cast<int>(fminf(fmaxf(rintf(widen<BF16>(pr[e >> 1], e & 1) / d), -8.f), 7.f)) + 8;
    code |= static_cast<uint32_t>(q) << (4 * e);
  }
  return code;
}

// The code word and scale of 8 of a block's 32 values, whose other lanes are the quad's.
template <bool BF16>
__device__ __forceinline__ uint32_t quantise(uint4 raw, int w, unsigned quad, __half& scale, bool& bad) {
  const uint32_t up = max_pair<BF16>(max_pair<BF16>(raw.x, raw.y), max_pair<BF16>(raw.z, raw.w));
  const uint32_t down = min_pair<BF16>(min_pair<BF16>(raw.x, raw.y), min_pair<BF16>(raw.z, raw.w));
  float hi = max_nan(widen<BF16>(up, 0), widen<BF16>(up, 1)), lo = -min_nan(widen<BF16>(down, 0), widen<BF16>(down, 1));
  hi = max_nan(hi, __shfl_xor_sync(quad, hi, 1));
  lo = max_nan(lo, __shfl_xor_sync(quad, lo, 1));
  hi = max_nan(hi, __shfl_xor_sync(quad, hi, 2));
  lo = max_nan(lo, __shfl_xor_sync(quad, lo, 2));
  const float top = max_nan(hi, lo);
  bad = !(top <= 65504.f);  // a value beyond FP16's range, an infinity or a NaN
  bool negative = lo > hi;
  if (hi == lo) negative = first_is_negative<BF16>(raw, w, quad, top);  // m with both signs, or all zeros
  scale = __float2half_rn(negative ? top * 0.125f : top * -0.125f);
  const float d = __half2float(scale);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(d));
  constexpr float MAGIC = 12582912.f;  // 1.5 2^23: adding it rounds to an integer, which its low bits then hold
  const uint32_t pr[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = widen<BF16>(pr[e >> 1], e & 1);
    y[e] = __float_as_uint(fminf(fmaf(x, inv, 96.f) + (MAGIC - 96.f), MAGIC + 7.f));
  }
  // low nibbles, plus 8: bytes of the even and the odd values, then side by side
  const uint32_t even = prmt(prmt(y[0], y[2], 0x0040u), prmt(y[4], y[6], 0x0040u), 0x5410u) & 0x0f0f0f0fu;
  const uint32_t odd = prmt(prmt(y[1], y[3], 0x0040u), prmt(y[5], y[7], 0x0040u), 0x5410u) & 0x0f0f0f0fu;
  uint32_t code = (even | odd << 4) ^ 0x88888888u;
  if (bad) {
    scale = __ushort_as_half(0);
    code = 0x88888888u;
  } else if (!(top * fabsf(inv) < 8.4f)) {  // (the same for the quad)
    code = divide_all<BF16>(raw, d);
  }
  return code;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(256) kv4_write_kernel(const CellArgs a) {
  using F = Kv4<D>;
  const int total = a.rows_of_block * a.n_kv * F::WORDS;
  const unsigned quad = 0xfu << (threadIdx.x & 28);
  for (int i = threadIdx.x; i < total; i += 256) {
    const Item t = item_of<D>(a, i);
    const long long row = static_cast<long long>(blockIdx.x) * a.rows_of_block + t.row;
    if (!t.in || row >= a.n_rows) continue;  // the same for the whole quad, as the slot's
    const int slot = a.slots[row];
    const long long cells = static_cast<long long>(a.n_pages) << a.page_shift;
    if (slot < 0 || slot >= cells) {
      if (slot >= cells && t.head == 0 && t.w == 0) set_status(a.status, DFLASH_DEV_CAPACITY);
      continue;
    }
    const int col = t.head * D + t.w * 8;
    const uint4 k = __ldcs(reinterpret_cast<const uint4*>(a.k + row * a.k_stride + col));
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(a.v + row * a.v_stride + col));
    __half ks, vs;
    bool kbad, vbad;
    const uint32_t kc = quantise<BF16>(k, t.w, quad, ks, kbad), vc = quantise<BF16>(v, t.w, quad, vs, vbad);
    uint8_t* g = group_of<D>(a, slot, t.head);
    const int cell = slot & 15;
    *reinterpret_cast<uint32_t*>(g + F::k_word(cell, t.w)) = kc;
    *reinterpret_cast<uint32_t*>(g + F::v_word(cell, t.w)) = vc;
    if ((t.w & 3) == 0) {
      *reinterpret_cast<__half*>(g + F::k_scale(cell, t.w >> 2)) = ks;
      *reinterpret_cast<__half*>(g + F::v_scale(cell, t.w >> 2)) = vs;
      if (kbad || vbad) set_status(a.status, DFLASH_DEV_NONFINITE);
    }
  }
}

__device__ __forceinline__ void put_values(float* out, uint32_t code, float d) {
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = d * static_cast<float>(static_cast<int>((code >> (4 * e)) & 15u) - 8);
  // one store of a whole 32-byte sector: two of 16 bytes would each write half of all the warp's sectors
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out), "f"(y[0]), "f"(y[1]), "f"(y[2]),
               "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7])
               : "memory");
}

template <int D>
__global__ void __launch_bounds__(256) kv4_read_kernel(const CellArgs a) {
  using F = Kv4<D>;
  const int total = a.rows_of_block * a.n_kv * F::WORDS;
  for (int i = threadIdx.x; i < total; i += 256) {
    const Item t = item_of<D>(a, i);
    const long long row = static_cast<long long>(blockIdx.x) * a.rows_of_block + t.row;
    if (!t.in || row >= a.n_rows) continue;
    const int slot = a.slots[row];
    const long long cells = static_cast<long long>(a.n_pages) << a.page_shift;
    uint32_t kc = 0, vc = 0;
    float kd = 0.f, vd = 0.f;
    if (slot >= 0 && slot < cells) {
      const uint8_t* g = group_of<D>(a, slot, t.head);
      const int cell = slot & 15;
      kc = *reinterpret_cast<const uint32_t*>(g + F::k_word(cell, t.w));
      vc = *reinterpret_cast<const uint32_t*>(g + F::v_word(cell, t.w));
      kd = __half2float(*reinterpret_cast<const __half*>(g + F::k_scale(cell, t.w >> 2)));
      vd = __half2float(*reinterpret_cast<const __half*>(g + F::v_scale(cell, t.w >> 2)));
    } else if (slot >= cells && t.head == 0 && t.w == 0) {
      set_status(a.status, DFLASH_DEV_CAPACITY);
    }
    const long long at = (row * a.n_kv + t.head) * D + t.w * 8;
    if (a.k_out) put_values(a.k_out + at, kc, kd);
    if (a.v_out) put_values(a.v_out + at, vc, vd);
  }
}

template <int D>
cudaError_t launch(CellArgs a, int type, bool write, cudaStream_t st) {
  const int words = a.n_kv * Kv4<D>::WORDS;  // 8 .. 8192
  a.rows_of_block = words >= 512 ? 1 : 512 / words;
  a.magic = static_cast<uint32_t>(((1ull << 32) + words - 1) / words);
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(a.n_rows) + a.rows_of_block - 1) / a.rows_of_block);
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
  if (!slots || reinterpret_cast<uintptr_t>(k_out) % 32 || reinterpret_cast<uintptr_t>(v_out) % 32)
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
