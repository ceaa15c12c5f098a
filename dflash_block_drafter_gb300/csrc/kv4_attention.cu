// dflash_kv4_attention: the choice of the kernel and its shape, the C entry.
#include <cstddef>

#include "kv4_attention_warp.cuh"

namespace dflash {
namespace {

// Shared memory of an SM, and what a CTA takes of it besides its dynamic part
// (its static arrays and the system's 1 KB).
constexpr int kSmemOfSm = 228 * 1024, kStaticSmem = 2560;
struct CtaCost {
  int smem, per_sm;
};
CtaCost cost_of(int d, int nt) {
  switch (d * 8 + nt) {
#define DFLASH_KV4_COST(D, NT) \
  case D * 8 + NT: return {Geo<D, NT>::SMEM, Geo<D, NT>::PER_SM};
#define DFLASH_KV4_COSTS(D) \
  DFLASH_KV4_COST(D, 1) DFLASH_KV4_COST(D, 2) DFLASH_KV4_COST(D, 3) DFLASH_KV4_COST(D, 4)
    DFLASH_KV4_COSTS(64)
    DFLASH_KV4_COSTS(128)
    DFLASH_KV4_COSTS(256)
#undef DFLASH_KV4_COSTS
#undef DFLASH_KV4_COST
  }
  return {kSmemOfSm, 1};
}

// More rows per kv head than this go to the tcgen05 kernel.  Measured, here and there:
//   16 sequences of 2048 .. 32768 cells, 2 kv heads of 256: 12 rows 58 and 98 us, 24 rows
//   81 and 100, 32 rows 91 and 101 (floor 25);
//   64 of 512 .. 8192 cells, 8 kv heads of 128: 24 rows 154 and 255, 32 rows 182 and 255
//   (floor 53); of 64: 24 rows 110 and 164, 32 rows 128 and 164 (floor 26).
// Beyond, a kernel of this kind would unpack every cell once per 32 rows.
constexpr int kTcRows = 32;

}  // namespace

cudaError_t kv4_tc_shape(const dflash_kv4_cache* c, long long segments, int table_stride, Kv4Shape* out) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  out->tc = true;
  out->nt = 0;
  const int tile = c->head_dim == 256 ? 64 : 128;
  const long long tiles = (static_cast<long long>(table_stride) * c->page_size + tile - 1) / tile + 1;
  out->most = static_cast<int>(segments * tiles < sms ? segments * tiles : sms);
  out->jobs = static_cast<int>(segments < out->most ? segments : out->most);
  return cudaSuccess;
}

cudaError_t kv4_shape_of(const dflash_kv4_cache* c, int n_q_heads, int n_seq, int max_rows, int table_stride, Kv4Shape* out) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int rows = n_q_heads / c->n_kv_heads * max_rows;
  if (rows > kTcRows) return kv4_tc_shape(c, static_cast<long long>(n_seq) * c->n_kv_heads, table_stride, out);
  out->tc = false;
  out->nt = (rows + 7) / 8;
  const int tile = 128;
  const long long segments = static_cast<long long>(n_seq) * c->n_kv_heads;
  // (a window may begin anywhere in a tile)
  const long long tiles = (static_cast<long long>(table_stride) * c->page_size + tile - 1) / tile + 1;
  const long long ctas = segments * (tiles + kOverhead);
  // one wave of CTAs: every one of them has the same share
  const CtaCost cost = cost_of(c->head_dim, out->nt);
  const int fit = kSmemOfSm / (cost.smem + kPlanBytes(n_seq) + kStaticSmem);
  const int per_sm = fit < cost.per_sm ? fit : cost.per_sm;
  out->most = static_cast<int>(ctas < per_sm * sms ? ctas : per_sm * sms);
  out->jobs = static_cast<int>(segments < out->most ? segments : out->most);
  return cudaSuccess;
}

int kv4_check_call(const dflash_kv4_cache* c, int n_q_heads, int n_seq, int max_rows, int table_stride) {
  if (const int e = dflash_kv4_check(c)) return e;
  if (n_seq < 1 || table_stride < 1 || n_q_heads < 1 || n_q_heads % c->n_kv_heads) return DFLASH_ERR_INVALID_ARG;
  if (max_rows < 1 || max_rows > DFLASH_MAX_BLOCK) return DFLASH_ERR_INVALID_ARG;
  // (positions up to a tile behind the table's last stay within 31 bits)
  if (n_seq > kKv4MaxSeq || static_cast<long long>(table_stride) * c->page_size > 0x7fffff00ll) return DFLASH_ERR_CAPACITY;
  if (n_q_heads / c->n_kv_heads * max_rows > 128) return DFLASH_ERR_UNSUPPORTED;
  return DFLASH_OK;
}

}  // namespace dflash

using namespace dflash;

extern "C" {

size_t dflash_kv4_attention_workspace(const dflash_kv4_cache* c, int32_t n_q_heads, int32_t n_seq, int32_t max_rows,
                                      int32_t table_stride) {
  Kv4Shape s;
  if (kv4_check_call(c, n_q_heads, n_seq, max_rows, table_stride) != DFLASH_OK ||
      kv4_shape_of(c, n_q_heads, n_seq, max_rows, table_stride, &s) != cudaSuccess)
    return 0;
  return kv4_pass_bytes(c, s);
}

int dflash_kv4_attention(const dflash_kv4_cache* c, const void* q, void* out, int32_t type, int64_t q_stride,
                         int64_t out_stride, int32_t n_tokens, int32_t n_q_heads, int32_t n_seq, int32_t max_rows,
                         const int32_t* row_offsets, const int32_t* kv_len, const int32_t* table, int32_t table_stride,
                         int32_t causal, int32_t window, float scale, void* workspace, size_t workspace_bytes,
                         int32_t* dev_status, dflash_stream_t stream) {
  if (const int e = kv4_check_call(c, n_q_heads, n_seq, max_rows, table_stride)) return e;
  if (type != DFLASH_T_BF16 && type != DFLASH_T_FP16) return DFLASH_ERR_UNSUPPORTED;
  const int64_t width = static_cast<int64_t>(n_q_heads) * c->head_dim;
  // (2^127: its product with log2(e) is still finite)
  if (n_tokens < 0 || window < 0 || !(scale > 0.f) || !(scale <= 0x1p127f)) return DFLASH_ERR_INVALID_ARG;
  if (!row_offsets || !kv_len || !table) return DFLASH_ERR_INVALID_ARG;
  if (n_tokens == 0) return DFLASH_OK;
  if (!q || !out || reinterpret_cast<uintptr_t>(q) % 16 || reinterpret_cast<uintptr_t>(out) % 16 || q_stride < width ||
      out_stride < width || q_stride % 8 || out_stride % 8)
    return DFLASH_ERR_INVALID_ARG;
  Kv4Shape s;
  cudaError_t e = kv4_shape_of(c, n_q_heads, n_seq, max_rows, table_stride, &s);
  if (e != cudaSuccess) return cuda_status(e, "kv4 attention");
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16) return DFLASH_ERR_INVALID_ARG;
  if (workspace_bytes < kv4_pass_bytes(c, s)) return DFLASH_ERR_CAPACITY;
  Kv4AttnArgs a{};
  a.cache = static_cast<const uint8_t*>(c->data);
  a.n_pages = c->n_pages;
  a.page_shift = log2_page(c);
  a.n_kv = c->n_kv_heads;
  a.G = n_q_heads / c->n_kv_heads;
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.bf16 = type == DFLASH_T_BF16;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.n_seq = n_seq;
  a.max_rows = max_rows;
  a.n_tokens = n_tokens;
  a.row_offsets = row_offsets;
  a.kv_len = kv_len;
  a.table = table;
  a.table_stride = table_stride;
  a.causal = causal != 0;
  a.window = window;
  a.scale_log2 = scale * 1.4426950408889634f;
  kv4_set_workspace(a, c, s, workspace);
  a.status = dev_status;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (s.tc) {
    e = launch_kv4_attn_tc(c->head_dim, a, s.most, s.jobs, st);
  } else {
    switch (c->head_dim) {
      case 64: e = launch_nt<64, kKv4Plain>(a, s, st); break;
      case 128: e = launch_nt<128, kKv4Plain>(a, s, st); break;
      default: e = launch_nt<256, kKv4Plain>(a, s, st); break;
    }
  }
  return cuda_status(e, "kv4 attention");
}

}  // extern "C"
