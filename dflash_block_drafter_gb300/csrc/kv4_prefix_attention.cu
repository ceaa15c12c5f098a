// Attention of requests that share a prefix, over the 4-bit paged K/V cache
// (dflash_kv4_prefix_attention in include/dflash.h).
//
//   o = (sum over prefix cells + sum over own cells) 2^(s_j - m) v_j / (the same of 2^(s_j - m)).
//
// Two passes (kv4_attention.cuh): all rows of a group over the group's prefix, whose cells
// are read and unpacked once per 128 query rows instead of once per request; and each request over its
// own cells, joined with the first where a row is written.  The
// first runs on the tcgen05 kernel, the second on the kernel that a call without a prefix would take.
// Between them lies FP32: each row's maximum, sum and unnormalised O.  The second begins as SMs come free of the first
// and waits for it where it needs what that has left (this step took 64 tokens from 130 to 125 us and 8 tokens over 8192 cells from 45 to 35; with
// the passes in the other order, the prefix's waiting for the own cells', 138 instead of 130).
//
// Measured, calls in a row: 64 tokens of 24 / 2 heads of 256 over 32768 shared and 1 .. 4096 own cells 122 to 126 us (floor 29), 16 blocks of 8 119 to
// 123 (floor 29), 200 tokens of 32 / 8 heads of 128 in five groups 106 (floor 21), 8 tokens over 8192 shared cells 35.  The 64 tokens' launches one by
// one under the profiler: the prefix's products 79 to 82 (480 TFLOP/s, tensor pipe 38 %: a tile's way through eight barriers, as without a
// prefix), its pieces' merge 11, the own cells 33, their merge 8.  Where no group has a prefix, 64 tokens of up to 1023 cells take 51 us, and 27 by
// dflash_kv4_attention.
#include <cstddef>

#include "kv4_attention_warp.cuh"

namespace dflash {
namespace {

struct Call {
  Kv4Shape prefix, own;
  int per_segment;
  size_t prefix_bytes, own_bytes, rows;  // rows: n_tokens * n_q_heads
  size_t bytes(int d) const { return prefix_bytes + own_bytes + rows * (d * 4 + 8); }
};

int check_prefix_call(const dflash_kv4_cache* c, int n_tokens, int n_q_heads, int n_groups, int prefix_stride, int n_seq,
                      int max_rows, int table_stride) {
  if (const int e = kv4_check_call(c, n_q_heads, n_seq, max_rows, table_stride)) return e;
  if (n_tokens < 0 || n_groups < 1 || prefix_stride < 1) return DFLASH_ERR_INVALID_ARG;
  // (rows of sequences; a row of no sequence is not counted in any group)
  if (n_groups > kKv4MaxSeq || static_cast<long long>(prefix_stride) * c->page_size > 0x7fffff00ll) return DFLASH_ERR_CAPACITY;
  if (static_cast<long long>(n_tokens) * n_q_heads > 0x7fffffffll) return DFLASH_ERR_CAPACITY;
  return DFLASH_OK;
}

cudaError_t shape_call(const dflash_kv4_cache* c, int n_tokens, int n_q_heads, int n_groups, int prefix_stride, int n_seq,
                       int max_rows, int table_stride, Call* out) {
  out->per_segment = 128 / (n_q_heads / c->n_kv_heads);
  // (also where a sequence has more than max_rows rows, which is refused: other groups' pieces have their merge)
  const long long segments = (static_cast<long long>(n_tokens / out->per_segment) + n_groups) * c->n_kv_heads;
  cudaError_t e = kv4_tc_shape(c, segments, prefix_stride, &out->prefix);
  if (e == cudaSuccess) e = kv4_shape_of(c, n_q_heads, n_seq, max_rows, table_stride, &out->own);
  if (e != cudaSuccess) return e;
  out->prefix_bytes = kv4_pass_bytes(c, out->prefix);
  out->own_bytes = kv4_pass_bytes(c, out->own);
  out->rows = static_cast<size_t>(n_tokens) * n_q_heads;
  return cudaSuccess;
}

}  // namespace
}  // namespace dflash

using namespace dflash;

extern "C" {

size_t dflash_kv4_prefix_attention_workspace(const dflash_kv4_cache* c, int32_t n_tokens, int32_t n_q_heads,
                                             int32_t n_groups, int32_t prefix_stride, int32_t n_seq, int32_t max_rows,
                                             int32_t table_stride) {
  Call s;
  if (check_prefix_call(c, n_tokens, n_q_heads, n_groups, prefix_stride, n_seq, max_rows, table_stride) != DFLASH_OK ||
      shape_call(c, n_tokens, n_q_heads, n_groups, prefix_stride, n_seq, max_rows, table_stride, &s) != cudaSuccess)
    return 0;
  return s.bytes(c->head_dim);
}

int dflash_kv4_prefix_attention(const dflash_kv4_cache* c, const void* q, void* out, int32_t type, int64_t q_stride,
                                int64_t out_stride, int32_t n_tokens, int32_t n_q_heads, int32_t n_groups,
                                const int32_t* group_offsets, const int32_t* prefix_len, const int32_t* prefix_table,
                                int32_t prefix_stride, int32_t n_seq, int32_t max_rows, const int32_t* row_offsets,
                                const int32_t* kv_len, const int32_t* table, int32_t table_stride, int32_t causal,
                                float scale, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                dflash_stream_t stream) {
  if (const int e = check_prefix_call(c, n_tokens, n_q_heads, n_groups, prefix_stride, n_seq, max_rows, table_stride)) return e;
  if (type != DFLASH_T_BF16 && type != DFLASH_T_FP16) return DFLASH_ERR_UNSUPPORTED;
  const int64_t width = static_cast<int64_t>(n_q_heads) * c->head_dim;
  // (2^127: its product with log2(e) is still finite)
  if (!(scale > 0.f) || !(scale <= 0x1p127f)) return DFLASH_ERR_INVALID_ARG;
  if (!group_offsets || !prefix_len || !prefix_table || !row_offsets || !kv_len || !table) return DFLASH_ERR_INVALID_ARG;
  if (n_tokens == 0) return DFLASH_OK;
  if (!q || !out || reinterpret_cast<uintptr_t>(q) % 16 || reinterpret_cast<uintptr_t>(out) % 16 || q_stride < width ||
      out_stride < width || q_stride % 8 || out_stride % 8)
    return DFLASH_ERR_INVALID_ARG;
  Call s;
  cudaError_t e = shape_call(c, n_tokens, n_q_heads, n_groups, prefix_stride, n_seq, max_rows, table_stride, &s);
  if (e != cudaSuccess) return cuda_status(e, "kv4 prefix attention");
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16) return DFLASH_ERR_INVALID_ARG;
  if (workspace_bytes < s.bytes(c->head_dim)) return DFLASH_ERR_CAPACITY;
  uint8_t* w = static_cast<uint8_t*>(workspace);
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
  a.max_rows = max_rows;
  a.n_tokens = n_tokens;
  a.row_offsets = row_offsets;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.status = dev_status;
  a.group_offsets = group_offsets;
  a.n_all = n_seq;
  a.per_segment = s.per_segment;
  a.pre = reinterpret_cast<float*>(w + s.prefix_bytes + s.own_bytes);
  a.pre_ml = reinterpret_cast<float2*>(a.pre + s.rows * c->head_dim);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);

  Kv4AttnArgs b = a;  // every row sees the whole prefix
  b.n_seq = n_groups;
  b.kv_len = prefix_len;
  b.table = prefix_table;
  b.table_stride = prefix_stride;
  kv4_set_workspace(b, c, s.prefix, w);
  e = launch_kv4_attn_tc_prefix(c->head_dim, b, s.prefix.most, s.prefix.jobs, st);
  if (e != cudaSuccess) return cuda_status(e, "kv4 prefix attention");

  a.n_seq = n_seq;
  a.kv_len = kv_len;
  a.table = table;
  a.table_stride = table_stride;
  a.causal = causal != 0;
  kv4_set_workspace(a, c, s.own, w + s.prefix_bytes);
  if (s.own.tc) {
    e = launch_kv4_attn_tc_own(c->head_dim, a, s.own.most, s.own.jobs, st);
  } else {
    switch (c->head_dim) {
      case 64: e = launch_nt<64, kKv4Own>(a, s.own, st); break;
      case 128: e = launch_nt<128, kKv4Own>(a, s.own, st); break;
      default: e = launch_nt<256, kKv4Own>(a, s.own, st); break;
    }
  }
  return cuda_status(e, "kv4 prefix attention");
}

}  // extern "C"
