// Log probabilities of given tokens with the distribution's entropy and its
// top alternatives (dflash_token_logprobs in include/dflash.h).
//
//   lse = m + ln s,  s = sum_x e^(x - m),  t = sum_x e^(x - m) (x - m)
//   logp(i) = (x_i - m) - ln s,  H = ln s - t / s,  m = max x.
//
// One pass over the logits: a thread keeps m, s and t of what it has read
// and rescales them when a batch of its values holds a larger one
// (t' = r (t + (m - m') s), s' = r s, r = e^(m - m')).  Everything is FP32; x - m
// is formed before the factor log2(e), so that large logits lose nothing.  A row's
// bytes bound the time: 16-byte loads, four in flight per thread.
//
// Top alternatives: each warp keeps the 32 largest (value, lower id first)
// keys it has met, sorted across its lanes.  A warp reads its row in
// ascending batches, so once its list is full only a value above the list's
// k-th can enter, which one comparison per batch decides; lists are joined
// by bitonic merges at the end.
//
// With few rows a row's batches are split over several CTAs, whose results
// a second kernel joins.
#include <cstddef>

#include "common.cuh"
#include "internal.h"
#include "kernels.h"

namespace dflash {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kLoads = 4;      // 16-byte loads of a thread per batch
constexpr int kMaxTop = 32;
constexpr int kMaxSplits = 32;
constexpr float kLog2e = 1.4426950408889634f;
using Key = unsigned long long;

struct LogprobArgs {
  const uint8_t* logits;
  long long row_bytes;
  int n_rows, vocab, splits, k;
  const int32_t* tokens;
  float* logprob;
  float* entropy;
  int32_t* top_ids;
  float* top_logprobs;
  float4* part;  // [rows][splits]: m, s, t
  Key* part_key; // [rows][splits][k]
  int32_t* status;
};

template <int TYPE>
struct Elem {
  static constexpr int BYTES = TYPE == DFLASH_T_FP32 ? 4 : 2;
  static constexpr int VEC = 16 / BYTES;
  static __device__ __forceinline__ void widen(uint4 v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (TYPE == DFLASH_T_FP32) {
        x[i] = __uint_as_float(w[i]);
      } else if constexpr (TYPE == DFLASH_T_BF16) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
  }
  static __device__ __forceinline__ float one(const uint8_t* row, int i) {
    if constexpr (TYPE == DFLASH_T_FP32) return __ldg(reinterpret_cast<const float*>(row) + i);
    const uint16_t h = __ldg(reinterpret_cast<const uint16_t*>(row) + i);
    if constexpr (TYPE == DFLASH_T_BF16) return __uint_as_float(static_cast<uint32_t>(h) << 16);
    return __half2float(__ushort_as_half(h));
  }
};

// m, s, t of two disjoint sets of values.
struct Stat {
  float m, s, t;
};
__device__ __forceinline__ Stat join(Stat a, Stat b) {
  Stat r;
  r.m = fmaxf(a.m, b.m);
  if (r.m == -INFINITY) {  // no finite value in either (a NaN shows in s)
    r.s = a.s + b.s;
    r.t = a.t + b.t;
    return r;
  }
  // a set without values has s = t = 0, whatever factor it gets
  const float da = a.m == -INFINITY ? 0.f : a.m - r.m, db = b.m == -INFINITY ? 0.f : b.m - r.m;
  // a difference below the clamp has factor 0: keep 0 * inf out of t
  const float fa = ex2_approx(da * kLog2e), fb = ex2_approx(db * kLog2e);
  r.s = a.s * fa + b.s * fb;
  r.t = fa * fmaf(fmaxf(da, -150.f), a.s, a.t) + fb * fmaf(fmaxf(db, -150.f), b.s, b.t);
  return r;
}

__device__ __forceinline__ Key make_key(float x, int id) {
  return (static_cast<Key>(float_order_key(x + 0.f)) << 32) | (0xffffffffu - static_cast<uint32_t>(id));
}

// 32 keys, one per lane, in descending order from a bitonic sequence.
__device__ __forceinline__ Key bitonic(Key v, int lane) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const Key u = __shfl_xor_sync(0xffffffffu, v, o);
    v = ((lane & o) != 0) == (u < v) ? u : v;
  }
  return v;
}
// The 32 largest of two descending lists (other: read backwards).
__device__ __forceinline__ Key join_lists(Key v, Key other_reversed, int lane) {
  return bitonic(v > other_reversed ? v : other_reversed, lane);
}

// Outputs of a row by one warp; lane i holds the i-th key.
template <int TYPE>
__device__ __forceinline__ void finish_row(const LogprobArgs& a, int row, Stat st, Key key, int lane) {
  const bool some = st.m > -INFINITY;
  const float ln_s = logf(st.s);
  if (lane == 0) {
    if (!(st.s < INFINITY) || !(st.m < INFINITY)) set_status(a.status, DFLASH_DEV_NONFINITE);
    if (a.entropy) a.entropy[row] = some ? ln_s - st.t / st.s : 0.f;
    if (a.logprob) {
      const int tok = a.tokens[row];
      float r = 0.f;
      if (tok >= 0 && tok < a.vocab) {
        const float x = Elem<TYPE>::one(a.logits + row * a.row_bytes, tok);
        r = some ? (x - st.m) - ln_s : -INFINITY;
      } else if (tok != -1) {
        set_status(a.status, DFLASH_DEV_BAD_TOKEN);
      }
      a.logprob[row] = r;
    }
  }
  if (lane < a.k) {
    const size_t at = static_cast<size_t>(row) * a.k + lane;
    a.top_ids[at] = key ? static_cast<int>(0xffffffffu - static_cast<uint32_t>(key)) : -1;
    a.top_logprobs[at] = key ? (float_from_order_key(static_cast<uint32_t>(key >> 32)) - st.m) - ln_s : -INFINITY;
  }
}

template <int TYPE, bool TOP>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LogprobArgs a) {
  using E = Elem<TYPE>;
  constexpr int VEC = E::VEC, N = kLoads * VEC, BATCH = 32 * N;
  __shared__ Stat s_stat[kWarps];
  __shared__ Key s_key[kWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x / a.splits, split = blockIdx.x - row * a.splits;
  const uint8_t* src = a.logits + row * a.row_bytes;
  // the row in a frame of whole 16-byte pieces: value i lies at place i + skip
  const int skip = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15) / E::BYTES;
  const uint4* frame = reinterpret_cast<const uint4*>(src - skip * E::BYTES);
  const long long places = static_cast<long long>(a.vocab) + skip;
  const int batches = static_cast<int>((places + BATCH - 1) / BATCH);
  Stat st{-INFINITY, 0.f, 0.f};
  Key list = 0, kth = 0;
  float bar = -INFINITY;  // value of the k-th key
  for (int b = split * kWarps + warp; b < batches; b += a.splits * kWarps) {
    float x[N];
    const long long p0 = static_cast<long long>(b) * BATCH;
    if (p0 >= skip && p0 + BATCH <= places) {
      uint4 v[kLoads];
#pragma unroll
      for (int j = 0; j < kLoads; ++j) v[j] = __ldg(frame + p0 / VEC + j * 32 + lane);
#pragma unroll
      for (int j = 0; j < kLoads; ++j) E::widen(v[j], x + j * VEC);
    } else {
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const long long p = p0 + (j * 32 + lane) * VEC;
        if (p >= skip && p + VEC <= places) {
          E::widen(__ldg(frame + p / VEC), x + j * VEC);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            x[j * VEC + e] = p + e >= skip && p + e < places ? E::one(src, static_cast<int>(p + e - skip)) : -INFINITY;
        }
      }
    }
    float top = x[0];
#pragma unroll
    for (int e = 1; e < N; ++e) top = fmaxf(top, x[e]);
    if (top > st.m) {
      if (st.m > -INFINITY) {
        const float d = st.m - top, r = ex2_approx(d * kLog2e);
        st.t = r * fmaf(fmaxf(d, -150.f), st.s, st.t);
        st.s *= r;
      }
      st.m = top;
    }
    const float from = st.m == -INFINITY ? 0.f : st.m;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float z = x[e] - from, w = ex2_approx(z * kLog2e);
      st.s += w;
      st.t = fmaf(w, fmaxf(z, -150.f), st.t);  // a value of no weight adds no 0 * inf
    }
    if constexpr (TOP) {
      if (__any_sync(0xffffffffu, top > bar)) {
        const int id0 = static_cast<int>(p0 - skip) + lane * VEC;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          unsigned in = __ballot_sync(0xffffffffu, x[e] >= bar && x[e] > -INFINITY);
          if (in) {
            const Key mine = make_key(x[e], id0 + (e / VEC) * 32 * VEC + e % VEC);
            for (; in; in &= in - 1) {
              const Key one = __shfl_sync(0xffffffffu, mine, __ffs(in) - 1);
              if (one <= kth) continue;
              const int at = __popc(__ballot_sync(0xffffffffu, list > one));
              const Key up = __shfl_up_sync(0xffffffffu, list, 1);
              list = lane < at ? list : lane == at ? one : up;
              kth = __shfl_sync(0xffffffffu, list, a.k - 1);
            }
            if (kth) bar = float_from_order_key(static_cast<uint32_t>(kth >> 32));
          }
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1)
    st = join(st, Stat{__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.s, o),
                       __shfl_xor_sync(0xffffffffu, st.t, o)});
  if (lane == 0) s_stat[warp] = st;
  if (TOP) s_key[warp][lane] = list;
  __syncthreads();
  if (warp) return;
  for (int w = 1; w < kWarps; ++w) {
    st = join(st, s_stat[w]);
    if (TOP) list = join_lists(list, s_key[w][31 - lane], lane);
  }
  if (a.splits == 1) {
    finish_row<TYPE>(a, row, st, list, lane);
    return;
  }
  if (lane == 0) a.part[blockIdx.x] = make_float4(st.m, st.s, st.t, 0.f);
  if (TOP && lane < a.k) a.part_key[static_cast<size_t>(blockIdx.x) * a.k + lane] = list;
}

// Joins the splits of a row; one warp each.
template <int TYPE, bool TOP>
__global__ void __launch_bounds__(32) logprobs_join_kernel(const LogprobArgs a) {
  const int row = blockIdx.x, lane = threadIdx.x;
  pdl_wait();
  Stat st{-INFINITY, 0.f, 0.f};
  if (lane < a.splits) {
    const float4 v = __ldcg(a.part + static_cast<size_t>(row) * a.splits + lane);
    st = Stat{v.x, v.y, v.z};
  }
#pragma unroll
  for (int o = 16; o; o >>= 1)
    st = join(st, Stat{__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.s, o),
                       __shfl_xor_sync(0xffffffffu, st.t, o)});
  Key list = 0;
  if (TOP) {
    const Key* keys = a.part_key + static_cast<size_t>(row) * a.splits * a.k;
    for (int i = 0; i < a.splits; ++i) {
      const int from = 31 - lane;
      list = join_lists(list, from < a.k ? __ldcg(keys + i * a.k + from) : 0, lane);
    }
  }
  finish_row<TYPE>(a, row, st, list, lane);
}

// CTAs per row: enough for two per SM, each warp with a batch at least.
cudaError_t splits_of(int n_rows, int vocab, int type, int* out) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int batch = 32 * kLoads * (type == DFLASH_T_FP32 ? 4 : 8);
  const int most = (vocab + batch * kWarps - 1) / (batch * kWarps);
  int s = (2 * sms + n_rows - 1) / n_rows;
  s = s < most ? s : most;
  s = s < kMaxSplits ? s : kMaxSplits;
  *out = s < 1 ? 1 : s;
  return cudaSuccess;
}

template <int TYPE, bool TOP>
cudaError_t launch_typed(const LogprobArgs& a, cudaStream_t st) {
  logprobs_kernel<TYPE, TOP><<<static_cast<unsigned>(a.n_rows) * a.splits, kThreads, 0, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.splits == 1) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.n_rows);
  cfg.blockDim = dim3(32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logprobs_join_kernel<TYPE, TOP>, a);
}

template <int TYPE>
cudaError_t launch(const LogprobArgs& a, cudaStream_t st) {
  return a.k ? launch_typed<TYPE, true>(a, st) : launch_typed<TYPE, false>(a, st);
}

bool known_type(int type) { return type == DFLASH_T_FP32 || type == DFLASH_T_BF16 || type == DFLASH_T_FP16; }

size_t bytes_of(int n_rows, int splits, int k) {
  return splits == 1 ? 0 : static_cast<size_t>(n_rows) * splits * (16 + 8 * static_cast<size_t>(k));
}

}  // namespace
}  // namespace dflash

using namespace dflash;

extern "C" {

size_t dflash_token_logprobs_workspace(int32_t n_rows, int32_t vocab, int32_t type, int32_t top_k) {
  int s = 0;
  if (n_rows < 1 || vocab < 1 || !known_type(type) || top_k < 0 || top_k > kMaxTop ||
      splits_of(n_rows, vocab, type, &s) != cudaSuccess)
    return 0;
  return bytes_of(n_rows, s, top_k);
}

int dflash_token_logprobs(const void* logits, int32_t type, int64_t row_stride, int32_t n_rows, int32_t vocab,
                          const int32_t* tokens, float* logprob, float* entropy, int32_t top_k, int32_t* top_ids,
                          float* top_logprobs, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                          dflash_stream_t stream) {
  if (!known_type(type)) return DFLASH_ERR_UNSUPPORTED;
  if (n_rows < 0 || vocab < 1 || vocab > (1 << 30) || row_stride < vocab || top_k < 0) return DFLASH_ERR_INVALID_ARG;
  if (top_k > kMaxTop) return DFLASH_ERR_CAPACITY;
  if (n_rows == 0) return DFLASH_OK;
  const int size = type == DFLASH_T_FP32 ? 4 : 2;
  if (!logits || reinterpret_cast<uintptr_t>(logits) % size) return DFLASH_ERR_INVALID_ARG;
  if (!tokens != !logprob || (top_k && (!top_ids || !top_logprobs))) return DFLASH_ERR_INVALID_ARG;
  if (!tokens && !entropy && !top_k) return DFLASH_ERR_INVALID_ARG;
  LogprobArgs a{};
  cudaError_t e = splits_of(n_rows, vocab, type, &a.splits);
  if (e != cudaSuccess) return cuda_status(e, "token logprobs");
  const size_t need = bytes_of(n_rows, a.splits, top_k);
  if (need) {
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16) return DFLASH_ERR_INVALID_ARG;
    if (workspace_bytes < need) return DFLASH_ERR_CAPACITY;
  }
  a.logits = static_cast<const uint8_t*>(logits);
  a.row_bytes = row_stride * size;
  a.n_rows = n_rows;
  a.vocab = vocab;
  a.k = top_k;
  a.tokens = tokens;
  a.logprob = logprob;
  a.entropy = entropy;
  a.top_ids = top_ids;
  a.top_logprobs = top_logprobs;
  a.part = static_cast<float4*>(workspace);
  a.part_key = reinterpret_cast<Key*>(a.part + static_cast<size_t>(n_rows) * a.splits);
  a.status = dev_status;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  e = type == DFLASH_T_FP32 ? launch<DFLASH_T_FP32>(a, st)
      : type == DFLASH_T_BF16 ? launch<DFLASH_T_BF16>(a, st)
                              : launch<DFLASH_T_FP16>(a, st);
  return cuda_status(e, "token logprobs");
}

}  // extern "C"
