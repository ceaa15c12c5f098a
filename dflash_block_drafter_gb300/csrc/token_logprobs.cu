// Log probabilities of given tokens with the distribution's entropy and its
// top alternatives (dflash_token_logprobs in include/dflash.h).
//
//   lse = m + ln s,  s = sum_x e^(x - m),  t = sum_x e^(x - m) (x - m)
//   logp(i) = (x_i - m) - ln s,  H = ln s - t / s,  m = max x.
//
// One pass over the logits: a thread keeps m, s and t of what it has read
// and rescales them when a batch of its values holds a larger one
// (t' = r (t + (m - m') s), s' = r s, r = e^(m - m')).  Everything is FP32; x - m
// is formed before the factor log2(e), so that large logits lose nothing.  Without
// alternatives a row's bytes bound the time: four 16-byte loads in flight per
// thread, and pairs of FP32 values in one instruction where there is one.  A masked value (-infinity) would add 0 * infinity to t: a batch that
// shows it is done again with x - m clamped, and so are the row's later ones.
//
// Top alternatives: each warp keeps the 32 largest (value, lower id first)
// keys it has met, sorted across its lanes.  A warp reads its row in
// ascending batches, so once its list is full only a value above the list's
// k-th can enter, and none below the k-th largest of what all warps have met;
// the warps compare their lists after the first and the fourth batch, after
// which few batches bring anything.  Lists are joined by bitonic merges.
//
// With few rows a row's batches are split over the CTAs of a cluster; their
// results meet in the first one's shared memory.
//
// Measured: 2000 rows of 151936 BF16 logits 108 us without alternatives (5.6 TB/s),
// 141 us with the top 5; 128 rows of 100003 FP32 with the top 20 31 us, of which half is
// the latency of insertions and joins.
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
constexpr int kMaxSplits = 16;  // CTAs of a cluster
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
  // the larger of two 32-bit words' values, value by value; the larger value of a word
  static __device__ __forceinline__ uint32_t max_words(uint32_t a, uint32_t b) {
    if constexpr (TYPE == DFLASH_T_FP32) {
      return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    } else if constexpr (TYPE == DFLASH_T_BF16) {
      const __nv_bfloat162 m = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
      return *reinterpret_cast<const uint32_t*>(&m);
    } else {
      const __half2 m = __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
      return *reinterpret_cast<const uint32_t*>(&m);
    }
  }
  static __device__ __forceinline__ float max_of(uint32_t w) {
    if constexpr (TYPE == DFLASH_T_FP32) return __uint_as_float(w);
    if constexpr (TYPE == DFLASH_T_BF16) return fmaxf(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return fmaxf(f.x, f.y);
  }
  // a word whose values are -infinity
  static constexpr uint32_t NOTHING = TYPE == DFLASH_T_FP32 ? 0xff800000u : TYPE == DFLASH_T_BF16 ? 0xff80ff80u : 0xfc00fc00u;
  // the word of two (one for FP32) values of a row
  static __device__ __forceinline__ uint32_t raw(const uint8_t* row, long long i, long long n) {
    if constexpr (TYPE == DFLASH_T_FP32) {
      return i >= 0 && i < n ? __ldg(reinterpret_cast<const uint32_t*>(row) + i) : NOTHING;
    } else {
      const uint32_t lo = i >= 0 && i < n ? __ldg(reinterpret_cast<const uint16_t*>(row) + i) : NOTHING & 0xffffu;
      const uint32_t hi = i + 1 >= 0 && i + 1 < n ? __ldg(reinterpret_cast<const uint16_t*>(row) + i + 1) : NOTHING & 0xffffu;
      return lo | hi << 16;
    }
  }
  // value i of a lane's pieces
  static __device__ __forceinline__ float shown(const uint4* p, int i) {
    if constexpr (TYPE == DFLASH_T_FP32) return reinterpret_cast<const float*>(p)[i];
    const uint16_t h = reinterpret_cast<const uint16_t*>(p)[i];
    if constexpr (TYPE == DFLASH_T_BF16) return __uint_as_float(static_cast<uint32_t>(h) << 16);
    return __half2float(__ushort_as_half(h));
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

// The lanes' values in descending order.
__device__ __forceinline__ float sort_down(float v, int lane) {
#pragma unroll
  for (int n = 2; n <= 32; n <<= 1)
#pragma unroll
    for (int o = n >> 1; o; o >>= 1) {
      const float u = __shfl_xor_sync(0xffffffffu, v, o);
      const bool up = (lane & n) != 0;  // (at n = 32 no lane)
      v = ((lane & o) != 0) != up ? fminf(u, v) : fmaxf(u, v);
    }
  return v;
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

// The running results of a thread: m, and s and t as two partial sums each.
struct Running {
  float m;
  uint64_t s, t;
};

template <int TYPE>
__device__ __forceinline__ void add_batch(Running& r, const uint4 (&v)[kLoads], float from, bool clamp) {
  using E = Elem<TYPE>;
  const uint64_t minus = pack2(-from, -from), log2e = pack2(kLog2e, kLog2e);
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    float x[E::VEC];
    E::widen(v[j], x);
#pragma unroll
    for (int e = 0; e < E::VEC; e += 2) {
      uint64_t z = add2(pack2(x[e], x[e + 1]), minus);
      float y0, y1;
      unpack2(mul2(z, log2e), y0, y1);
      const uint64_t w = pack2(ex2_approx(y0), ex2_approx(y1));
      r.s = add2(r.s, w);
      if (clamp) {  // a value of no weight adds no 0 * infinity
        float z0, z1;
        unpack2(z, z0, z1);
        z = pack2(fmaxf(z0, -150.f), fmaxf(z1, -150.f));
      }
      r.t = fma2(w, z, r.t);
    }
  }
}

template <int TYPE, bool TOP>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(const LogprobArgs a) {
  using E = Elem<TYPE>;
  constexpr int VEC = E::VEC, BATCH = 32 * kLoads * VEC;
  __shared__ Stat s_stat[kWarps], s_other[kMaxSplits];
  __shared__ Key s_key[kWarps][32], s_other_key[kMaxSplits][32];
  __shared__ uint4 s_row[kWarps][kLoads];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x / a.splits, split = blockIdx.x - row * a.splits;
  const uint8_t* src = a.logits + row * a.row_bytes;
  // the row in a frame of whole 16-byte pieces: value i lies at place i + skip
  const int skip = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15) / E::BYTES;
  const uint4* frame = reinterpret_cast<const uint4*>(src - skip * E::BYTES);
  const long long places = static_cast<long long>(a.vocab) + skip;
  const int batches = static_cast<int>((places + BATCH - 1) / BATCH);
  const int step = a.splits * kWarps;
  auto load = [&](int b, uint4 (&v)[kLoads]) {
    const long long p0 = static_cast<long long>(b) * BATCH;
    if (p0 >= skip && p0 + BATCH <= places) {
#pragma unroll
      for (int j = 0; j < kLoads; ++j) v[j] = __ldg(frame + p0 / VEC + j * 32 + lane);
    } else {  // the row's ends: value by value
#pragma unroll 1
      for (int j = 0; j < kLoads; ++j) {
        const long long i = p0 + (j * 32 + lane) * VEC - skip;
        constexpr int W = VEC / 4;  // values of a word
        uint4 u;
        u.x = E::raw(src, i, a.vocab);
        u.y = E::raw(src, i + W, a.vocab);
        u.z = E::raw(src, i + 2 * W, a.vocab);
        u.w = E::raw(src, i + 3 * W, a.vocab);
        if (j == 0) v[0] = u;
        else if (j == 1) v[1] = u;
        else if (j == 2) v[2] = u;
        else v[3] = u;
      }
    }
  };
  static_assert(kLoads == 4, "load");
  Running r{-INFINITY, 0, 0};
  bool masked = false;
  Key list = 0, kth = 0;
  float own = -INFINITY, all = -INFINITY;  // k-th value of this warp's list; of what all warps had met
  uint4 v[kLoads];
  int b = split * kWarps + warp;
  if (b < batches) load(b, v);
  int stage = 0;
  for (int it = 0;; ++it, b += step) {
    if (TOP && (it == 1 || it == 4)) {
      // the k-th largest of all warps' lists
      s_key[warp][lane] = list;
      __syncthreads();
      Key top = s_key[0][lane];
      for (int w = 1; w < kWarps; ++w) top = join_lists(top, s_key[w][31 - lane], lane);
      const Key k = __shfl_sync(0xffffffffu, top, a.k - 1);
      if (k) all = float_from_order_key(static_cast<uint32_t>(k >> 32));
      __syncthreads();
      ++stage;
    }
    if (b >= batches) {
      if (TOP && stage < 2) continue;  // the other warps still compare lists
      break;
    }
    uint32_t mw = E::NOTHING;
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      mw = E::max_words(E::max_words(mw, E::max_words(v[j].x, v[j].y)), E::max_words(v[j].z, v[j].w));
    const float top = E::max_of(mw);
    if (top > r.m) {
      if (r.m > -INFINITY) {
        const float d = r.m - top, f = ex2_approx(d * kLog2e), dc = fmaxf(d, -150.f);
        r.t = mul2(fma2(pack2(dc, dc), r.s, r.t), pack2(f, f));
        r.s = mul2(r.s, pack2(f, f));
      }
      r.m = top;
    }
    const float from = r.m == -INFINITY ? 0.f : r.m;
    const Running before = r;
    const long long p0 = static_cast<long long>(b) * BATCH;
    bool clamp = masked || p0 < skip || p0 + BATCH > places;  // (places beyond the row are filled as masked ones)
    if (!clamp) {
      add_batch<TYPE>(r, v, from, false);
      float t0, t1;
      unpack2(r.t, t0, t1);
      clamp = masked = __any_sync(0xffffffffu, !(t0 + t1 > -INFINITY));  // (NaN or -infinity)
      if (clamp) r = before;
    }
    if (clamp) add_batch<TYPE>(r, v, from, true);
    if constexpr (TOP) {
      if (it == 0) {
        // the k-th largest of the lanes' maxima bounds the k-th largest value
        const float k_top = __shfl_sync(0xffffffffu, sort_down(top, lane), a.k - 1);
        all = fmaxf(all, k_top);
      }
      // lanes that may have a value that enters (equal to `all`: it may have the
      // lower id): each shows its values to the warp, one per lane
      for (unsigned hits = __ballot_sync(0xffffffffu, top > own && top >= all && top > -INFINITY); hits; hits &= hits - 1) {
        const int from_lane = __ffs(hits) - 1;
        if (lane == from_lane)
#pragma unroll
          for (int j = 0; j < kLoads; ++j) s_row[warp][j] = v[j];
        __syncwarp();
        constexpr int N = kLoads * VEC;  // values of a lane
        const float x = lane < N ? E::shown(s_row[warp], lane) : -INFINITY;
        __syncwarp();
        const int id = static_cast<int>(p0 - skip) + from_lane * VEC + (lane / VEC) * 32 * VEC + lane % VEC;
        const Key mine = make_key(x, id);
        for (unsigned in = __ballot_sync(0xffffffffu, x >= own && x >= all && x > -INFINITY); in; in &= in - 1) {
          const Key one = __shfl_sync(0xffffffffu, mine, __ffs(in) - 1);
          if (one <= kth) continue;
          const int at = __popc(__ballot_sync(0xffffffffu, list > one));
          const Key up = __shfl_up_sync(0xffffffffu, list, 1);
          list = lane < at ? list : lane == at ? one : up;
          kth = __shfl_sync(0xffffffffu, list, a.k - 1);
        }
        if (kth) own = float_from_order_key(static_cast<uint32_t>(kth >> 32));
      }
    }
    if (b + step < batches) load(b + step, v);
  }
  float s0, s1, t0, t1;
  unpack2(r.s, s0, s1);
  unpack2(r.t, t0, t1);
  Stat st{r.m, s0 + s1, t0 + t1};
#pragma unroll
  for (int o = 16; o; o >>= 1)
    st = join(st, Stat{__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.s, o),
                       __shfl_xor_sync(0xffffffffu, st.t, o)});
  if (lane == 0) s_stat[warp] = st;
  if (TOP) s_key[warp][lane] = list;
  __syncthreads();
  if (warp == 0) {
    for (int w = 1; w < kWarps; ++w) {
      st = join(st, s_stat[w]);
      if (TOP) list = join_lists(list, s_key[w][31 - lane], lane);
    }
  }
  if (a.splits > 1) {
    // to the cluster's first CTA, once all have started
    __syncwarp();
    cluster_arrive_relaxed();
    cluster_wait();
    if (warp == 0) {
      const uint32_t stat = mapa_shared(smem_u32(&s_other[split]), 0);
      if (lane == 0) {
        st_cluster_f32(stat, st.m);
        st_cluster_f32(stat + 4, st.s);
        st_cluster_f32(stat + 8, st.t);
      }
      if (TOP) {
        const uint32_t key = mapa_shared(smem_u32(&s_other_key[split][lane]), 0);
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(key), "l"(list) : "memory");
      }
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (split == 0 && warp == 0) {
      for (int i = 1; i < a.splits; ++i) {
        st = join(st, s_other[i]);
        if (TOP) list = join_lists(list, s_other_key[i][31 - lane], lane);
      }
    }
  }
  if (split == 0 && warp == 0) finish_row<TYPE>(a, row, st, list, lane);
}

// CTAs per row: until every SM has one, each warp with a batch at least (128
// rows of 100003 FP32 values: 34 us with two CTAs a row, 36 with four).
cudaError_t splits_of(int n_rows, int vocab, int type, int* out) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int batch = 32 * kLoads * (type == DFLASH_T_FP32 ? 4 : 8);
  const int most = (vocab + batch * kWarps - 1) / (batch * kWarps);
  int s = 1;  // powers of two
  while (2 * s <= kMaxSplits && 2 * s <= most && static_cast<long long>(n_rows) * s < sms) s *= 2;
  *out = s;
  return cudaSuccess;
}

template <int TYPE, bool TOP>
cudaError_t launch_typed(const LogprobArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.n_rows) * a.splits);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.splits;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.splits > 1 ? 1 : 0;
  if (a.splits > 8) {  // beyond the portable size
    const cudaError_t e = cudaFuncSetAttribute(logprobs_kernel<TYPE, TOP>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<TYPE, TOP>, a);
}

template <int TYPE>
cudaError_t launch(const LogprobArgs& a, cudaStream_t st) {
  return a.k ? launch_typed<TYPE, true>(a, st) : launch_typed<TYPE, false>(a, st);
}

bool known_type(int type) { return type == DFLASH_T_FP32 || type == DFLASH_T_BF16 || type == DFLASH_T_FP16; }

}  // namespace
}  // namespace dflash

using namespace dflash;

extern "C" {

int dflash_token_logprobs(const void* logits, int32_t type, int64_t row_stride, int32_t n_rows, int32_t vocab,
                          const int32_t* tokens, float* logprob, float* entropy, int32_t top_k, int32_t* top_ids,
                          float* top_logprobs, int32_t* dev_status, dflash_stream_t stream) {
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
  a.status = dev_status;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  e = type == DFLASH_T_FP32 ? launch<DFLASH_T_FP32>(a, st)
      : type == DFLASH_T_BF16 ? launch<DFLASH_T_BF16>(a, st)
                              : launch<DFLASH_T_FP16>(a, st);
  return cuda_status(e, "token logprobs");
}

}  // extern "C"
