// Tokens drawn from rows of logits (dflash_sample_tokens in include/dflash.h).
//
//   w_i = e^((x_i - m) / T),  m = max x
//   kept: x_i >= the k-th largest;  A(x_i) < p S, where A(v) is the weight of the kept
//   tokens above v and S that of all;  w_i >= min_p;  x_i > -infinity
//   token: the first id whose kept weights up to it, in order of ids, exceed u times all of them.
//
// All of this is a matter of comparisons, so that a row's id has to be the one of the
// definition whatever the order of additions: weights are whole numbers of
// 2^-F (F = 45 for up to 2^17 tokens, one less for each doubling), right to about
// 2^-43 relative, and sums of them are exact.  e^y is computed in pairs of FP32
// numbers by a table of 2^(j/32) and a short series (Tang, "Table-driven
// implementation of the exponential function", 1989): FP64 instructions are
// sixty times as slow here.
//
// The CTAs of a cluster hold a row in their shared memory, so that it is read once
// from global memory however often it is looked at.  Few tokens decide most rows, and
// plain FP32 finds them:
//  - With a filter, a bound below the threshold.  Of top-k: the k-th largest of the threads' own maxima, by a
//    histogram of them.  Of top-p: the first of 512 ranges of logits below which less than
//    (1 - p) S can lie, counted with each range's largest weight.  Of min-p: itself.  The
//    tokens above the bound, if they are at most kList, go to the first CTA, which
//    sorts them and decides everything with exact weights.  S itself, which a top-p without top-k compares with, comes
//    from FP32 sums with a bound on their error; where that leaves it open which token is
//    the last (or which u names, without a filter), S is added up exactly.
//  - Without one, FP32 sums by CTA, warp and lane lead to the token; the exact ones are formed if a border
//    of it lies within the error's bound.
// Else (long lists) a threshold is found digit by digit: counts (and exact weights) of up to
// 1024 ranges of the keys, then of the ranges of the one in which the threshold lies, until it is one key.
//
// The bound of an FP32 sum, relative to S, in units of 2^-24: a weight's exponent y = (x - m) c is off by 3 |y| (difference, c,
// product), and the mean of |y| over the weights, their entropy less log2 S, is 19 at most for 2^19 tokens: 40 with ln 2;
// 2^y 4; additions, of 16 pieces in a thread, in it, over warps and CTAs: 16 + 3 + 5 + 16 + 16.  In all under 128: kError.
#include <cstddef>

#include "common.cuh"
#include "internal.h"
#include "kernels.h"
#include "logits.cuh"

namespace dflash {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kBins = 1024;
constexpr int kMaxSplits = 16;             // CTAs of a cluster
constexpr int kMaxRowBytes = 160 * 1024;   // of a row in one CTA
constexpr int kList = 2048;                // tokens that the first CTA sorts
constexpr int kQuickBins = kThreads;       // ranges of the first bounds
constexpr float kError = 0x1p-17f;         // of an FP32 sum of weights, relative
constexpr int kFixed = 45;                 // binary places of a weight
constexpr float kMaxTemperature = 0x1p64f;

struct SampleArgs {
  const uint8_t* logits;
  long long row_bytes;
  int n_rows, vocab, splits, pieces;  // pieces: 16-byte pieces of a row that a CTA holds
  int drop;                           // places less than kFixed
  const float* uniform;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int32_t* tokens;
  float* logprob;
  int32_t* kept;
  int32_t* status;
};

// ------------------------------------------------------------- exact weights
struct TableEntry {
  uint64_t fixed;  // 2^(j/32) in units of 2^-45
  float hi, lo;    // the same, as the sum of two
};
__constant__ TableEntry kTable[32] = {
    {35184372088832ull, 0x1.000000p+0f, 0x0.0p+0f},
    {35954809514763ull, 0x1.059b0ep+0f, -0x1.9d4f52p-25f},
    {36742117323538ull, 0x1.0b5586p+0f, 0x1.9f3122p-25f},
    {37546664928439ull, 0x1.11301ep+0f, -0x1.fdb496p-25f},
    {38368829831843ull, 0x1.172b84p+0f, -0x1.c15742p-27f},
    {39208997802355ull, 0x1.1d4874p+0f, -0x1.d2e8cap-25f},
    {40067563055812ull, 0x1.2387a6p+0f, 0x1.ceac48p-25f},
    {40944928440254ull, 0x1.29e9e0p+0f, -0x1.5c0424p-25f},
    {41841505624942ull, 0x1.306fe0p+0f, 0x1.4636e2p-25f},
    {42757715293524ull, 0x1.371a74p+0f, -0x1.18aac6p-25f},
    {43693987341416ull, 0x1.3dea64p+0f, 0x1.824684p-25f},
    {44650761077522ull, 0x1.44e086p+0f, 0x1.8624b4p-30f},
    {45628485430356ull, 0x1.4bfdaep+0f, -0x1.593abcp-25f},
    {46627619158687ull, 0x1.5342b6p+0f, -0x1.2c5610p-25f},
    {47648631066792ull, 0x1.5ab07ep+0f, -0x1.5bd5ecp-27f},
    {48692000224427ull, 0x1.6247ecp+0f, -0x1.f8b550p-25f},
    {49758216191608ull, 0x1.6a09e6p+0f, 0x1.9fcef4p-26f},
    {50847779248319ull, 0x1.71f75ep+0f, 0x1.1d8beep-25f},
    {51961200629251ull, 0x1.7a1148p+0f, -0x1.829fd0p-25f},
    {53099002763676ull, 0x1.82589ap+0f, -0x1.accc7cp-26f},
    {54261719520578ull, 0x1.8ace54p+0f, 0x1.15506ep-27f},
    {55449896459148ull, 0x1.93737cp+0f, -0x1.e6474p-25f},
    {56664091084769ull, 0x1.9c4918p+0f, 0x1.51f848p-27f},
    {57904873110603ull, 0x1.a5503cp+0f, -0x1.b83b54p-25f},
    {59172824724903ull, 0x1.ae89fap+0f, -0x1.a94b14p-26f},
    {60468540864189ull, 0x1.b7f770p+0f, -0x1.a09438p-25f},
    {61792629492389ull, 0x1.c199bep+0f, -0x1.3d56b2p-27f},
    {63145711886113ull, 0x1.cb720ep+0f, -0x1.8837ccp-27f},
    {64528422926153ull, 0x1.d5818ep+0f, -0x1.822dbcp-27f},
    {65941411395383ull, 0x1.dfc974p+0f, -0x1.908c94p-25f},
    {67385340283170ull, 0x1.ea4afap+0f, 0x1.52486cp-27f},
    {68860887096459ull, 0x1.f50766p+0f, -0x1.246eb0p-26f},
};

// What a weight depends on besides its logit: m, and log2(e) / T as the sum of two.
struct Scale {
  float m, hi, lo;
  int drop;
};

// e^((x - m) / T) in units of 2^-(kFixed - drop).  (Products and sums are written out: the
// compiler must not contract them.)
__device__ __forceinline__ uint64_t weight(float x, const Scale& c, const TableEntry* table) {
  // x - m = s + e exactly
  const float b = -c.m;
  const float s = __fadd_rn(x, b), v = __fsub_rn(s, x);
  const float e = __fadd_rn(__fsub_rn(x, __fsub_rn(s, v)), __fsub_rn(b, v));
  // times log2(e) / T: p + q
  const float p = __fmul_rn(s, c.hi);
  if (!(p > -48.f)) return 0;  // (masked values too)
  const float q = __fmaf_rn(e, c.hi, __fmaf_rn(s, c.lo, __fmaf_rn(s, c.hi, -p)));
  // = n + j / 32 + r, |r| <= 1/64
  constexpr float ROUND = 393216.f;  // 1.5 2^18: adding it leaves multiples of 1/32
  const float t = __fadd_rn(p, ROUND);
  const int k = __float_as_int(t) - __float_as_int(ROUND);
  const float r = __fsub_rn(p, __fsub_rn(t, ROUND));
  const float rh = __fadd_rn(r, q), rl = __fsub_rn(q, __fsub_rn(rh, r));
  // a = r ln 2, u = e^a - 1
  constexpr float LN2 = 0x1.62e430p-1f, LN2_LO = -0x1.05c610p-29f;
  const float ah = __fmul_rn(rh, LN2);
  const float al = __fadd_rn(__fmaf_rn(rh, LN2, -ah), __fmaf_rn(rh, LN2_LO, __fmul_rn(rl, LN2)));
  const float h = __fmul_rn(0.5f, ah), s2 = __fmul_rn(h, ah);
  const float s2l = __fmaf_rn(ah, al, __fmaf_rn(h, ah, -s2));
  const float cubic = __fmul_rn(__fmul_rn(s2, ah), __fmaf_rn(ah, __fmaf_rn(ah, 1.f / 60, 1.f / 12), 1.f / 3));  // a^3/6 + a^4/24 + a^5/120
  const float uh = __fadd_rn(ah, s2);
  const float ul = __fadd_rn(__fsub_rn(s2, __fsub_rn(uh, ah)), __fadd_rn(al, __fadd_rn(s2l, cubic)));
  // times 2^(j / 32): its own whole number, and the rest in two steps of 2^-23 and 2^-45
  const TableEntry f = table[k & 31];
  const float vh = __fmul_rn(f.hi, uh);
  const float vl = __fadd_rn(__fmaf_rn(f.hi, uh, -vh), __fmaf_rn(f.hi, ul, __fmul_rn(f.lo, uh)));
  constexpr float STEP1 = 1.5f, STEP2 = 1.5f * 0x1p-22f;
  const float t1 = __fadd_rn(__fadd_rn(vh, vl), STEP1);
  const float rest = __fadd_rn(__fsub_rn(vh, __fsub_rn(t1, STEP1)), vl);
  const float t2 = __fadd_rn(rest, STEP2);
  const long long add = (static_cast<long long>(__float_as_int(t1) - __float_as_int(STEP1)) << 22) +
                        (__float_as_int(t2) - __float_as_int(STEP2));
  return (f.fixed + add) >> (c.drop - (k >> 5));
}

// ------------------------------------------------------------------ keys
// Whole numbers in the order of the values, -0 with +0.
template <int TYPE>
struct Keys {
  static constexpr bool WIDE = TYPE == DFLASH_T_FP32;
  static constexpr uint32_t SIGN = WIDE ? 0x80000000u : 0x8000u, ALL = WIDE ? 0xffffffffu : 0xffffu;
  static constexpr uint32_t INF = WIDE ? 0x7f800000u : TYPE == DFLASH_T_BF16 ? 0x7f80u : 0x7c00u;
  // the lowest key of a value that is not masked
  static constexpr uint32_t LOWEST = (~(SIGN | INF) & ALL) + 1;
  static __device__ __forceinline__ uint32_t of(uint32_t bits) {
    if (bits == SIGN) bits = 0;
    return bits & SIGN ? ~bits & ALL : bits | SIGN;
  }
  static __device__ __forceinline__ uint32_t bits(const uint4& v, int e) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (WIDE) return w[e];
    return e & 1 ? w[e >> 1] >> 16 : w[e >> 1] & 0xffffu;
  }
  static __device__ __forceinline__ float value(uint32_t b) {
    if constexpr (WIDE) return __uint_as_float(b);
    if constexpr (TYPE == DFLASH_T_BF16) return __uint_as_float(b << 16);
    return __half2float(__ushort_as_half(static_cast<uint16_t>(b)));
  }
  static __device__ __forceinline__ uint32_t of_value(float x) {
    if constexpr (WIDE) return of(__float_as_uint(x));
    if constexpr (TYPE == DFLASH_T_BF16) return of(__float_as_uint(x) >> 16);
    return of(__half_as_ushort(__float2half_rn(x)));
  }
  static __device__ __forceinline__ float value_of(uint32_t key) { return value(key & SIGN ? key & ~SIGN : ~key & ALL); }
  // the larger of two words' values, value by value, NaN if either is one
  static __device__ __forceinline__ uint32_t max_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (WIDE) {
      float f;
      asm("max.NaN.f32 %0, %1, %2;" : "=f"(f) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
      r = __float_as_uint(f);
    } else if constexpr (TYPE == DFLASH_T_BF16) {
      asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    } else {
      asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    }
    return r;
  }
  static __device__ __forceinline__ bool has_nan(uint32_t w) {
    if constexpr (WIDE) return (w & 0x7fffffffu) > INF;
    return (w & 0x7fffu) > INF || (w >> 16 & 0x7fffu) > INF;
  }
  static __device__ __forceinline__ float top_of(const uint4& v) {
    using E = Elem<TYPE>;
    return E::max_of(E::max_words(E::max_words(v.x, v.y), E::max_words(v.z, v.w)));
  }
  // FP32 weights of a piece
  static __device__ __forceinline__ float quick_sum(const uint4& v, float m, float c) {
    constexpr int VEC = Elem<TYPE>::VEC;
    float x[VEC];
    Elem<TYPE>::widen(v, x);
    const uint64_t minus = pack2(-m, -m), c2 = pack2(c, c);
    uint64_t s[VEC / 2];
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      float y0, y1;
      unpack2(mul2(add2(pack2(x[e], x[e + 1]), minus), c2), y0, y1);
      s[e / 2] = pack2(ex2_approx(y0), ex2_approx(y1));
    }
#pragma unroll
    for (int o = VEC / 4; o; o >>= 1)
#pragma unroll
      for (int e = 0; e < o; ++e) s[e] = add2(s[e], s[e + o]);
    float s0, s1;
    unpack2(s[0], s0, s1);
    return s0 + s1;
  }
  // values of a piece above -infinity
  static __device__ __forceinline__ int unmasked(const uint4& v) {
    constexpr int VEC = Elem<TYPE>::VEC;
    int c = 0;
#pragma unroll
    for (int e = 0; e < VEC; ++e) c += bits(v, e) != (SIGN | INF);
    return c;
  }
  // the key of the smallest value that is not below x
  static __device__ __forceinline__ uint32_t at_least(double x) {
    const float f = __double2float_ru(x);
    if constexpr (WIDE) return of(__float_as_uint(f));
    if constexpr (TYPE == DFLASH_T_BF16) return of(__bfloat16_as_ushort(__float2bfloat16_ru(f)));
    return of(__half_as_ushort(__float2half_ru(f)));
  }
};

// ------------------------------------------------------------------ clusters
__device__ __forceinline__ void cluster_sync(int splits) {
  if (splits > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
}
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t ld_cluster64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ uint64_t shfl_up(uint64_t v, int o) { return __shfl_up_sync(0xffffffffu, v, o); }
template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct Found {
  uint32_t lo, hi;      // keys of the range
  uint32_t above;       // tokens above it
  uint32_t all;         // fewer tokens than are asked for: all are kept
  uint64_t above_w;     // their weight, if weights are asked for
  uint64_t with_w;      // the same with the range's own
};

struct Shared {
  union {
    struct {
      uint32_t count[kBins], lo[kBins], hi[kBins];  // of this CTA's tokens; weights in two words
      uint32_t all_count[kBins];                    // of the cluster's, in its first CTA
      uint64_t all_w[kBins];
    } digits;
    struct {
      uint64_t list[kList];    // (key, id) in order of ids
      uint64_t sorted[kList];  // (key, place in `list`), largest first
      uint64_t upto[kList];    // weights before each of them
      uint32_t hist[kQuickBins];
    } quick;
  };
  TableEntry table[32];
  Found found;
  uint64_t cta_w[kMaxSplits], warp_w[kWarps];
  uint32_t cta_top[kMaxSplits], cta_low[kMaxSplits], cta_n[kMaxSplits], warp_u[kWarps], warp_low[kWarps], warp_n[kWarps];
  float cta_f[kMaxSplits], warp_f[kWarps];
  double log_min_p;
  Scale scale;
  float bound;
  uint32_t verdict;
};
constexpr int kSharedBytes = (sizeof(Shared) + 15) / 16 * 16;
// What the first CTA (or the one that u names) says of a quick answer.
enum Verdict : uint32_t { kDone, kExactSum, kDigits };

template <int TYPE>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
  using E = Elem<TYPE>;
  using K = Keys<TYPE>;
  constexpr int VEC = E::VEC;
  extern __shared__ uint4 smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  uint4* data = smem + kSharedBytes / 16;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = blockIdx.x / a.splits, rank = blockIdx.x - row * a.splits;
  const int n = a.splits;
  if (n > 1) cluster_arrive_relaxed();  // (every CTA has started before another writes to it)

  // ---- what the row asks for
  const float t_asked = a.temperature ? a.temperature[row] : 1.f;
  const bool t_fine = t_asked >= 0.f && t_asked <= kMaxTemperature;
  const float temperature = t_asked > kMaxTemperature ? kMaxTemperature : t_asked;
  const bool greedy = !(temperature > 0.f);
  const int k_asked = a.top_k ? a.top_k[row] : 0;
  const bool by_k = k_asked > 0 && k_asked < a.vocab;
  const float p = a.top_p ? a.top_p[row] : 1.f;
  const bool by_p = p < 1.f;
  const float min_p = a.min_p ? a.min_p[row] : 0.f;
  const bool by_min = min_p > 0.f;
  const float u_asked = a.uniform[row];
  const bool u_fine = u_asked >= 0.f && u_asked < 1.f;
  const float u = u_fine ? u_asked : u_asked >= 1.f ? 0x1.fffffep-1f : 0.f;
  if (tid < 32) sh.table[tid] = kTable[tid];
  if (tid == kThreads - 1) {
    if (rank == 0 && (!t_fine || !u_fine || p != p || !(min_p <= 1.f))) set_status(a.status, DFLASH_DEV_BAD_VALUE);
    if (!greedy) {
      const double c = fmin(1.4426950408889634 / static_cast<double>(temperature), 1e38);
      sh.scale.hi = static_cast<float>(c);
      sh.scale.lo = static_cast<float>(c - static_cast<double>(sh.scale.hi));
      sh.scale.drop = a.drop;
      if (by_min) sh.log_min_p = static_cast<double>(temperature) * log(static_cast<double>(fminf(min_p, 1.f)));
    }
  }

  // ---- the row into shared memory: value i lies at place i + skip of whole pieces
  const uint8_t* src = a.logits + row * a.row_bytes;
  const int skip = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15) / E::BYTES;
  const uint4* frame = reinterpret_cast<const uint4*>(src - skip * E::BYTES);
  const int all_pieces = (a.vocab + skip + VEC - 1) / VEC;
  const int first = rank * a.pieces;  // the CTA's pieces
  const int mine = max(min(a.pieces, all_pieces - first), 0);
  float top = -INFINITY;  // of the thread's values
  {
    constexpr int U = 4;
    uint32_t tops = E::NOTHING;
    for (int i0 = tid; i0 < mine; i0 += U * kThreads) {
      uint4 v[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int i = i0 + j * kThreads;
        const int p0 = (first + i) * VEC - skip;  // value of the piece's first place
        v[j] = make_uint4(E::NOTHING, E::NOTHING, E::NOTHING, E::NOTHING);
        if (i < mine && p0 >= 0 && p0 + VEC <= a.vocab) v[j] = __ldcs(frame + first + i);
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int i = i0 + j * kThreads;
        if (i >= mine) break;
        const int p0 = (first + i) * VEC - skip;
        if (p0 < 0 || p0 + VEC > a.vocab) {  // the row's ends: value by value
          constexpr int W = VEC / 4;
          v[j].x = E::raw(src, p0, a.vocab);
          v[j].y = E::raw(src, p0 + W, a.vocab);
          v[j].z = E::raw(src, p0 + 2 * W, a.vocab);
          v[j].w = E::raw(src, p0 + 3 * W, a.vocab);
        }
        data[i] = v[j];
        tops = K::max_nan(tops, K::max_nan(K::max_nan(v[j].x, v[j].y), K::max_nan(v[j].z, v[j].w)));
      }
    }
    const bool nan = K::has_nan(tops);
    top = E::max_of(tops);
    uint32_t key = nan ? 0xffffffffu : float_order_key(top);  // (no value's key is that large)
    uint32_t low = top > -INFINITY ? key : 0xffffffffu;
    const uint32_t some = __popc(__ballot_sync(0xffffffffu, top > -INFINITY));
    key = __reduce_max_sync(0xffffffffu, key);
    low = __reduce_min_sync(0xffffffffu, low);
    if (lane == 0) sh.warp_u[warp] = key, sh.warp_low[warp] = low, sh.warp_n[warp] = some;
    if (tid == 0) sh.verdict = kExactSum;
    sh.quick.hist[tid] = 0;
    __syncthreads();
    if (n > 1) cluster_wait();
    if (tid < 32) {
      const bool w = lane < kWarps;
      key = __reduce_max_sync(0xffffffffu, w ? sh.warp_u[lane] : 0u);
      low = __reduce_min_sync(0xffffffffu, w ? sh.warp_low[lane] : 0xffffffffu);
      const uint32_t all = __reduce_add_sync(0xffffffffu, w ? sh.warp_n[lane] : 0u);
      if (n == 1) {
        if (lane == 0) sh.cta_top[0] = key, sh.cta_low[0] = low, sh.cta_n[0] = all;
      } else if (lane < n) {
        st_cluster(mapa_shared(smem_u32(&sh.cta_top[rank]), lane), key);
        st_cluster(mapa_shared(smem_u32(&sh.cta_low[rank]), lane), low);
        st_cluster(mapa_shared(smem_u32(&sh.cta_n[rank]), lane), all);
      }
    }
  }
  cluster_sync(n);
  uint32_t top_key = 0, low_key = 0xffffffffu, maxima = 0;
  for (int i = 0; i < n; ++i) {
    top_key = max(top_key, sh.cta_top[i]);
    low_key = min(low_key, sh.cta_low[i]);
    maxima += sh.cta_n[i];
  }
  const float m = float_from_order_key(top_key);
  if (top_key == 0xffffffffu || !(m < INFINITY) || m == -INFINITY) {  // not finite, or nothing to draw from
    if (rank == 0 && tid == 0) {
      if (m != -INFINITY) set_status(a.status, DFLASH_DEV_NONFINITE);
      a.tokens[row] = -1;
      if (a.logprob) a.logprob[row] = -INFINITY;
      if (a.kept) a.kept[row] = 0;
    }
    return;
  }

  // this warp's pieces, one after the other
  const int per_warp = (mine + kWarps - 1) / kWarps;
  const int w0 = min(warp * per_warp, mine), w1 = min(w0 + per_warp, mine);

  if (greedy) {  // the first id of the largest value
    uint32_t id = 0xffffffffu;
    for (int i = w0 + lane; i < w1; i += 32) {
      const uint4 v = data[i];
      if (K::top_of(v) < m) continue;
#pragma unroll
      for (int e = VEC - 1; e >= 0; --e)
        if (K::value(K::bits(v, e)) == m) id = min(id, static_cast<uint32_t>((first + i) * VEC + e - skip));
    }
    id = __reduce_min_sync(0xffffffffu, id);
    if (lane == 0) sh.warp_u[warp] = id;
    __syncthreads();
    if (tid < 32) {
      id = __reduce_min_sync(0xffffffffu, lane < kWarps ? sh.warp_u[lane] : 0xffffffffu);
      // (not the array that the maxima lie in: a CTA may still read them)
      if (lane == 0) {
        if (n == 1) sh.cta_w[0] = id;
        else st_cluster(mapa_shared(smem_u32(&sh.cta_w[rank]), 0), static_cast<uint64_t>(id));
      }
    }
    cluster_sync(n);
    if (rank == 0 && tid == 0) {
      uint64_t best = sh.cta_w[0];
      for (int i = 1; i < n; ++i) best = min(best, sh.cta_w[i]);
      a.tokens[row] = static_cast<int32_t>(best);
      if (a.logprob) a.logprob[row] = 0.f;
      if (a.kept) a.kept[row] = 1;
    }
    return;
  }

  if (tid == 0) sh.scale.m = m;
  __syncthreads();
  const Scale scale = sh.scale;
  const uint32_t most = K::of_value(m);
  uint32_t least = K::LOWEST;
  if (by_min) least = max(least, min(most, K::at_least(static_cast<double>(m) + sh.log_min_p)));

  // ln(w / total) of a token, where w <= 1 and the largest weight, 1, is among those of the total
  auto log_of = [&](float x, float others) { return (x - m) / temperature - log1pf(others); };
  auto others_of = [&](uint64_t total) {
    return static_cast<float>(total - (1ull << (kFixed - a.drop))) * exp2f(static_cast<float>(a.drop - kFixed));
  };

  // The sum over the cluster of a value per thread, and the CTAs' sums in sh.cta_w.
  auto cluster_total = [&](uint64_t v) {
    v = warp_sum(v);
    cluster_sync(n);  // the last values in these arrays have been read
    if (lane == 0) sh.warp_w[warp] = v;
    __syncthreads();
    if (tid < 32) {
      v = warp_sum(lane < kWarps ? sh.warp_w[lane] : uint64_t(0));
      if (n == 1) {
        if (lane == 0) sh.cta_w[0] = v;
      } else if (lane < n) {
        st_cluster(mapa_shared(smem_u32(&sh.cta_w[rank]), lane), v);
      }
    }
    cluster_sync(n);
    uint64_t sum = 0;
    for (int i = 0; i < n; ++i) sum += sh.cta_w[i];
    return sum;
  };
  // The exact weight of all tokens.
  auto exact_sum = [&]() {
    uint64_t sum = 0;
    for (int i = w0 + lane; i < w1; i += 32) {
      const uint4 v = data[i];
#pragma unroll
      for (int e = 0; e < VEC; ++e) sum += weight(K::value(K::bits(v, e)), scale, sh.table);
    }
    return cluster_total(sum);
  };
  // The sum of a value per thread over this CTA's threads before it, and over all of them.
  auto scan = [&](uint64_t v, uint64_t& all) {
    uint64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = shfl_up(x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();  // the last scan's values have been read
    if (lane == 31) sh.warp_w[warp] = x;
    __syncthreads();
    x -= v;
    all = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const uint64_t y = sh.warp_w[i];
      if (i < warp) x += y;
      all += y;
    }
    return x;
  };
  auto tell_verdict = [&](uint32_t v) {  // (one thread)
    for (int r = 0; r < n; ++r) {
      if (n == 1) sh.verdict = v;
      else st_cluster(mapa_shared(smem_u32(&sh.verdict), r), v);
    }
  };

  const bool filter = by_k || by_p || by_min;
  if (!filter) {
    // ---- FP32 sums of the weights lead to the token
    float sum = 0.f;
    uint32_t count = 0;
    for (int i = w0 + lane; i < w1; i += 32) {
      const uint4 v = data[i];
      sum += K::quick_sum(v, m, scale.hi);
      count += K::unmasked(v);
    }
    float ws = sum;
#pragma unroll
    for (int o = 16; o; o >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, o);
    count = __reduce_add_sync(0xffffffffu, count);
    if (lane == 0) sh.warp_f[warp] = ws, sh.warp_n[warp] = count;
    __syncthreads();
    if (tid < 32) {
      float cs = 0.f;
      for (int i = 0; i < kWarps; ++i) cs += sh.warp_f[i];
      const uint32_t c = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.warp_n[lane] : 0u);
      if (n == 1) {
        if (lane == 0) sh.cta_f[0] = cs, sh.cta_w[0] = c;
      } else if (lane < n) {
        st_cluster(mapa_shared(smem_u32(&sh.cta_f[rank]), lane), __float_as_uint(cs));
        st_cluster(mapa_shared(smem_u32(&sh.cta_w[rank]), lane), static_cast<uint64_t>(c));
      }
    }
    cluster_sync(n);
    float total = 0.f, below = 0.f, own = 0.f;
    for (int i = 0; i < n; ++i) {
      if (i == rank) below = total, own = sh.cta_f[i];
      total += sh.cta_f[i];
    }
    const float at = u * total, off = kError * total;
    if (at >= below && (at < below + own || rank == n - 1)) {  // (one CTA, by these sums)
      float from = below;
      int w = 0;
      for (; w < kWarps - 1 && !(at < from + sh.warp_f[w]); ++w) from += sh.warp_f[w];
      if (warp == w) {
        for (int i0 = w0; i0 < w1; i0 += 32) {
          const int i = i0 + lane;
          const uint4 v = i < w1 ? data[i] : make_uint4(E::NOTHING, E::NOTHING, E::NOTHING, E::NOTHING);
          const float part = K::quick_sum(v, m, scale.hi);
          float upto = part;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const float y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
          }
          upto += from;
          const unsigned over = __ballot_sync(0xffffffffu, upto > at);
          if (over) {
            if (lane == __ffs(over) - 1) {
              float c = upto - part;
#pragma unroll
              for (int e = 0; e < VEC; ++e) {
                const float x = K::value(K::bits(v, e)), before = c;
                c += ex2_approx((x - m) * scale.hi);
                // the first past u, further from both of its borders than the sums may be off
                if (before <= at && c > at) {
                  if (before + off <= at && c - off > at) {
                    a.tokens[row] = (first + i) * VEC + e - skip;
                    if (a.logprob) a.logprob[row] = log_of(x, total - 1.f);
                    if (a.kept) {
                      uint64_t all = 0;
                      for (int r = 0; r < n; ++r) all += sh.cta_w[r];
                      a.kept[row] = static_cast<int32_t>(all);
                    }
                    tell_verdict(kDone);
                  }
                  break;
                }
              }
            }
            break;
          }
          from = __shfl_sync(0xffffffffu, upto, 31);
        }
      }
    }
    __syncwarp();
    cluster_sync(n);
    if (sh.verdict == kDone) return;
  } else {
    // ---- a bound below the thresholds
    float bound = -INFINITY;  // logits from here on
    bool quick = true;
    float sum = 0.f;  // of all weights, by top-p alone
    if (a.vocab <= kList) {  // the whole row is a list
    } else if (by_k) {
      const float low = float_from_order_key(low_key), per = m > low ? (kQuickBins - 1) / (m - low) : 0.f;
      quick = maxima >= static_cast<uint32_t>(k_asked) && per < 1e30f && per > 0.f;
      if (quick) {
        if (top > -INFINITY) atomicAdd(&sh.quick.hist[min(static_cast<int>((m - top) * per), kQuickBins - 1)], 1u);
        cluster_sync(n);
        uint32_t c = 0;
        if (n == 1) c = sh.quick.hist[tid];
        else
          for (int r = 0; r < n; ++r) c += ld_cluster(mapa_shared(smem_u32(&sh.quick.hist[tid]), r));
        uint64_t all;
        const uint64_t before = scan(c, all);
        // (the values of range b lie above m - (b + 1) / per, to FP32)
        if (before < k_asked && before + c >= k_asked) sh.bound = m - (tid + 1) / per * (1.f + 0x1p-20f);
        __syncthreads();
        bound = sh.bound;
      }
    } else if (by_p) {
      // tokens whose exponent is beyond `cut` weigh (1 - p) / 4 together at most
      const float rest = 1.f - fmaxf(p, 0.f), cut = log2f(static_cast<float>(a.vocab) * 4.f / rest);
      const float per = kQuickBins / cut;
      quick = cut < 40.f;
      if (quick) {
        for (int i = w0 + lane; i < w1; i += 32) {
          const uint4 v = data[i];
          sum += K::quick_sum(v, m, scale.hi);
          if ((m - K::top_of(v)) * scale.hi < cut) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              const float z = (m - K::value(K::bits(v, e))) * scale.hi;
              if (z < cut) atomicAdd(&sh.quick.hist[min(static_cast<int>(z * per), kQuickBins - 1)], 1u);
            }
          }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) sh.warp_f[warp] = sum;
        __syncthreads();
        if (tid < 32) {
          float cs = 0.f;
          for (int i = 0; i < kWarps; ++i) cs += sh.warp_f[i];
          if (n == 1) {
            if (lane == 0) sh.cta_f[0] = cs;
          } else if (lane < n) {
            st_cluster(mapa_shared(smem_u32(&sh.cta_f[rank]), lane), __float_as_uint(cs));
          }
        }
        cluster_sync(n);
        sum = 0.f;
        for (int i = 0; i < n; ++i) sum += sh.cta_f[i];
        // what the ranges from the last one up to this thread's weigh at most
        const int bin = kQuickBins - 1 - tid;
        uint32_t c = 0;
        if (n == 1) c = sh.quick.hist[bin];
        else
          for (int r = 0; r < n; ++r) c += ld_cluster(mapa_shared(smem_u32(&sh.quick.hist[bin]), r));
        const float w = static_cast<float>(c) * ex2_approx(-static_cast<float>(bin) / per);
        float x = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        __syncthreads();  // warp_f has been read
        if (lane == 31) sh.warp_f[warp] = x;
        if (tid == 0) sh.bound = -INFINITY;
        __syncthreads();
        x += rest * 0.25f;
        for (int i = 0; i < warp; ++i) x += sh.warp_f[i];
        // (2^-10: more than the sums and ranges are off)
        const float most_left = rest * sum * (1.f - 0x1p-10f);
        // the first range that has to be kept: with it more than may be left out would be
        if (x > most_left && x - w <= most_left) sh.bound = m - (bin + 1) / per / scale.hi * (1.f + 0x1p-20f);
        __syncthreads();
        bound = sh.bound;
        quick = bound > -INFINITY;
      }
    }
    // (top-p needs the whole of what top-k leaves, and in a short row of all)
    if (by_min && !(by_p && (by_k || a.vocab <= kList))) bound = fmaxf(bound, K::value_of(least));

    if (quick) {
      // ---- the tokens from the bound on, in order of their ids, in each CTA
      uint32_t count = 0;
      for (int i = w0 + lane; i < w1; i += 32) {
        const uint4 v = data[i];
        if (K::top_of(v) < bound) continue;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float x = K::value(K::bits(v, e));
          count += x >= bound && x > -INFINITY;
        }
      }
      uint64_t all;
      uint32_t to;
      {
        const uint32_t w = __reduce_add_sync(0xffffffffu, count);
        __syncthreads();
        if (lane == 0) sh.warp_n[warp] = w;
        __syncthreads();
        to = 0;
        uint32_t c = 0;
        for (int i = 0; i < kWarps; ++i) {
          if (i < warp) to += sh.warp_n[i];
          c += sh.warp_n[i];
        }
        all = c;
      }
      if (all <= kList && sh.warp_n[warp]) {
        for (int i0 = w0; i0 < w1; i0 += 32) {
          const int i = i0 + lane;
          const uint4 v = i < w1 ? data[i] : make_uint4(E::NOTHING, E::NOTHING, E::NOTHING, E::NOTHING);
          const bool any = K::top_of(v) >= bound && K::top_of(v) > -INFINITY;
          if (!__any_sync(0xffffffffu, any)) continue;
          uint32_t c = 0;
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float x = K::value(K::bits(v, e));
            c += x >= bound && x > -INFINITY;
          }
          uint32_t upto = c;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
          }
          uint32_t at = to + upto - c;
          if (c) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              const uint32_t b = K::bits(v, e);
              const float x = K::value(b);
              if (x >= bound && x > -INFINITY)
                sh.quick.list[at++] = static_cast<uint64_t>(K::of(b)) << 32 | static_cast<uint32_t>((first + i) * VEC + e - skip);
            }
          }
          to += __shfl_sync(0xffffffffu, upto, 31);
        }
      }
      if (tid == 0) {
        // (not the array that the numbers of maxima lie in: a CTA may still read them)
        if (n == 1) sh.cta_w[0] = all;
        else st_cluster(mapa_shared(smem_u32(&sh.cta_w[rank]), 0), all);
      }
      cluster_sync(n);
      uint32_t keep = 0, size = 0;
      uint64_t kept_w = 0;
      uint32_t cut_key = 0;
      // what the first CTA makes of its list, once it is sorted: false if S has to be exact
      auto decide = [&](double s_lo, double s_hi) {
        auto key_at = [&](uint32_t i) { return static_cast<uint32_t>(sh.quick.sorted[i] >> 32); };
        // how many of the first `of` have the property, which holds down to some place
        auto number = [&](uint32_t of, auto&& has) {
          uint32_t c = 0;
          for (uint32_t i = tid; i < of; i += kThreads) c += has(i);
          c = __reduce_add_sync(0xffffffffu, c);
          __syncthreads();
          if (lane == 0) sh.warp_n[warp] = c;
          __syncthreads();
          c = 0;
          for (int i = 0; i < kWarps; ++i) c += sh.warp_n[i];
          return c;
        };
        uint32_t of = size;
        cut_key = least;
        if (by_k) {
          const uint32_t k_key = key_at(min(static_cast<uint32_t>(k_asked), size) - 1);
          cut_key = max(cut_key, k_key);
          of = number(size, [&](uint32_t i) { return key_at(i) >= k_key; });
        }
        if (by_p) {
          const double whole = by_k ? static_cast<double>(of < size ? sh.quick.upto[of] : kept_w) : 0.0;
          const double lo = static_cast<double>(p) * (by_k ? whole : s_lo), hi = static_cast<double>(p) * (by_k ? whole : s_hi);
          const uint32_t c = number(of, [&](uint32_t i) { return static_cast<double>(sh.quick.upto[i]) < lo; });
          if (lo != hi) {
            const uint32_t d = number(of, [&](uint32_t i) { return static_cast<double>(sh.quick.upto[i]) < hi; });
            if (c != d) return false;
          }
          cut_key = max(cut_key, key_at(c ? c - 1 : 0));
        }
        keep = number(size, [&](uint32_t i) { return key_at(i) >= cut_key; });
        return true;
      };
      // and the token, in order of ids
      auto draw = [&]() {
        const uint64_t total = keep < size ? sh.quick.upto[keep] : kept_w;
        const uint64_t at = static_cast<uint64_t>(static_cast<double>(u) * static_cast<double>(total));
        const uint32_t per = (size + kThreads - 1) / kThreads;
        const uint32_t j0 = min(tid * per, size), j1 = min(j0 + per, size);
        uint64_t w = 0, all_w;
        for (uint32_t j = j0; j < j1; ++j) {
          const uint32_t key = static_cast<uint32_t>(sh.quick.list[j] >> 32);
          if (key >= cut_key) w += weight(K::value_of(key), scale, sh.table);
        }
        uint64_t c = scan(w, all_w);
        if (c <= at && at < c + w) {  // (one thread)
          for (uint32_t j = j0; j < j1; ++j) {
            const uint64_t entry = sh.quick.list[j];
            const uint32_t key = static_cast<uint32_t>(entry >> 32);
            if (key < cut_key) continue;
            const float x = K::value_of(key);
            c += weight(x, scale, sh.table);
            if (c > at) {
              a.tokens[row] = static_cast<int32_t>(entry);
              if (a.logprob) a.logprob[row] = log_of(x, others_of(total));
              if (a.kept) a.kept[row] = static_cast<int32_t>(keep);
              break;
            }
          }
        }
      };
      if (rank == 0) {
        // the CTAs' lists one behind the other
        uint64_t upto = 0;
        for (int r = 0; r < n; ++r) upto += sh.cta_w[r];
        uint32_t verdict = kDigits;
        if (upto <= kList) {
          size = static_cast<uint32_t>(upto);
          for (uint32_t i = tid; i < size; i += kThreads) {
            uint32_t r = 0, j = i;
            while (j >= sh.cta_w[r]) j -= static_cast<uint32_t>(sh.cta_w[r++]);
            uint64_t entry;
            if (r == 0) {
              entry = sh.quick.list[i];
            } else {
              entry = ld_cluster64(mapa_shared(smem_u32(&sh.quick.list[j]), r));
              sh.quick.list[i] = entry;
            }
            sh.quick.sorted[i] = (entry & 0xffffffff00000000ull) | i;
          }
          uint32_t full = 2;
          while (full < size) full *= 2;
          for (uint32_t i = size + tid; i < full; i += kThreads) sh.quick.sorted[i] = 0;
          __syncthreads();
          for (uint32_t span = 2; span <= full; span *= 2)
            for (uint32_t step = span / 2; step; step /= 2) {
              for (uint32_t i = tid; i < full / 2; i += kThreads) {
                const uint32_t x = 2 * i - (i & (step - 1)), y = x + step;
                const uint64_t f = sh.quick.sorted[x], g = sh.quick.sorted[y];
                if ((f < g) == ((x & span) == 0)) sh.quick.sorted[x] = g, sh.quick.sorted[y] = f;
              }
              __syncthreads();
            }
          // exact weights before each
          const uint32_t per = (size + kThreads - 1) / kThreads;
          const uint32_t j0 = min(tid * per, size), j1 = min(j0 + per, size);
          uint64_t w = 0;
          for (uint32_t j = j0; j < j1; ++j) {
            const uint64_t x = weight(K::value_of(static_cast<uint32_t>(sh.quick.sorted[j] >> 32)), scale, sh.table);
            sh.quick.upto[j] = x;
            w += x;
          }
          uint64_t c = scan(w, kept_w);
          for (uint32_t j = j0; j < j1; ++j) {
            const uint64_t x = sh.quick.upto[j];
            sh.quick.upto[j] = c;
            c += x;
          }
          __syncthreads();
          double s_lo = 0.0, s_hi = 0.0;
          if (by_p && !by_k) {
            const double s = a.vocab <= kList ? static_cast<double>(kept_w)
                                              : static_cast<double>(sum) * static_cast<double>(1ull << (kFixed - a.drop));
            const double off = a.vocab <= kList ? 0.0 : static_cast<double>(kError);
            s_lo = s - s * off, s_hi = s + s * off;
          }
          verdict = decide(s_lo, s_hi) ? kDone : kExactSum;
          if (verdict == kDone) draw();
        }
        if (tid == 0) tell_verdict(verdict);
      }
      cluster_sync(n);
      const uint32_t verdict = sh.verdict;
      if (verdict == kDone) return;
      if (verdict == kExactSum) {
        const double whole = static_cast<double>(exact_sum());
        if (rank == 0) {
          decide(whole, whole);
          draw();
        }
        return;
      }
    }
  }
  // ---- digit by digit, and exact sums of all that is kept
  // One thread of the first CTA tells all CTAs what it found.
  auto tell = [&](const Found& g) {
    const uint64_t* words = reinterpret_cast<const uint64_t*>(&g);
    for (int r = 0; r < n; ++r)
#pragma unroll
      for (int q = 0; q < static_cast<int>(sizeof(Found) / 8); ++q) {
        uint64_t* to = reinterpret_cast<uint64_t*>(&sh.found) + q;
        if (n == 1) *to = words[q];
        else st_cluster(mapa_shared(smem_u32(to), r), words[q]);
      }
  };
  // The lowest key kept by a count (weights false: tokens above it < k) or by weight (above it < target):
  // found key by key range, `with_w` is the weight down to and with it.
  auto search = [&](uint32_t lo, bool by_weight, bool weights, uint32_t k, double target) {
    Found f{lo, most, 0, 0, 0, 0};
    for (int round = 0; round < 4; ++round) {  // (ten bits a round)
      const uint32_t range = f.hi - f.lo;
      const int shift = max(22 - __clz(range | 1), 0);
      for (int i = tid; i < kBins; i += kThreads) {
        sh.digits.count[i] = 0;
        if (weights) sh.digits.lo[i] = sh.digits.hi[i] = 0;
      }
      __syncthreads();
      for (int i = w0 + lane; i < w1; i += 32) {
        const uint4 v = data[i];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const uint32_t b = K::bits(v, e), key = K::of(b);
          if (key < f.lo || key > f.hi) continue;
          const int bin = (f.hi - key) >> shift;
          atomicAdd(&sh.digits.count[bin], 1u);
          if (weights) {
            const uint64_t w = weight(K::value(b), scale, sh.table);
            const uint32_t w_lo = static_cast<uint32_t>(w), old = atomicAdd(&sh.digits.lo[bin], w_lo);
            const uint32_t w_hi = static_cast<uint32_t>(w >> 32) + (old + w_lo < old ? 1u : 0u);
            if (w_hi) atomicAdd(&sh.digits.hi[bin], w_hi);
          }
        }
      }
      cluster_sync(n);
      // each CTA adds up a share of the bins over all CTAs, for the first one
      const int share = kBins / n;
      for (int i = tid; i < share; i += kThreads) {
        const int bin = rank * share + i;
        uint32_t c = 0;
        uint64_t w = 0;
        if (n == 1) {
          c = sh.digits.count[bin];
          if (weights) w = static_cast<uint64_t>(sh.digits.hi[bin]) << 32 | sh.digits.lo[bin];
        } else {
          for (int r = 0; r < n; ++r) {
            c += ld_cluster(mapa_shared(smem_u32(&sh.digits.count[bin]), r));
            if (weights)
              w += (static_cast<uint64_t>(ld_cluster(mapa_shared(smem_u32(&sh.digits.hi[bin]), r))) << 32) +
                   ld_cluster(mapa_shared(smem_u32(&sh.digits.lo[bin]), r));
          }
        }
        if (n == 1) {
          sh.digits.all_count[bin] = c;
          sh.digits.all_w[bin] = w;
        } else {
          st_cluster(mapa_shared(smem_u32(&sh.digits.all_count[bin]), 0), c);
          st_cluster(mapa_shared(smem_u32(&sh.digits.all_w[bin]), 0), w);
        }
      }
      cluster_sync(n);
      if (rank == 0) {
        // sums down to each bin, two a thread
        constexpr int B = kBins / kThreads;
        uint32_t c[B], cs = 0;
        uint64_t w[B], ws = 0;
#pragma unroll
        for (int j = 0; j < B; ++j) {
          c[j] = sh.digits.all_count[tid * B + j];
          w[j] = sh.digits.all_w[tid * B + j];
          cs += c[j];
          ws += w[j];
        }
        uint32_t ci = cs;
        uint64_t wi = ws;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t x = __shfl_up_sync(0xffffffffu, ci, o);
          const uint64_t y = shfl_up(wi, o);
          if (lane >= o) ci += x, wi += y;
        }
        if (lane == 31) sh.warp_u[warp] = ci, sh.warp_w[warp] = wi;
        __syncthreads();
        ci += f.above - cs, wi += f.above_w - ws;
        for (int i = 0; i < warp; ++i) ci += sh.warp_u[i], wi += sh.warp_w[i];
#pragma unroll
        for (int j = 0; j < B; ++j) {
          // the range in which the threshold lies: the last one kept
          const bool here = by_weight ? static_cast<double>(wi) < target && !(static_cast<double>(wi + w[j]) < target)
                                      : ci < k && ci + c[j] >= k;
          if (here && c[j]) {
            const uint32_t hi = f.hi - (static_cast<uint32_t>(tid * B + j) << shift);
            const uint32_t width = (1u << shift) - 1;
            tell(Found{hi - f.lo > width ? hi - width : f.lo, hi, ci, 0, wi, wi + w[j]});
          }
          ci += c[j], wi += w[j];
        }
        if (tid == kThreads - 1 && !by_weight && ci < k) tell(Found{f.lo, f.hi, ci, 1, wi, wi});
      }
      cluster_sync(n);
      f = sh.found;
      if (shift == 0 || f.all) break;
    }
    return f;
  };

  uint64_t whole = 0;  // weight of all that top-k leaves
  if (by_k) {
    const Found f = search(K::LOWEST, false, by_p, k_asked, 0.0);
    least = max(least, f.lo);
    whole = f.with_w;
    if (by_p) {
      const double target = static_cast<double>(p) * static_cast<double>(whole);
      least = max(least, target > 0.0 ? search(f.lo, true, true, 0, target).lo : most);
    }
  } else if (by_p) {
    whole = exact_sum();
    const double target = static_cast<double>(p) * static_cast<double>(whole);
    least = max(least, target > 0.0 ? search(K::LOWEST, true, true, 0, target).lo : most);
  }

  // ---- the kept weights, and the place that u names
  uint64_t sum = 0;
  uint32_t count = 0;
  for (int i = w0 + lane; i < w1; i += 32) {
    const uint4 v = data[i];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const uint32_t b = K::bits(v, e);
      if (K::of(b) >= least) {
        sum += weight(K::value(b), scale, sh.table);
        ++count;
      }
    }
  }
  const uint64_t total = cluster_total(sum);
  const uint64_t at = static_cast<uint64_t>(static_cast<double>(u) * static_cast<double>(total));
  uint64_t below = 0;
  for (int i = 0; i < rank; ++i) below += sh.cta_w[i];
  if (at >= below && at < below + sh.cta_w[rank]) {  // (one CTA)
    for (int i = 0; i < warp; ++i) below += sh.warp_w[i];
    if (at >= below && at < below + sh.warp_w[warp]) {  // (one warp)
      for (int i0 = w0;; i0 += 32) {
        const int i = i0 + lane;
        const uint4 v = i < w1 ? data[i] : make_uint4(E::NOTHING, E::NOTHING, E::NOTHING, E::NOTHING);
        uint64_t part = 0;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const uint32_t b = K::bits(v, e);
          if (K::of(b) >= least) part += weight(K::value(b), scale, sh.table);
        }
        uint64_t upto = part;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t y = shfl_up(upto, o);
          if (lane >= o) upto += y;
        }
        upto += below;
        const unsigned over = __ballot_sync(0xffffffffu, upto > at);
        if (over || i0 + 32 >= w1) {
          if (over && lane == __ffs(over) - 1) {
            uint64_t c = upto - part;
            bool done = false;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              const uint32_t b = K::bits(v, e);
              const float x = K::value(b);
              if (!done && K::of(b) >= least) {
                c += weight(x, scale, sh.table);
                if (c > at) {
                  done = true;
                  a.tokens[row] = (first + i) * VEC + e - skip;
                  if (a.logprob) a.logprob[row] = log_of(x, others_of(total));
                }
              }
            }
          }
          break;
        }
        below = __shfl_sync(0xffffffffu, upto, 31);
      }
    }
  }
  __syncwarp();
  if (a.kept) {
    const uint64_t c = cluster_total(count);
    if (rank == 0 && tid == 0) a.kept[row] = static_cast<int32_t>(c);
  }
}

// CTAs per row: as many as its bytes need, more until every SM has one or a CTA has
// little left.
cudaError_t splits_of(int n_rows, long long row_pieces, int* splits, int* pieces) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  int s = 1;
  while (s < kMaxSplits && (row_pieces * 16 > 56ll * 1024 * s || (static_cast<long long>(n_rows) * s < sms && row_pieces > 2 * kThreads * s))) s *= 2;
  *splits = s;
  *pieces = static_cast<int>((row_pieces + s - 1) / s);
  return cudaSuccess;
}

template <int TYPE>
cudaError_t launch(const SampleArgs& a, cudaStream_t st) {
  const size_t smem = kSharedBytes + static_cast<size_t>(a.pieces) * 16;
  cudaError_t e = cudaFuncSetAttribute(sample_kernel<TYPE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedBytes + kMaxRowBytes);
  if (e == cudaSuccess && a.splits > 8)  // beyond the portable size
    e = cudaFuncSetAttribute(sample_kernel<TYPE>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.n_rows) * a.splits);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.splits;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.splits > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, sample_kernel<TYPE>, a);
}

}  // namespace
}  // namespace dflash

using namespace dflash;

extern "C" {

int dflash_sample_tokens(const void* logits, int32_t type, int64_t row_stride, int32_t n_rows, int32_t vocab,
                         const float* uniform, const float* temperature, const int32_t* top_k, const float* top_p,
                         const float* min_p, int32_t* tokens, float* logprob, int32_t* kept, int32_t* dev_status,
                         dflash_stream_t stream) {
  if (type != DFLASH_T_FP32 && type != DFLASH_T_BF16 && type != DFLASH_T_FP16) return DFLASH_ERR_UNSUPPORTED;
  if (n_rows < 0 || vocab < 1 || row_stride < vocab) return DFLASH_ERR_INVALID_ARG;
  if (vocab > (1 << 19) || n_rows > (1 << 24)) return DFLASH_ERR_CAPACITY;
  if (n_rows == 0) return DFLASH_OK;
  const int size = type == DFLASH_T_FP32 ? 4 : 2;
  if (!logits || reinterpret_cast<uintptr_t>(logits) % size || !uniform || !tokens) return DFLASH_ERR_INVALID_ARG;
  SampleArgs a{};
  const int vec = 16 / size;
  const long long row_pieces = (vocab + vec - 1) / vec + 1;  // (a row may begin inside a piece)
  cudaError_t e = splits_of(n_rows, row_pieces, &a.splits, &a.pieces);
  if (e != cudaSuccess) return cuda_status(e, "sample tokens");
  a.logits = static_cast<const uint8_t*>(logits);
  a.row_bytes = row_stride * size;
  a.n_rows = n_rows;
  a.vocab = vocab;
  while ((1ll << (17 + a.drop)) < vocab) ++a.drop;
  a.uniform = uniform;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.tokens = tokens;
  a.logprob = logprob;
  a.kept = kept;
  a.status = dev_status;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  e = type == DFLASH_T_FP32 ? launch<DFLASH_T_FP32>(a, st)
      : type == DFLASH_T_BF16 ? launch<DFLASH_T_BF16>(a, st)
                              : launch<DFLASH_T_FP16>(a, st);
  return cuda_status(e, "sample tokens");
}

}  // extern "C"
