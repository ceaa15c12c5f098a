// What the kernels that draw tokens share: exact weights, keys, and the row's settings.
//
// A drawn id is a matter of comparisons, so that it has to be the one of the
// definition whatever the order of additions: weights are whole numbers of
// 2^-F, right to about 2^-43 relative or half a unit, and sums of them are exact.  F is as large as
// sums below 2^62 allow (45 if 2^17 tokens may weigh 1 each, 61 if all weigh less than 2), so that the roundings of a whole
// vocabulary are 2^-43 of its weight at most.  e^y is computed in pairs of FP32
// numbers by a table of 2^(j/32) and a short series (Tang, "Table-driven
// implementation of the exponential function", 1989): FP64 instructions are
// sixty times as slow here.
//
// Plain FP32 sums decide wherever their error leaves no doubt.
#pragma once

#include "common.cuh"
#include "internal.h"
#include "kernels.h"
#include "logits.cuh"

namespace dflash {

constexpr int kMaxSplits = 16;       // CTAs of a cluster
constexpr int kFixed = 45;           // binary places of a weight as it is computed
constexpr float kMinTemperature = 0x1p-125f, kMaxTemperature = 0x1p64f;

struct SampleArgs {
  const uint8_t* logits;
  long long row_bytes;
  int n_rows, vocab, splits, pieces;  // pieces: 16-byte pieces of a row that a CTA holds
  int drop;                           // places less than kFixed that sums of any row allow
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
static __constant__ TableEntry kTable[32] = {
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

// e^((x - m) / T) in units of 2^-(kFixed - drop), drop >= -16, N of them side by side: one is a chain of 45 instructions, and the compiler
// does not mix the chains of several by itself (a batch of 32 in a lane: 4.2 us one by one).  Products and sums are written
// out: the compiler must not contract them.
template <int N>
__device__ __forceinline__ void weights(const float (&x)[N], const Scale& c, const TableEntry* table, uint64_t (&w)[N]) {
  constexpr float ROUND = 393216.f;  // 1.5 2^18: adding it leaves multiples of 1/32
  constexpr float LN2 = 0x1.62e430p-1f, LN2_LO = -0x1.05c610p-29f;
  constexpr float STEP1 = 1.5f, STEP2 = 1.5f * 0x1p-22f;
  const float b = -c.m;
  float s[N], e[N], whole[N], p[N], q[N], t[N], rh[N], rl[N], ah[N], al[N], s2[N], s2l[N], cubic[N], uh[N], ul[N], vh[N], vl[N], t1[N], t2[N];
  int k[N];
  TableEntry f[N];
#define DFLASH_EACH _Pragma("unroll") for (int i = 0; i < N; ++i)
  DFLASH_EACH s[i] = __fadd_rn(x[i], b);  // x - m = s + e exactly
  DFLASH_EACH whole[i] = __fmul_rn(s[i], c.hi);
  // (2^-72 is 0, as a masked value's weight is: without a branch)
  DFLASH_EACH p[i] = fmaxf(whole[i], -72.f);
  DFLASH_EACH t[i] = __fadd_rn(p[i], ROUND);
  DFLASH_EACH k[i] = __float_as_int(t[i]) - __float_as_int(ROUND);
  DFLASH_EACH f[i] = table[k[i] & 31];
  DFLASH_EACH {
    const float v = __fsub_rn(s[i], x[i]);
    e[i] = __fadd_rn(__fsub_rn(x[i], __fsub_rn(s[i], v)), __fsub_rn(b, v));
  }
  // times log2(e) / T: p + q = n + j / 32 + r, |r| <= 1/64
  DFLASH_EACH q[i] = __fmaf_rn(e[i], c.hi, __fmaf_rn(s[i], c.lo, __fmaf_rn(s[i], c.hi, -whole[i])));
  DFLASH_EACH {
    const float r = __fsub_rn(p[i], __fsub_rn(t[i], ROUND));
    rh[i] = __fadd_rn(r, q[i]);
    rl[i] = __fsub_rn(q[i], __fsub_rn(rh[i], r));
  }
  // a = r ln 2, u = e^a - 1
  DFLASH_EACH ah[i] = __fmul_rn(rh[i], LN2);
  DFLASH_EACH al[i] = __fadd_rn(__fmaf_rn(rh[i], LN2, -ah[i]), __fmaf_rn(rh[i], LN2_LO, __fmul_rn(rl[i], LN2)));
  DFLASH_EACH s2[i] = __fmul_rn(__fmul_rn(0.5f, ah[i]), ah[i]);
  DFLASH_EACH s2l[i] = __fmaf_rn(ah[i], al[i], __fmaf_rn(__fmul_rn(0.5f, ah[i]), ah[i], -s2[i]));
  // a^3/6 + a^4/24 + a^5/120
  DFLASH_EACH cubic[i] = __fmul_rn(__fmul_rn(s2[i], ah[i]), __fmaf_rn(ah[i], __fmaf_rn(ah[i], 1.f / 60, 1.f / 12), 1.f / 3));
  DFLASH_EACH uh[i] = __fadd_rn(ah[i], s2[i]);
  DFLASH_EACH ul[i] = __fadd_rn(__fsub_rn(s2[i], __fsub_rn(uh[i], ah[i])), __fadd_rn(al[i], __fadd_rn(s2l[i], cubic[i])));
  // times 2^(j / 32): its own whole number, and the rest in two steps of 2^-23 and 2^-45
  DFLASH_EACH vh[i] = __fmul_rn(f[i].hi, uh[i]);
  DFLASH_EACH vl[i] = __fadd_rn(__fmaf_rn(f[i].hi, uh[i], -vh[i]), __fmaf_rn(f[i].hi, ul[i], __fmul_rn(f[i].lo, uh[i])));
  DFLASH_EACH t1[i] = __fadd_rn(__fadd_rn(vh[i], vl[i]), STEP1);
  DFLASH_EACH t2[i] = __fadd_rn(__fadd_rn(__fsub_rn(vh[i], __fsub_rn(t1[i], STEP1)), vl[i]), STEP2);
  DFLASH_EACH {
    const long long add = (static_cast<long long>(__float_as_int(t1[i]) - __float_as_int(STEP1)) << 22) +
                          (__float_as_int(t2[i]) - __float_as_int(STEP2));
    const int places = c.drop + 17 - (k[i] >> 5), right = min(places, 63);  // (1 or more)
    w[i] = places < 64 ? (((f[i].fixed + add) << 17) + (1ull << (right - 1))) >> right : 0;
  }
#undef DFLASH_EACH
}
__device__ __forceinline__ uint64_t weight(float x, const Scale& c, const TableEntry* table) {
  const float in[1] = {x};
  uint64_t out[1];
  weights(in, c, table, out);
  return out[0];
}
// By a call, for steps that few rows take: their instructions come from L2, so that there is one copy.
__device__ __noinline__ static uint64_t weight_by_call(float x, const Scale* c, const TableEntry* table) { return weight(x, *c, table); }

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
  // the smaller of two words' values, value by value; whether a word holds a -infinity
  static __device__ __forceinline__ uint32_t min_words(uint32_t a, uint32_t b) {
    if constexpr (WIDE) {
      return __float_as_uint(fminf(__uint_as_float(a), __uint_as_float(b)));
    } else if constexpr (TYPE == DFLASH_T_BF16) {
      const __nv_bfloat162 m = __hmin2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
      return *reinterpret_cast<const uint32_t*>(&m);
    } else {
      const __half2 m = __hmin2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
      return *reinterpret_cast<const uint32_t*>(&m);
    }
  }
  static __device__ __forceinline__ bool masked(uint32_t w) {
    if constexpr (WIDE) return w == (SIGN | INF);
    return (w & 0xffffu) == (SIGN | INF) || w >> 16 == (SIGN | INF);
  }
  static __device__ __forceinline__ bool has_nan(uint32_t w) {
    if constexpr (WIDE) return (w & 0x7fffffffu) > INF;
    return (w & 0x7fffu) > INF || (w >> 16 & 0x7fffu) > INF;
  }
  static __device__ __forceinline__ float top_of(const uint4& v) {
    using E = Elem<TYPE>;
    return E::max_of(E::max_words(E::max_words(v.x, v.y), E::max_words(v.z, v.w)));
  }
  // FP32 sum of 2^(x c + k) of a piece: an exponent is rounded once.  (Pairs of values in one instruction
  // take fewer instructions and more time: 65 us instead of 59 for 1000 rows of 151936.)
  static __device__ __forceinline__ float quick_sum_from(const uint4& v, float c, float k) {
    constexpr int VEC = Elem<TYPE>::VEC;
    float x[VEC];
    Elem<TYPE>::widen(v, x);
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = ex2_approx(fmaf(x[e], c, k));
#pragma unroll
    for (int o = VEC / 2; o; o >>= 1)
#pragma unroll
      for (int e = 0; e < o; ++e) x[e] += x[e + o];
    return x[0];
  }
  // exact weight of a piece's values, four side by side
  static __device__ __forceinline__ uint64_t exact_sum(uint4 v, const Scale& c, const TableEntry* table) {
    constexpr int VEC = Elem<TYPE>::VEC, N = 4;
    uint64_t sum = 0;
    // (not unrolled: the instructions of a piece in line are fetched slower than they run)
#pragma unroll 1
    for (int e0 = 0; e0 < VEC; e0 += N) {
      float x[N];
      uint64_t w[N];
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] = value(bits(v, e));
      v.x = v.z, v.y = v.w;  // (16-bit values: the other four)
      weights(x, c, table, w);
#pragma unroll
      for (int e = 0; e < N; ++e) sum += w[e];
    }
    return sum;
  }
  // The first value of a piece (the same in all lanes) with which the exact weights from `from` on exceed `place`: the lane
  // that has it.  Each lane has one value.
  static __device__ __forceinline__ bool exact_find(const uint4& v, uint64_t from, uint64_t place, const Scale& c,
                                                    const TableEntry* table, int lane, float& x) {
    constexpr int VEC = Elem<TYPE>::VEC;
    uint32_t b = SIGN | INF;
#pragma unroll
    for (int e = 0; e < VEC; ++e) b = lane == e ? bits(v, e) : b;
    x = value(b);
    uint64_t upto = lane < VEC ? weight(x, c, table) : 0;
#pragma unroll
    for (int o = 1; o < VEC; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    const unsigned over = __ballot_sync(0xffffffffu, from + upto > place);
    return lane == __ffs(over) - 1;
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
  static __device__ __forceinline__ uint32_t at_least(double x) { return at_least(__double2float_ru(x)); }
  static __device__ __forceinline__ uint32_t at_least(float f) {
    if constexpr (WIDE) return of(__float_as_uint(f));
    if constexpr (TYPE == DFLASH_T_BF16) return of(__bfloat16_as_ushort(__float2bfloat16_ru(f)));
    return of(__half_as_ushort(__float2half_ru(f)));
  }
};

// ------------------------------------------------------------------ clusters
// (The aligned barrier wants its warp's lanes together, which a branch by lane before it does not promise.)
__device__ __forceinline__ void cluster_sync(int splits) {
  if (splits > 1) {
    __syncwarp();
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
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
// The sum of a word over the CTAs of a cluster: all reads first, which take long (one after the other 4 us with 16 CTAs).
__device__ __forceinline__ uint64_t cluster_sum(const uint32_t* word, int n) {
  const uint32_t at = smem_u32(word);
  uint32_t v[kMaxSplits];
#pragma unroll
  for (int r = 0; r < kMaxSplits; ++r) v[r] = r < n ? ld_cluster(mapa_shared(at, r)) : 0;
  uint64_t sum = 0;
#pragma unroll
  for (int r = 0; r < kMaxSplits; ++r) sum += v[r];
  return sum;
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

// A row's settings, made safe.
struct Settings {
  float temperature, p, min_p, u;
  int k;
  bool greedy, by_k, by_p, by_min, fine;
  __device__ __forceinline__ Settings(const SampleArgs& a, int row) {
    const float t = a.temperature ? a.temperature[row] : 1.f;
    temperature = t > kMaxTemperature ? kMaxTemperature : t > 0.f && t < kMinTemperature ? kMinTemperature : t;
    greedy = !(temperature > 0.f);
    k = a.top_k ? a.top_k[row] : 0;
    by_k = k > 0 && k < a.vocab;
    p = a.top_p ? a.top_p[row] : 1.f;
    by_p = p < 1.f;
    min_p = a.min_p ? a.min_p[row] : 0.f;
    by_min = min_p > 0.f;
    u = a.uniform[row];
    fine = t >= 0.f && t <= kMaxTemperature && u >= 0.f && u < 1.f && p == p && min_p <= 1.f;
    if (!(u >= 0.f)) u = 0.f;
    if (u >= 1.f) u = 0x1.fffffep-1f;
  }
  // log2(e) / T as the sum of two
  __device__ __forceinline__ void scale(Scale& s, int drop) const {
    const double c = 1.4426950408889634 / static_cast<double>(temperature);
    s.hi = static_cast<float>(c);
    s.lo = static_cast<float>(c - static_cast<double>(s.hi));
    s.drop = drop;
  }
  // ln(w / total) of a token, where the largest weight, 1, is among those of the total: `others` are the total less 1
  __device__ __forceinline__ float log_of(float x, float m, float others) const { return (x - m) / temperature - log1pf(others); }
};
// The places less than kFixed of the weights of tokens that weigh `sum` together, as FP32 sums have it.
__device__ __forceinline__ int drop_of(float sum, int most) {
  return min(max((__float_as_int(sum * (1.f + 0x1p-9f)) >> 23) - 127, 0) - 16, most);
}
__device__ __forceinline__ float others_of(uint64_t total, int drop) {
  return static_cast<float>(total - (1ull << (kFixed - drop))) * exp2f(static_cast<float>(drop - kFixed));
}

// Numbers below this leave the token to sums in FP64, in which small weights keep all their places.  (In whole numbers u times the sum would be few units
// or none, and a weight that rounds to 0 could never be drawn, not even by 0.)
constexpr float kSmallNumber = 0x1p-24f;

// Draws by such a number, by one CTA: the first token with which the weights of keys from `cut` on, which come to `total` with `drop` places less
// and are `kept` tokens, exceed u times that.  Reads the row in order of ids, as far as it has to.  (Eight rows of 151936 values, all with such a
// number: 60 to 115 us where the first ids have weight, 170 to 260 where only the last 100 have.)
template <int TYPE>
__device__ __noinline__ void draw_small(const SampleArgs& a, int row, uint32_t cut, float m, uint64_t total, int drop, uint32_t kept, double* sums) {
  constexpr int PER = 8;  // neighbours of a thread
  const Settings set(a, row);
  const uint8_t* src = a.logits + row * a.row_bytes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
  // (below the largest weight, 1, so that one passes it)
  const double target = static_cast<double>(set.u) * static_cast<double>(total) * static_cast<double>(exp2f(static_cast<float>(drop - kFixed)));
  auto value = [&](int i) { return i < a.vocab ? Elem<TYPE>::one(src, i) : -INFINITY; };
  auto weight_of = [&](float x) {  // (those that FP64 has as 0 without its exponential)
    if (!(x > -INFINITY) || Keys<TYPE>::of_value(x) < cut || (x - m) / set.temperature < -750.f) return 0.0;
    const double z = (static_cast<double>(x) - static_cast<double>(m)) / static_cast<double>(set.temperature);
    // (2^-1074, its smallest number, from ln 2^-1075 on: the exponential may have the last of them as 0)
    return fmax(exp(z), z > -745.13321910194110842 ? 0x1p-1074 : 0.0);
  };
  double from = 0.0;  // weights before the threads' values
#pragma unroll 1
  for (int i0 = 0; i0 < a.vocab; i0 += PER * blockDim.x) {
    const int first = i0 + tid * PER;
    double sum = 0.0;
#pragma unroll 1
    for (int e = 0; e < PER; ++e) sum += weight_of(value(first + e));
    if (!__syncthreads_or(sum > 0.0)) continue;  // (and the last sums have been read)
    double upto = sum;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    double before = __shfl_up_sync(0xffffffffu, upto, 1);
    if (lane == 0) before = 0.0;
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < warps; ++i) {
      if (i == warp) upto += from, before += from;
      from += sums[i];
    }
    // (a lane without weight may have a sum that differs in its last place from the one before)
    const unsigned past = __ballot_sync(0xffffffffu, sum > 0.0 && upto > target);
    if (!__syncthreads_or(past != 0)) continue;
    int* lanes = reinterpret_cast<int*>(sums);  // the first of each warp
    if (lane == 0) lanes[warp] = __ffs(past) - 1;
    __syncthreads();
    int who = 0;
    while (lanes[who] < 0) ++who;
    if (warp == who && lane == lanes[who]) {
      int id = 0;
#pragma unroll 1
      for (int e = 0; e < PER; ++e) {
        const double w = weight_of(value(first + e));
        if (!(w > 0.0)) continue;
        id = first + e;  // (one with a weight, also where the sums before it and with it end a place beside those above)
        before += w;
        if (before > target) break;
      }
      a.tokens[row] = id;
      if (a.logprob) a.logprob[row] = set.log_of(value(id), m, others_of(total, drop));
      if (a.kept) a.kept[row] = static_cast<int32_t>(kept);
    }
    return;
  }
}

// Rows without a filter (sample_plain.cu).
cudaError_t launch_sample_plain(SampleArgs a, int type, cudaStream_t st);

}  // namespace dflash
