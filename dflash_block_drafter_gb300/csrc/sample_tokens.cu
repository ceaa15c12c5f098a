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
// from global memory however often it is looked at.  A threshold is found
// digit by digit: counts (and weights) of up to 1024 ranges of the keys, in which
// the largest key comes first, then of the ranges of the one in which the
// threshold lies, until it is one key.
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
constexpr int kMaxRowBytes = 184 * 1024;   // of a row in one CTA
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
  uint32_t count[kBins], lo[kBins], hi[kBins];  // of this CTA's tokens; weights in two words
  uint32_t all_count[kBins];                    // of the cluster's, in its first CTA
  uint64_t all_w[kBins];
  TableEntry table[32];
  Found found;
  uint64_t cta_w[kMaxSplits], warp_w[kWarps];
  uint32_t cta_u[kMaxSplits], warp_u[kWarps];
  double log_min_p;
  Scale scale;
};

template <int TYPE>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
  using E = Elem<TYPE>;
  using K = Keys<TYPE>;
  constexpr int VEC = E::VEC;
  extern __shared__ uint4 data[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = blockIdx.x / a.splits, rank = blockIdx.x - row * a.splits;
  const int n = a.splits;

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
  float top = -INFINITY;
  bool nan = false;
  for (int i = tid; i < mine; i += kThreads) {
    const long long p0 = static_cast<long long>(first + i) * VEC - skip;  // value of the piece's first place
    uint4 v;
    if (p0 >= 0 && p0 + VEC <= a.vocab) {
      v = __ldcs(frame + first + i);
    } else {
      constexpr int W = VEC / 4;
      v.x = E::raw(src, p0, a.vocab);
      v.y = E::raw(src, p0 + W, a.vocab);
      v.z = E::raw(src, p0 + 2 * W, a.vocab);
      v.w = E::raw(src, p0 + 3 * W, a.vocab);
    }
    data[i] = v;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float x = K::value(K::bits(v, e));
      nan |= x != x;
      top = fmaxf(top, x);
    }
  }
  {
    uint32_t key = nan ? 0xffffffffu : float_order_key(top);  // (no value's key is that large)
    key = __reduce_max_sync(0xffffffffu, key);
    if (lane == 0) sh.warp_u[warp] = key;
    __syncthreads();
    if (tid < 32) {
      key = __reduce_max_sync(0xffffffffu, lane < kWarps ? sh.warp_u[lane] : 0u);
      if (n == 1) {
        if (lane == 0) sh.cta_u[0] = key;
      } else if (lane < n) {
        st_cluster(mapa_shared(smem_u32(&sh.cta_u[rank]), lane), key);
      }
    }
  }
  cluster_sync(n);
  uint32_t top_key = 0;
  for (int i = 0; i < n; ++i) top_key = max(top_key, sh.cta_u[i]);
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
  const uint32_t most = [&] {  // the key of m
    if constexpr (K::WIDE) return K::of(__float_as_uint(m));
    else if constexpr (TYPE == DFLASH_T_BF16) return K::of(__float_as_uint(m) >> 16);
    else return K::of(__half_as_ushort(__float2half_rn(m)));
  }();
  uint32_t least = K::LOWEST;
  if (by_min) least = max(least, min(most, K::at_least(static_cast<double>(m) + sh.log_min_p)));

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
        sh.count[i] = 0;
        if (weights) sh.lo[i] = sh.hi[i] = 0;
      }
      __syncthreads();
      for (int i = w0 + lane; i < w1; i += 32) {
        const uint4 v = data[i];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const uint32_t b = K::bits(v, e), key = K::of(b);
          if (key < f.lo || key > f.hi) continue;
          const int bin = (f.hi - key) >> shift;
          atomicAdd(&sh.count[bin], 1u);
          if (weights) {
            const uint64_t w = weight(K::value(b), scale, sh.table);
            const uint32_t w_lo = static_cast<uint32_t>(w), old = atomicAdd(&sh.lo[bin], w_lo);
            const uint32_t w_hi = static_cast<uint32_t>(w >> 32) + (old + w_lo < old ? 1u : 0u);
            if (w_hi) atomicAdd(&sh.hi[bin], w_hi);
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
          c = sh.count[bin];
          if (weights) w = static_cast<uint64_t>(sh.hi[bin]) << 32 | sh.lo[bin];
        } else {
          for (int r = 0; r < n; ++r) {
            c += ld_cluster(mapa_shared(smem_u32(&sh.count[bin]), r));
            if (weights)
              w += (static_cast<uint64_t>(ld_cluster(mapa_shared(smem_u32(&sh.hi[bin]), r))) << 32) +
                   ld_cluster(mapa_shared(smem_u32(&sh.lo[bin]), r));
          }
        }
        if (n == 1) {
          sh.all_count[bin] = c;
          sh.all_w[bin] = w;
        } else {
          st_cluster(mapa_shared(smem_u32(&sh.all_count[bin]), 0), c);
          st_cluster(mapa_shared(smem_u32(&sh.all_w[bin]), 0), w);
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
          c[j] = sh.all_count[tid * B + j];
          w[j] = sh.all_w[tid * B + j];
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
    uint64_t sum = 0;
    for (int i = w0 + lane; i < w1; i += 32) {
      const uint4 v = data[i];
#pragma unroll
      for (int e = 0; e < VEC; ++e) sum += weight(K::value(K::bits(v, e)), scale, sh.table);
    }
    whole = cluster_total(sum);
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
                  // ln(w / total): the largest weight, 1, is among the kept ones
                  if (a.logprob)
                    a.logprob[row] = (x - m) / temperature -
                                     log1pf(static_cast<float>(total - (1ull << (kFixed - a.drop))) * exp2f(static_cast<float>(a.drop - kFixed)));
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
  while (s < kMaxSplits && (row_pieces * 16 > 72ll * 1024 * s || (static_cast<long long>(n_rows) * s < sms && row_pieces > 2 * kThreads * s))) s *= 2;
  *splits = s;
  *pieces = static_cast<int>((row_pieces + s - 1) / s);
  return cudaSuccess;
}

template <int TYPE>
cudaError_t launch(const SampleArgs& a, cudaStream_t st) {
  const size_t smem = static_cast<size_t>(a.pieces) * 16;
  cudaError_t e = cudaFuncSetAttribute(sample_kernel<TYPE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxRowBytes);
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
