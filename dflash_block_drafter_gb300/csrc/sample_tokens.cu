// Tokens drawn from rows of logits (dflash_sample_tokens in include/dflash.h).
//
//   w_i = e^((x_i - m) / T),  m = max x
//   kept: x_i >= the k-th largest;  A(x_i) < p S, where A(v) is the weight of the kept
//   tokens above v and S that of all;  w_i >= min_p;  x_i > -infinity
//   token: the first id whose kept weights up to it, in order of ids, exceed u times all of them.
//
// (Exact weights: sampling.cuh.)
//
// Rows with a filter; calls without any go to sample_plain.cu.  The CTAs of a cluster hold a row in their
// shared memory, so that it is read once from global memory however often it is looked at.  Few tokens decide
// most rows, and plain FP32 finds them:
//  - A bound below the threshold.  Of top-k: the k-th largest of the threads' own maxima, by a
//    histogram of them.  Of top-p: the first of 512 ranges of logits below which less than
//    (1 - p) S can lie, counted with each range's largest weight.  Of min-p: itself.  The
//    tokens above the bound, if they are at most kList, go to the first CTA, which
//    compares them (or sorts them) and decides everything with exact weights.  S itself, which a top-p without top-k
//    compares with, comes from FP32 sums; where their error leaves it open which token is the last, S is added up exactly.
// Else (long lists) a threshold is found digit by digit: counts, or weights, of up to
// 2048 ranges of the keys, then of the ranges of the one in which the threshold lies, until it is one key; and the token by
// the sums of the CTAs and threads.  FP32 weights do first, in whole numbers, whose sums are exact, and exact ones if those leave a
// decision open: whether a border of the token, or of the last key, lies within their error of what it is compared with.
//
// That error, in units of 2^-24 of the sum S: a weight is 2^(x c + k), k = -m c as FP32 has it (what it is off by is the same for all weights).
// The exponent y is off by 2 |y| (its own rounding and c's, |y| each at most), and the mean of |y| over the weights is their entropy less log2 S,
// log2(vocab / S) at most: with ln 2, 1.39 log2(vocab / S).  2^y 4, its rounding to a whole number less than 1.  A border and u S (or p S) are sums of
// the same numbers, so that a weight's error counts 1 - u times before the border and u times behind it: 1.39 log2(vocab / S) + 5 / 2, below
// 1.4 log2(vocab / S) + 4.  S itself against exact weights has a piece's sum, 3, and the largest weight that it is divided by, 4, besides: 12, and 13 is taken.
//
// Measured, calls in a row: 8 rows of 151936 BF16 values, top-p, 24 to 31 us, of which 24 are the host's (floor 0.4); 256 rows of FP16 values, top-k 50,
// 62 to 65 us (floor 11), top-k 50 with top-p 70, min-p 52, top-p 0.9 to 0.99 142 to 245, top-p 0.9 of flat rows 288; 128 rows of 100003 FP32 values
// with settings of their own 53 to 125 us, 88 in the mean of 80 seeds (floor 7.5).  A row takes its cluster 12 to 15 us,
// a chain of seven short phases between barriers (maximum, bound, list, weights, decision; issue slots 35 %), and there are two or three rows
// behind one another; the last kind ends with a flat row whose nucleus goes digit by digit, 40 us if FP32 decides it and 80 if not.
#include <cstddef>

#include "common.cuh"
#include "internal.h"
#include "kernels.h"
#include "sampling.cuh"

namespace dflash {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kBins = 2048;
constexpr int kMaxRowBytes = 160 * 1024;   // of a row in one CTA
constexpr int kPerSm = 2;                  // CTAs
// Lists.  256 rows of 151936 FP16 values: with the 600 best of each, 118 us, and 222 without lists of more than 512, whose rows go digit by
// digit; with the 90, 130 and 200 best (lists are somewhat longer) 71, 82 and 96 us, and 70, 86 and 89 if no more than 128 are compared each
// with each, 81, 85 and 88 if no more than 64.
constexpr int kList = 1024;                // tokens that the first CTA sorts
constexpr int kOwn = kList / kWarps;       // of a warp
constexpr int kFew = 256;                  // tokens that it compares each with each
constexpr int kListDrop = -7;              // places less than kFixed of a list's weights
// A row that is a list as a whole.  (400 rows of 300 and 500 values: 29 to 31 us; with a bound first 19 to 25 by top-k and 29 to 34 by top-p.  Rows of few
// pieces have no bound: their threads' maxima are too few.)
constexpr int kShort = kList / 2;
constexpr int kQuickBins = kThreads;       // ranges of the first bounds

// The keys among which the lowest one kept lies, the weight (or number) of the tokens above them and of all, and whether it is
// known to lie there.
struct Found {
  uint32_t lo, hi;
  uint64_t above, whole, certain;
};

struct Shared {
  union {
    struct {
      uint32_t lo[kBins], hi[kBins];  // weights of this CTA's tokens, in two words
      uint64_t all[kBins];            // of the cluster's, in its first CTA
    } digits;
    struct {
      uint64_t own[kWarps][kOwn];  // (key, id) of each warp's tokens, in order of ids
      uint64_t list[kList];        // the same of the cluster, in its first CTA
      uint64_t sorted[kList];      // (key, place in `list`), largest first
      uint64_t upto[kList];        // weights before each of them; of few tokens: of each
      uint32_t hist[kQuickBins];
      uint32_t many[kMaxSplits * kWarps];  // tokens of each warp of the cluster
    } quick;
  };
  TableEntry table[32];
  Found found;
  uint64_t cta_w[kMaxSplits], warp_w[kWarps];
  uint64_t cta_above[kMaxSplits], cta_rest[kMaxSplits];  // weights outside of the ranges, in the first CTA
  uint32_t cta_top[kMaxSplits], cta_low[kMaxSplits], cta_n[kMaxSplits], cta_c[kMaxSplits], warp_u[kWarps], warp_low[kWarps], warp_n[kWarps];
  float warp_f[kWarps];
  double log_min_p;
  Scale scale;
  float bound, upper;
  uint64_t target;
  uint32_t verdict;
  int where;      // the values in which u lies, and the weight before them
  uint64_t from;
};
// (a CTA that goes on to the digits leaves a slower one its histogram)
static_assert(offsetof(Shared, quick.hist) >= sizeof(Shared::digits), "the digits lie before the histogram");
static_assert(kList <= 64 * kWarps && kFew <= kThreads / 2, "a warp sorts 64 tokens, two threads compare one");
constexpr int kSharedBytes = (sizeof(Shared) + 15) / 16 * 16;
// What the first CTA (or the one that u names) says of a quick answer.
enum Verdict : uint32_t { kDone, kExactSum, kDigits };

// The exact weights of a thread's values, by a call: few rows have to know them.
template <int TYPE>
__device__ __noinline__ uint64_t exact_values(const uint4* data, int t0, int t1, const Scale* c, const TableEntry* table) {
  uint64_t sum = 0;
#pragma unroll 1
  for (int i = t0; i < t1; ++i) {
    uint32_t b;
    if constexpr (Keys<TYPE>::WIDE) b = reinterpret_cast<const uint32_t*>(data)[i];
    else b = reinterpret_cast<const uint16_t*>(data)[i];
    sum += weight(Keys<TYPE>::value(b), *c, table);
  }
  return sum;
}

template <int TYPE>
__global__ void __launch_bounds__(kThreads, kPerSm) sample_kernel(const __grid_constant__ SampleArgs a) {
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

  const Settings set(a, row);
  const bool by_k = set.by_k, by_p = set.by_p, by_min = set.by_min;
  const int k_asked = set.k;
  const float p = set.p, u = set.u;
  if (tid < 32) sh.table[tid] = kTable[tid];
  if (tid == kThreads - 1) {
    if (rank == 0 && !set.fine) set_status(a.status, DFLASH_DEV_BAD_VALUE);
    if (!set.greedy) {
      set.scale(sh.scale, kListDrop);
      if (by_min) sh.log_min_p = static_cast<double>(set.temperature) * log(static_cast<double>(fminf(set.min_p, 1.f)));
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
  const bool of_cta = lane < n;
  const uint32_t top_key = __reduce_max_sync(0xffffffffu, of_cta ? sh.cta_top[lane] : 0u);
  const uint32_t low_key = __reduce_min_sync(0xffffffffu, of_cta ? sh.cta_low[lane] : 0xffffffffu);
  const uint32_t maxima = __reduce_add_sync(0xffffffffu, of_cta ? sh.cta_n[lane] : 0u);
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

  if (set.greedy) {  // the first id of the largest value
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
  const Scale* const scale = &sh.scale;
  const float c_hi = sh.scale.hi;
  const uint32_t most = K::of_value(m);
  uint32_t least = K::LOWEST;
  if (by_min) least = max(least, min(most, K::at_least(static_cast<double>(m) + sh.log_min_p)));

  // FP32 weights, 2^(x c + k), in the units of the exact ones: sums are whole numbers too.
  const float k_hi = -(m * c_hi);
  const bool in_range = fabsf(m) * c_hi < 0x1p20f;  // (k is off by 2^-4 at most)
  const float one = ex2_approx(fmaf(m, c_hi, k_hi));  // the largest of them
  const float unit = __int_as_float((127 + kFixed - a.drop) << 23);
  auto fixed = [&](float w) { return static_cast<uint64_t>(__float2ull_rn(w * unit)); };
  auto quick_weight = [&](float x) { return fixed(ex2_approx(fmaf(x, c_hi, k_hi))); };
  // What such sums may be off by, relative: `more` units of 2^-24 and those of the exponents
  auto error_of = [&](uint64_t sum, float more) {
    return 0x1p-24f * (more + 1.4f * log2f(static_cast<float>(a.vocab) * unit / static_cast<float>(sum)));
  };
  auto one_weight = [&](float x) { return weight_by_call(x, scale, sh.table); };
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
  // The sum over the cluster of the CTAs' v and counts, and that of the CTAs before this one.
  auto exchange = [&](uint64_t v, uint32_t& count, uint64_t& below) {
    if (n == 1) {
      below = 0;
      return v;
    }
    cluster_sync(n);  // the last values have been read
    if (tid < n) {
      st_cluster(mapa_shared(smem_u32(&sh.cta_w[rank]), tid), v);
      st_cluster(mapa_shared(smem_u32(&sh.cta_c[rank]), tid), count);
    }
    __syncwarp();
    cluster_sync(n);
    const uint64_t w = lane < n ? sh.cta_w[lane] : 0;
    count = __reduce_add_sync(0xffffffffu, lane < n ? sh.cta_c[lane] : 0u);
    below = warp_sum(lane < rank ? w : uint64_t(0));
    return warp_sum(w);
  };
  // The rare steps take a thread's values one by one, neighbours in the row: few instructions (unrolled over pieces they took 5 us
  // each the first time, most of it to fetch them), and a thread's sum leads to its values.
  const int per_thread = (mine * VEC + kThreads - 1) / kThreads | 1;  // odd: no two lanes in a bank
  const int t0 = min(tid * per_thread, mine * VEC), t1 = min(t0 + per_thread, mine * VEC);
  auto bits_at = [&](int i) -> uint32_t {
    if constexpr (K::WIDE) return reinterpret_cast<const uint32_t*>(data)[i];
    else return reinterpret_cast<const uint16_t*>(data)[i];
  };
  // The exact weight of all tokens.
  auto exact_sum = [&]() {
    uint64_t all, below;
    uint32_t none = 0;
    scan(exact_values<TYPE>(data, t0, t1, scale, sh.table), all);
    return exchange(all, none, below);
  };
  auto tell_verdict = [&](uint32_t v) {  // (one thread)
    for (int r = 0; r < n; ++r) {
      if (n == 1) sh.verdict = v;
      else st_cluster(mapa_shared(smem_u32(&sh.verdict), r), v);
    }
  };

  const bool filter = by_k || by_p || by_min;
  uint32_t from_key = K::LOWEST;  // no threshold of top-k and top-p lies below
  uint32_t to_key = most;         // nor one of top-p alone above
  uint64_t quick_total = 0;       // FP32 weights of all tokens, by top-p alone
  if (filter && u >= kSmallNumber) {  // (smaller numbers draw by FP64 weights: their rows find their thresholds digit by digit)
    // ---- a bound below the thresholds
    float bound = -INFINITY;  // logits from here on
    bool quick = true;
    if (a.vocab <= kShort) {  // the whole row is a list
    } else if (by_k) {
      const float low = float_from_order_key(low_key), per = m > low ? (kQuickBins - 1) / (m - low) : 0.f;
      quick = maxima >= static_cast<uint32_t>(k_asked) && per < 1e30f && per > 0.f;
      if (quick) {
        if (top > -INFINITY) atomicAdd(&sh.quick.hist[min(static_cast<int>((m - top) * per), kQuickBins - 1)], 1u);
        cluster_sync(n);
        const uint32_t c = n == 1 ? sh.quick.hist[tid] : static_cast<uint32_t>(cluster_sum(&sh.quick.hist[tid], n));
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
      quick = cut < 40.f && in_range;
      if (quick) {
        for (int i = w0 + lane; i < w1; i += 32) {
          const uint4 v = data[i];
          quick_total += fixed(K::quick_sum_from(v, c_hi, k_hi));
          if ((m - K::top_of(v)) * c_hi < cut) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              const float z = (m - K::value(K::bits(v, e))) * c_hi;
              if (z < cut) atomicAdd(&sh.quick.hist[min(static_cast<int>(z * per), kQuickBins - 1)], 1u);
            }
          }
        }
        quick_total = warp_sum(quick_total);
        if (lane == 0) sh.warp_w[warp] = quick_total;
        __syncthreads();
        if (tid < 32) {
          const uint64_t v = warp_sum(lane < kWarps ? sh.warp_w[lane] : uint64_t(0));
          if (n == 1) {
            if (lane == 0) sh.cta_w[0] = v;
          } else if (lane < n) {
            st_cluster(mapa_shared(smem_u32(&sh.cta_w[rank]), lane), v);
          }
        }
        cluster_sync(n);
        quick_total = warp_sum(lane < n ? sh.cta_w[lane] : uint64_t(0));
        // what the ranges from the last one up to this thread's weigh at most
        const int bin = kQuickBins - 1 - tid;
        const uint32_t c = n == 1 ? sh.quick.hist[bin] : static_cast<uint32_t>(cluster_sum(&sh.quick.hist[bin], n));
        const float w = static_cast<float>(c) * ex2_approx(-static_cast<float>(bin) / per);
        float x = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        __syncthreads();  // warp_f has been read
        if (lane == 31) sh.warp_f[warp] = x;
        if (tid == 0) sh.bound = -INFINITY, sh.upper = INFINITY;
        __syncthreads();
        float every = 0.f;
        for (int i = 0; i < kWarps; ++i) {
          const float y = sh.warp_f[i];
          if (i < warp) x += y;
          every += y;
        }
        const float over = every * (1.f + 0x1p-13f) - x;  // the ranges above this one, at most (2^-13: more than all roundings)
        x += rest * 0.25f;
        // (2^-10: more than the sums and ranges are off; the FP32 weights are relative to 2^(m c + k))
        const float sum = static_cast<float>(quick_total) / unit / one, whole = sum * (1.f - 0x1p-10f);
        const float most_left = rest * whole, least_kept = p * whole;
        if (tid == 0) sh.scale.drop = drop_of(sum, a.drop);
        // the first range that has to be kept: with it more than may be left out would be
        if (x > most_left && x - w <= most_left) sh.bound = m - (bin + 1) / per / c_hi * (1.f + 0x1p-20f);
        // and the last one that has to be left for others to be kept
        if (over <= least_kept && over + w > least_kept) sh.upper = m - bin / per / c_hi * (1.f - 0x1p-20f);
        __syncthreads();
        bound = sh.bound;
        if (sh.upper < INFINITY) to_key = min(most, K::at_least(sh.upper));
        if (bound > -INFINITY) from_key = max(from_key, min(most, K::at_least(bound)));
        // (too long a list is not made; min-p may shorten it)
        const uint32_t listed = __reduce_add_sync(0xffffffffu, (m - bound) * c_hi * per > bin ? c : 0u);
        if (lane == 0) sh.warp_n[warp] = listed;
        __syncthreads();
        uint32_t all = 0;
        for (int i = 0; i < kWarps; ++i) all += sh.warp_n[i];
        quick = bound > -INFINITY && (by_min || all <= kList);
      }
    }
    if (by_k && bound > -INFINITY) from_key = max(from_key, min(most, K::at_least(bound)));
    // (top-p needs the whole of what top-k leaves, and in a short row of all)
    if (by_min && !(by_p && (by_k || a.vocab <= kShort))) bound = fmaxf(bound, K::value_of(least));

    if (quick) {
      // ---- the tokens from the bound on, in order of their ids: each warp's own
      uint32_t own = 0;
      for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        const uint4 v = i < w1 ? data[i] : make_uint4(E::NOTHING, E::NOTHING, E::NOTHING, E::NOTHING);
        const float most_of = K::top_of(v);
        if (!__any_sync(0xffffffffu, most_of >= bound && most_of > -INFINITY)) continue;
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
        uint32_t at = own + upto - c;
        if (c) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const uint32_t b = K::bits(v, e);
            const float x = K::value(b);
            if (x >= bound && x > -INFINITY) {
              if (at < kOwn) sh.quick.own[warp][at] = static_cast<uint64_t>(K::of(b)) << 32 | static_cast<uint32_t>((first + i) * VEC + e - skip);
              ++at;
            }
          }
        }
        own += __shfl_sync(0xffffffffu, upto, 31);
      }
      if (lane == 0) {
        if (n == 1) sh.quick.many[warp] = own;
        else st_cluster(mapa_shared(smem_u32(&sh.quick.many[rank * kWarps + warp]), 0), own);
      }
      cluster_sync(n);
      uint32_t keep = 0, size = 0;
      uint64_t kept_w = 0;
      uint32_t cut_key = 0;
      // Few tokens: four or two threads for each compare it with all others.
      bool few = false;
      uint32_t each = 4, me = 0;
      uint32_t my_key = 0, larger = 0;  // tokens above this one
      uint64_t my_w = 0, above = 0;     // and their weight
      auto decide_few = [&](double s_lo, double s_hi) {  // false if S has to be exact
        const bool real = me < size && tid % each == 0;
        bool stays = real && my_key >= least, open = false;
        if (by_k) stays = stays && larger < static_cast<uint32_t>(k_asked);
        if (by_p) {
          if (by_k) {
            uint64_t all;
            // (what top-k leaves, whatever min-p says of it)
            scan(real && larger < static_cast<uint32_t>(k_asked) ? my_w : 0, all);
            s_lo = s_hi = static_cast<double>(all);
          }
          const double lo = static_cast<double>(p) * s_lo, hi = static_cast<double>(p) * s_hi, over = static_cast<double>(above);
          open = stays && larger > 0 && over >= lo && over < hi;
          stays = stays && (larger == 0 || over < lo);
        }
        keep = __syncthreads_count(stays);
        if (real) sh.quick.upto[me] = stays ? my_w : 0;
        return !__syncthreads_or(open);
      };
      auto draw_few = [&]() {
        if (warp != 0) return;
        constexpr int EACH = kFew / 32;
        uint64_t w[EACH], mine_w = 0;
#pragma unroll
        for (int j = 0; j < EACH; ++j) {
          w[j] = lane * EACH + j < size ? sh.quick.upto[lane * EACH + j] : 0;
          mine_w += w[j];
        }
        uint64_t upto = mine_w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t y = shfl_up(upto, o);
          if (lane >= o) upto += y;
        }
        const uint64_t total = __shfl_sync(0xffffffffu, upto, 31);
        const uint64_t at = static_cast<uint64_t>(static_cast<double>(u) * static_cast<double>(total));
        uint64_t c = upto - mine_w;
        if (c <= at && at < upto) {  // (one lane)
          int j = 0;
#pragma unroll
          for (int i = 0; i + 1 < EACH; ++i)
            if (at >= c + w[i] && j == i) c += w[i], ++j;
          const uint64_t entry = sh.quick.list[lane * EACH + j];
          a.tokens[row] = static_cast<int32_t>(entry);
          if (a.logprob) a.logprob[row] = set.log_of(K::value_of(static_cast<uint32_t>(entry >> 32)), m, others_of(total, scale->drop));
          if (a.kept) a.kept[row] = static_cast<int32_t>(keep);
        }
      };
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
          if (key >= cut_key) w += one_weight(K::value_of(key));
        }
        uint64_t c = scan(w, all_w);
        if (c <= at && at < c + w) {  // (one thread)
          for (uint32_t j = j0; j < j1; ++j) {
            const uint64_t entry = sh.quick.list[j];
            const uint32_t key = static_cast<uint32_t>(entry >> 32);
            if (key < cut_key) continue;
            const float x = K::value_of(key);
            c += one_weight(x);
            if (c > at) {
              a.tokens[row] = static_cast<int32_t>(entry);
              if (a.logprob) a.logprob[row] = set.log_of(x, m, others_of(total, scale->drop));
              if (a.kept) a.kept[row] = static_cast<int32_t>(keep);
              break;
            }
          }
        }
      };
      if (rank == 0) {
        // the warps' lists one behind the other
        const uint32_t c = tid < n * kWarps ? sh.quick.many[tid] : 0;
        const bool wide = __syncthreads_or(c > kOwn);
        uint64_t all;
        const uint32_t to = static_cast<uint32_t>(scan(c, all));
        uint32_t verdict = kDigits;
        if (!wide && all <= kList) {
          size = static_cast<uint32_t>(all);
          few = size <= kFew;
          for (uint32_t j = 0; j < c; ++j) {
            const uint64_t* from = &sh.quick.own[tid % kWarps][j];
            sh.quick.list[to + j] = tid < kWarps ? *from : ld_cluster64(mapa_shared(smem_u32(from), tid / kWarps));
          }
          __syncthreads();
        }
        double s_lo = 0.0, s_hi = 0.0;
        if (by_p && !by_k && a.vocab > kShort) {
          // (the FP32 weights are relative to 2^(m c + k))
          const double whole = static_cast<double>(quick_total) / static_cast<double>(one) * static_cast<double>(exp2f(a.drop - scale->drop));
          const double off = whole * static_cast<double>(error_of(quick_total, 13.f));
          s_lo = whole - off, s_hi = whole + off;
        }
        if (size > 0 && few) {
          if (tid < size) sh.quick.upto[tid] = weight(K::value_of(static_cast<uint32_t>(sh.quick.list[tid] >> 32)), *scale, sh.table);
          __syncthreads();
          uint64_t every = 0;
          if (size > kThreads / 4) each = 2;
          me = tid / each;
          if (me < size) my_key = static_cast<uint32_t>(sh.quick.list[me] >> 32), my_w = sh.quick.upto[me];
          for (uint32_t j = tid % each; j < size; j += each) {
            const uint32_t key = static_cast<uint32_t>(sh.quick.list[j] >> 32);
            const uint64_t w = sh.quick.upto[j];
            every += w;
            if (key > my_key) above += w, ++larger;
          }
#pragma unroll
          for (uint32_t o = 1; o < 4; o <<= 1) {
            if (o >= each) break;
            above += __shfl_xor_sync(0xffffffffu, above, o);
            every += __shfl_xor_sync(0xffffffffu, every, o);
            larger += __shfl_xor_sync(0xffffffffu, larger, o);
          }
          __syncthreads();  // the weights have been read
          if (by_p && !by_k && a.vocab <= kShort) s_lo = s_hi = static_cast<double>(every);
          verdict = decide_few(s_lo, s_hi) ? kDone : kExactSum;
          if (verdict == kDone) draw_few();
        } else if (size > 0) {
          for (uint32_t i = tid; i < size; i += kThreads) sh.quick.sorted[i] = (sh.quick.list[i] & 0xffffffff00000000ull) | i;
          uint32_t full = kFew;
          while (full < size) full *= 2;
          for (uint32_t i = size + tid; i < full; i += kThreads) sh.quick.sorted[i] = 0;
          __syncthreads();
          // A bitonic sort, largest first.  A warp has 64 neighbours in registers, so that only steps of 64 and more go through
          // shared memory.
          const uint32_t x0 = warp * 64 + lane;
          for (uint32_t span = 64; span <= full; span *= 2) {
            for (uint32_t step = span / 2; step >= 64; step /= 2) {
              for (uint32_t i = tid; i < full / 2; i += kThreads) {
                const uint32_t x = 2 * i - (i & (step - 1)), y = x + step;
                const uint64_t f = sh.quick.sorted[x], g = sh.quick.sorted[y];
                if ((f < g) == ((x & span) == 0)) sh.quick.sorted[x] = g, sh.quick.sorted[y] = f;
              }
              __syncthreads();
            }
            if (warp * 64 < full) {
              uint64_t x[2] = {sh.quick.sorted[x0], sh.quick.sorted[x0 + 32]};
              for (uint32_t inner = span == 64 ? 2 : span;; inner = inner < 64 ? inner * 2 : 128) {  // (the first time all spans up to 64)
                if (inner >= 64) {
                  if ((x[0] < x[1]) == ((x0 & inner) == 0)) {
                    const uint64_t t = x[0];
                    x[0] = x[1], x[1] = t;
                  }
                }
#pragma unroll 1
                for (uint32_t step = min(inner / 2, 16u); step; step /= 2)
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    const uint64_t y = __shfl_xor_sync(0xffffffffu, x[h], step);
                    const bool larger_here = ((lane & step) == 0) == (((x0 + 32 * h) & inner) == 0);
                    x[h] = larger_here == (x[h] > y) ? x[h] : y;
                  }
                if (inner >= 64) break;
              }
              sh.quick.sorted[x0] = x[0], sh.quick.sorted[x0 + 32] = x[1];
            }
            __syncthreads();
          }
          // exact weights before each
          const uint32_t per = (size + kThreads - 1) / kThreads;
          const uint32_t j0 = min(tid * per, size), j1 = min(j0 + per, size);
          uint64_t w = 0;
          for (uint32_t j = j0; j < j1; ++j) {
            const uint64_t x = one_weight(K::value_of(static_cast<uint32_t>(sh.quick.sorted[j] >> 32)));
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
          if (by_p && !by_k && a.vocab <= kShort) s_lo = s_hi = static_cast<double>(kept_w);
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
          if (few) {
            decide_few(whole, whole);
            draw_few();
          } else {
            decide(whole, whole);
            draw();
          }
        }
        return;
      }
    }
  }
  // ---- digit by digit, and sums of all that is kept
  // The lowest key kept among [lo, hi]: the one down to which the tokens from `base` on weigh p of them all or more (in
  // numbers: down to which there are `number` of them), found range by range.  `sure`: the last range in which it lies whatever
  // the errors of the weights; true if it is the last.
  auto search = [&](uint32_t base, uint32_t lo, uint32_t hi, bool numbers, uint64_t number, bool exact, Found& sure) {
    Found f{lo, hi, 0, 0, 1};
    for (int round = 0;; ++round) {  // (eleven bits a round)
      const int shift = max(21 - __clz((f.hi - f.lo) | 1), 0);
      for (int i = tid; i < kBins; i += kThreads) sh.digits.lo[i] = sh.digits.hi[i] = 0;
      __syncthreads();
      uint64_t above = 0, rest = 0;  // (the first time)
      const uint32_t first_key = round ? f.lo : base, last_key = round ? f.hi : most;
#pragma unroll 1
      for (int i = t0; i < t1; ++i) {
        const uint32_t b = bits_at(i), key = K::of(b);
        if (key < first_key || key > last_key) continue;
        const uint64_t w = numbers ? 1 : exact ? one_weight(K::value(b)) : quick_weight(K::value(b));
        if (key > f.hi) {
          above += w;
        } else if (key < f.lo) {
          rest += w;
        } else {
          const int bin = (f.hi - key) >> shift;
          const uint32_t w_lo = static_cast<uint32_t>(w), old = atomicAdd(&sh.digits.lo[bin], w_lo);
          const uint32_t w_hi = static_cast<uint32_t>(w >> 32) + (old + w_lo < old ? 1u : 0u);
          if (w_hi) atomicAdd(&sh.digits.hi[bin], w_hi);
        }
      }
      uint64_t all;
      if (round == 0) {
        scan(above, all);
        if (tid == 0) n == 1 ? void(sh.cta_above[0] = all) : st_cluster(mapa_shared(smem_u32(&sh.cta_above[rank]), 0), all);
        scan(rest, all);
        if (tid == 0) n == 1 ? void(sh.cta_rest[0] = all) : st_cluster(mapa_shared(smem_u32(&sh.cta_rest[rank]), 0), all);
      }
      cluster_sync(n);
      // each CTA adds up a share of the bins over all CTAs, for the first one
      const int share = (kBins + n - 1) / n, last = min((rank + 1) * share, kBins);
      for (int bin = rank * share + tid; bin < last; bin += kThreads) {
        if (n == 1) {
          sh.digits.all[bin] = static_cast<uint64_t>(sh.digits.hi[bin]) << 32 | sh.digits.lo[bin];
        } else {
          const uint64_t w = (cluster_sum(&sh.digits.hi[bin], n) << 32) + cluster_sum(&sh.digits.lo[bin], n);
          st_cluster(mapa_shared(smem_u32(&sh.digits.all[bin]), 0), w);
        }
      }
      cluster_sync(n);
      if (rank == 0) {
        // sums down to each bin, four a thread
        constexpr int B = kBins / kThreads;
        uint64_t w[B], sum = 0;
#pragma unroll
        for (int j = 0; j < B; ++j) sum += w[j] = sh.digits.all[tid * B + j];
        uint64_t upto = scan(sum, all);
        if (round == 0) {
          f.whole = all;
          for (int r = 0; r < n; ++r) f.above += sh.cta_above[r], f.whole += sh.cta_above[r] + sh.cta_rest[r];
          // (FP64 is slow: in one thread)
          if (tid == 0) sh.target = numbers ? number : static_cast<uint64_t>(ceil(static_cast<double>(p) * static_cast<double>(f.whole)));
          __syncthreads();
        }
        upto += f.above;
        const uint64_t target = sh.target;
#pragma unroll
        for (int j = 0; j < B; ++j) {
          // the range in which the threshold lies: the last one kept
          if (upto < target && upto + w[j] >= target) {
            const uint32_t to = f.hi - (static_cast<uint32_t>(tid * B + j) << shift), width = (1u << shift) - 1;
            const uint64_t off = numbers || exact ? 0 : fixed(static_cast<float>(f.whole) / unit * error_of(f.whole, 4.f));
            sh.found = Found{to - f.lo > width ? to - width : f.lo, to, upto, f.whole, upto + off < target && upto + w[j] >= target + off};
          }
          upto += w[j];
        }
        // (fewer tokens than are asked for: all are kept)
        if (tid == kThreads - 1 && upto < target) sh.found = Found{base, base, 0, f.whole, 1};
        __syncthreads();
        constexpr int WORDS = sizeof(Found) / 8;
        if (tid >= WORDS && tid < n * WORDS) {
          uint64_t* word = reinterpret_cast<uint64_t*>(&sh.found) + tid % WORDS;
          st_cluster(mapa_shared(smem_u32(word), tid / WORDS), *word);
        }
      }
      cluster_sync(n);
      f = sh.found;
      if (f.certain) sure = f;
      if (shift == 0 || f.lo == f.hi || round == 3) return f.certain != 0;
    }
  };

  float weight_of_all = 0.f;  // of the tokens that matter, by FP32 weights (0: not known)
  // The token among those whose key is `cut` or more; false if the FP32 weights leave it open.
  auto draw_from = [&](uint32_t cut, bool exact) {
    auto weight_at = [&](int i) -> uint64_t {
      const uint32_t b = bits_at(i);
      if (K::of(b) < cut) return 0;
      return exact ? one_weight(K::value(b)) : quick_weight(K::value(b));
    };
    uint64_t sum = 0, all, below;
    uint32_t count = 0;
#pragma unroll 1
    for (int i = t0; i < t1; ++i) {
      sum += weight_at(i);
      count += K::of(bits_at(i)) >= cut;
    }
    count = __reduce_add_sync(0xffffffffu, count);
    uint64_t before = scan(sum, all);
    if (lane == 0) sh.warp_n[warp] = count;
    if (tid == 0) sh.where = -1;
    __syncthreads();
    count = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.warp_n[lane] : 0u);
    const uint64_t total = exchange(all, count, below);
    if (!exact) weight_of_all = static_cast<float>(total) / unit / one;
    if (exact && u < kSmallNumber) {
      if (rank == 0) draw_small<TYPE>(a, row, cut, m, total, scale->drop, count, reinterpret_cast<double*>(sh.warp_w));
      return true;
    }
    const uint64_t at = static_cast<uint64_t>(static_cast<double>(u) * static_cast<double>(total));
    const uint64_t off = exact ? 0 : fixed(static_cast<float>(total) / unit * error_of(total, 4.f));
    before += below;
    if (before <= at && at < before + sum) sh.where = t0, sh.from = before;  // (one thread of the cluster)
    __syncthreads();
    if (warp == 0 && sh.where >= 0) {
      uint64_t from = sh.from;
      const int end = min(sh.where + per_thread, mine * VEC);
      for (int i0 = sh.where; i0 < end; i0 += 32) {
        const int i = i0 + lane;
        const uint64_t w = i < end ? weight_at(i) : 0;
        uint64_t upto = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t y = shfl_up(upto, o);
          if (lane >= o) upto += y;
        }
        upto += from;
        const unsigned past = __ballot_sync(0xffffffffu, upto > at);
        if (past) {
          // (further from both of its borders than the FP32 sums may be off)
          if (lane == __ffs(past) - 1 && upto - w + off <= at && upto > at + off) {
            a.tokens[row] = first * VEC + i - skip;
            if (a.kept) a.kept[row] = static_cast<int32_t>(count);
            if (a.logprob) {
              const uint64_t top_w = exact ? 1ull << (kFixed - scale->drop) : quick_weight(m);
              a.logprob[row] = set.log_of(K::value(bits_at(i)), m, static_cast<float>(total > top_w ? total - top_w : 0) / static_cast<float>(top_w));
            }
            if (!exact) tell_verdict(kDone);
          }
          break;
        }
        from = __shfl_sync(0xffffffffu, upto, 31);
      }
      __syncwarp();
    }
    if (exact) return true;
    cluster_sync(n);
    return sh.verdict == kDone;
  };

  if (by_k) {
    Found f;
    search(K::LOWEST, from_key, most, true, k_asked, true, f);
    from_key = f.lo;
  }
  uint32_t cut = max(least, by_k ? from_key : K::LOWEST);
  // By FP32 weights first, and by exact ones what they leave open.
  Found sure{from_key, max(to_key, from_key), 0, 0, 1};
  bool known = !by_p;
  if (by_p && !(p > 0.f)) cut = most, known = true;
  auto exact_from_here = [&]() {
    if (!(weight_of_all > 0.f)) {  // not known: by the fewest places first
      __syncthreads();
      if (tid == 0) sh.scale.drop = a.drop;
      __syncthreads();
      weight_of_all = static_cast<float>(exact_sum()) * exp2f(static_cast<float>(a.drop - kFixed));
    }
    __syncthreads();
    if (tid == 0) sh.scale.drop = drop_of(weight_of_all, a.drop);
    __syncthreads();
  };
  for (bool exact = !in_range; !known; exact = true) {
    if (exact) exact_from_here();
    known = search(by_k ? from_key : K::LOWEST, sure.lo, sure.hi, false, 0, exact, sure) || exact;
    if (!exact) weight_of_all = static_cast<float>(sure.whole) / unit / one;
  }
  if (by_p && p > 0.f) cut = max(cut, sure.lo);
  if (in_range && u >= kSmallNumber && draw_from(cut, false)) return;
  exact_from_here();
  draw_from(cut, true);
}

// CTAs per row: as many as its bytes need for two CTAs on an SM, more until every SM has one or a CTA has
// little left.  (A row takes its CTAs 12 to 15 us, of which its bytes are on their way for 3 to 5.  256 rows of 151936 FP16 values,
// the 50 largest of each, calls in a row: 63 us with two CTAs of 512 threads, 66 with four of 256, which are better with cold
// caches, 62 to 69, and for 128 FP32 rows of 100003, 88 to 91, but worse for a block of 8 rows, 34 to 28.)
constexpr int kSmemOfSm = 228 * 1024;
cudaError_t splits_of(int n_rows, long long row_pieces, int* splits, int* pieces) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  constexpr long long fits = (kSmemOfSm / kPerSm - 1024 - kSharedBytes) / 16;
  long long s = (row_pieces + fits - 1) / fits;
  if (s > kMaxSplits) s = kMaxSplits;
  while (2 * s <= kMaxSplits && n_rows * s < sms && row_pieces > 2 * kThreads * s) s *= 2;
  *splits = static_cast<int>(s);
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
  if (!top_k && !top_p && !min_p) return cuda_status(launch_sample_plain(a, type, st), "sample tokens");
  const int vec = 16 / size;
  const long long row_pieces = (vocab + vec - 1) / vec + 1;  // (a row may begin inside a piece)
  cudaError_t e = splits_of(n_rows, row_pieces, &a.splits, &a.pieces);
  if (e != cudaSuccess) return cuda_status(e, "sample tokens");
  e = type == DFLASH_T_FP32 ? launch<DFLASH_T_FP32>(a, st)
      : type == DFLASH_T_BF16 ? launch<DFLASH_T_BF16>(a, st)
                              : launch<DFLASH_T_FP16>(a, st);
  return cuda_status(e, "sample tokens");
}

}  // extern "C"
