// Tokens drawn from the whole distribution, and greedy ones: dflash_sample_tokens without a filter.
//
// One pass over the logits.  A warp takes a batch of 2 KB at a time from its ring of bulk copies and leaves
// its sum of 2^((x - r) c) with the reference r, the largest value the warp has met; the
// batches' sums, brought to one reference, lead to the batch in which u lies, which is
// read once more.  The token stands if both of its borders are further from u than these sums
// may be off (for u below 2^-24 none is); else the row is left to a second kernel, which forms exact sums with clusters of
// eight CTAs (one CTA alone takes 70 us for 151936 tokens, the tail of a call of 1000 rows).  A greedy row is one look: the
// first batch whose reference is the largest value holds its first id.
//
// The bound, in units of 2^-24 of the row's sum S: a weight is 2^(x c + k) 2^d, where k = -r c as FP32 has it for the batch's reference r and
// d = k_m - k brings it to the row's; what the row's own k is off by is the same for all weights.  Of the exponent Y = (x - m) c the constant c is off by
// |Y| at most (one rounding), and x c + k and d, which are Y together, by one rounding each, |Y| in all: with ln 2, 1.39 |Y|.  The mean of |Y| over the
// weights is their entropy less log2 S, log2(vocab / S) at most.  Then 2^y 4, a piece's sum 3, the batch's 7, its factor 5, a CTA's number 6: 25.
// The border of a token, which lies about u S, and u S are sums of the same numbers, so that a weight's error counts 1 - u times before the border and u
// times behind it: 1.39 log2(vocab / S) + 25 / 2.  Only in the batch in which u lies are pieces and single weights not what S was made of: 12 more for the
// batch's sum, its product and a piece's sum.  Together below 28 + 1.4 log2(vocab / S).
//
// Few rows: a row's batches are split over the CTAs of a cluster.
//
// Measured, calls in a row: 1000 rows of 151936 BF16 values 88 to 91 us (floor 45), greedy ones 74.  The first kernel takes 58 to 60 (5.1 TB/s, issue
// slots at 70 %: an exponential and seven instructions a value), the second 25 to 30 for the 15 or so rows left to it: a claim, 16 us of exact
// weights, the search for the token.
#include <cstddef>

#include "sampling.cuh"

namespace dflash {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kLoads = 4;  // 16-byte loads of a thread per batch
constexpr int kBatchBytes = 32 * kLoads * 16;
constexpr int kStages = 2;  // batches of a warp on their way
constexpr int kRingBytes = kWarps * kStages * kBatchBytes;
constexpr int kRestCtas = 8;         // CTAs for a row that the FP32 sums leave open
constexpr int32_t kClaimed = -2, kUndecided = -3;  // the token of such a row, between the kernels: kUndecided less the places (plus 16) that its weights have less
constexpr int kRestWarps = 8, kRestThreads = 32 * kRestWarps, kRestLoads = 2;  // of its CTAs
constexpr int kMaxBatches = (1 << 19) * 4 / kBatchBytes + 1;  // (a row may begin inside a piece)

// The largest of the warp's values (no NaN among them).
__device__ __forceinline__ float warp_max(float v) { return float_from_order_key(__reduce_max_sync(0xffffffffu, float_order_key(v))); }

// Inclusive sums over the lanes.
template <typename T>
__device__ __forceinline__ T warp_upto(T v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// A lane's pieces of a batch of a row.
template <int TYPE, int LOADS>
__device__ __forceinline__ void load_batch(const uint8_t* src, const uint4* frame, int skip, int places, int vocab, int b, int lane,
                                           uint4 (&v)[LOADS]) {
  using E = Elem<TYPE>;
  constexpr int VEC = E::VEC, BATCH = 32 * LOADS * VEC;
  const int p0 = b * BATCH;
  if (p0 >= skip && p0 + BATCH <= places) {
#pragma unroll
    for (int j = 0; j < LOADS; ++j) v[j] = __ldg(frame + p0 / VEC + j * 32 + lane);
  } else {  // the row's ends: value by value
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const long long i = p0 + (j * 32 + lane) * VEC - skip;
      constexpr int W = VEC / 4;  // values of a word
      v[j].x = E::raw(src, i, vocab);
      v[j].y = E::raw(src, i + W, vocab);
      v[j].z = E::raw(src, i + 2 * W, vocab);
      v[j].w = E::raw(src, i + 3 * W, vocab);
    }
  }
}

// An FP32 sum of weights in units of 2^-40, in which sums of sums are exact.
__device__ __forceinline__ uint64_t units(float x) { return static_cast<uint64_t>(__float2ull_rn(x * 0x1p40f)); }

template <int TYPE>
__global__ void __launch_bounds__(kThreads, 4) sample_plain_kernel(const SampleArgs a) {
  using E = Elem<TYPE>;
  using K = Keys<TYPE>;
  constexpr int VEC = E::VEC, BATCH = 32 * kLoads * VEC;
  extern __shared__ __align__(128) uint8_t ring[];  // [kWarps][kStages] batches
  __shared__ float2 part[kMaxBatches];  // reference and sum of this CTA's batches
  __shared__ uint64_t full[kWarps][kStages];
  __shared__ Scale s_scale;
  __shared__ float s_ref[kWarps];
  __shared__ uint64_t s_sum[kWarps];
  __shared__ uint32_t s_count[kWarps], s_nan[kWarps];
  __shared__ float cta_ref[kMaxSplits], cta_sum[kMaxSplits];
  __shared__ uint32_t cta_count[kMaxSplits], cta_nan[kMaxSplits];
  __shared__ int s_batch, s_done;
  __shared__ uint64_t s_from;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = blockIdx.x / a.splits, rank = blockIdx.x - row * a.splits, n = a.splits;
  if (n > 1) cluster_arrive_relaxed();
  pdl_launch_dependents();

  const uint8_t* src = a.logits + row * a.row_bytes;
  const int skip = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15) / E::BYTES;
  const uint4* frame = reinterpret_cast<const uint4*>(src - skip * E::BYTES);
  const int places = a.vocab + skip;
  const int batches = (places + BATCH - 1) / BATCH;
  // this CTA's batches
  const int b0 = static_cast<int>(static_cast<long long>(batches) * rank / n), b1 = static_cast<int>(static_cast<long long>(batches) * (rank + 1) / n);
  auto load = [&](int b, uint4 (&v)[kLoads]) { load_batch<TYPE, kLoads>(src, frame, skip, places, a.vocab, b, lane, v); };
  // whole batches come through the warp's ring by bulk copies, those at the row's ends by loads
  auto inside = [&](int b) { return b * BATCH >= skip && b * BATCH + BATCH <= places; };
  uint8_t* mine_ring = ring + warp * kStages * kBatchBytes;
  auto copy = [&](int b, int st) {  // (one lane)
    mbar_arrive_expect_tx(&full[warp][st], kBatchBytes);
    bulk_g2s(mine_ring + st * kBatchBytes, frame + static_cast<size_t>(b) * (kBatchBytes / 16), kBatchBytes, &full[warp][st]);
  };
  if (lane == 0) {
    for (int st = 0; st < kStages; ++st) mbar_init(&full[warp][st], 1);
    fence_barrier_init();
    for (int st = 0; st < kStages; ++st) {
      const int b = b0 + warp + st * kWarps;
      if (b < b1 && inside(b)) copy(b, st);
    }
  }
  __syncwarp();
  const Settings set(a, row);
  if (tid == kThreads - 1) {
    if (rank == 0 && !set.fine) set_status(a.status, DFLASH_DEV_BAD_VALUE);
    s_scale.hi = 1.f;
    if (!set.greedy) set.scale(s_scale, a.drop);
    s_batch = 0x7fffffff;
    s_done = 0;
  }
  __syncthreads();  // (c)
  const float c = s_scale.hi;
  // what a reference adds to an exponent; one so low (masked values) that nothing has weight beside any other: 0
  auto none = [&](float r) { return !(r * c > -0x1p21f); };
  auto start = [&](float r) { return none(r) ? 0.f : -(r * c); };

  // ---- the pass
  float ref = -INFINITY;
  uint32_t count = 0, tops = E::NOTHING;
  bool ok = true;
  {
    int st = 0;
    uint32_t phases = 0;  // bit st: parity of the stage's next copy
    for (int b = b0 + warp; b < b1; b += kWarps, st = st + 1 == kStages ? 0 : st + 1) {
      uint4 v[kLoads];
      if (inside(b)) {
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&full[warp][st], phases >> st & 1));
        phases ^= 1u << st;
        const uint4* from = reinterpret_cast<const uint4*>(mine_ring + st * kBatchBytes);
#pragma unroll
        for (int j = 0; j < kLoads; ++j) v[j] = from[j * 32 + lane];
        __syncwarp();
      } else {
        load(b, v);
      }
      const int next = b + kStages * kWarps;
      // (the lanes' reads of the stage are done: their values are in registers)
      if (ok && lane == 0 && next < b1 && inside(next)) copy(next, st);
      uint32_t top = E::NOTHING, low = v[0].x;
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        top = K::max_nan(top, K::max_nan(K::max_nan(v[j].x, v[j].y), K::max_nan(v[j].z, v[j].w)));
        low = K::min_words(low, K::min_words(K::min_words(v[j].x, v[j].y), K::min_words(v[j].z, v[j].w)));
      }
      tops = K::max_nan(tops, top);
      ref = fmaxf(ref, warp_max(fmaxf(E::max_of(top), -INFINITY)));
      float sum = 0.f;
      if (!set.greedy) {
        const float k = start(ref);
        float s[kLoads];
#pragma unroll
        for (int j = 0; j < kLoads; ++j) s[j] = K::quick_sum_from(v[j], c, k);
        sum = (s[0] + s[1]) + (s[2] + s[3]);
        if (__any_sync(0xffffffffu, K::masked(low))) {
#pragma unroll
          for (int j = 0; j < kLoads; ++j) count += K::unmasked(v[j]);
        } else {
          count += kLoads * VEC;
        }
      }
      static_assert(kLoads == 4, "sum");
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) part[b - b0] = make_float2(ref, sum);
    }
    if (!ok) {
      // a copy did not come in time: none is issued any more, and what is in flight lands before the CTA ends
      for (int i = 0; i < kStages; ++i) mbar_wait(&full[warp][i], phases >> i & 1);
      if (lane == 0) set_status(a.status, DFLASH_DEV_TIMEOUT);
    }
  }
  count = __reduce_add_sync(0xffffffffu, count);
  const bool nan = __any_sync(0xffffffffu, K::has_nan(tops));
  if (lane == 0) s_ref[warp] = ref, s_count[warp] = count, s_nan[warp] = nan;
  __syncthreads();
  float m = -INFINITY;
  uint32_t all = 0, bad = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_ref[w]), all += s_count[w], bad |= s_nan[w];
  const int mine = b1 - b0, per = (mine + kThreads - 1) / kThreads;
  const int j0 = min(tid * per, mine), j1 = min(j0 + per, mine);  // the thread's batches, one behind the other
  auto of_batch = [&](int j) {  // relative to m as it is by then
    const float2 x = part[j];
    return none(x.x) ? 0 : units(x.y * ex2_approx(start(m) - start(x.x)));
  };
  uint64_t own, before, cta;  // of the thread's batches, of those before them, of the CTA's
  auto add_up = [&]() {
    own = 0;
    for (int j = j0; j < j1; ++j) own += of_batch(j);
    const uint64_t upto = warp_upto(own, lane);
    if (lane == 31) s_sum[warp] = upto;
    __syncthreads();
    before = upto - own, cta = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s_sum[w];
      cta += s_sum[w];
    }
  };
  add_up();
  // ---- the CTAs' results
  uint64_t total = cta, below = 0;
  bool owner = true;
  if (n > 1) {
    cluster_wait();  // every CTA has started
    if (tid < n) {
      auto put = [&](void* to, uint32_t v) {
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(to), tid)), "r"(v) : "memory");
      };
      put(&cta_ref[rank], __float_as_uint(m));
      put(&cta_sum[rank], __float_as_uint(static_cast<float>(cta) * 0x1p-40f));
      put(&cta_count[rank], all);
      put(&cta_nan[rank], bad);
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    const float m_own = m;
    all = bad = 0;
    for (int r = 0; r < n; ++r) m = fmaxf(m, cta_ref[r]), all += cta_count[r], bad |= cta_nan[r];
    auto of_cta = [&](int r) { return none(cta_ref[r]) ? 0 : units(cta_sum[r] * ex2_approx(start(m) - start(cta_ref[r]))); };
    total = 0;
    uint64_t share = 0;
    for (int r = 0; r < n; ++r) {
      const uint64_t x = of_cta(r);
      total += x;
      if (r == rank) share = x;
    }
    // the one CTA that goes on: the first whose sums pass u, or that has the largest value
    const uint64_t at = static_cast<uint64_t>(static_cast<double>(set.u) * static_cast<double>(total));
    int who = 0;
    for (; who < n - 1; ++who) {
      if (set.greedy) {
        if (cta_ref[who] == m) break;
        continue;
      }
      const uint64_t x = of_cta(who);
      if (at < below + x) break;
      below += x;
    }
    owner = who == rank;
    if (owner && !set.greedy) {
      if (m != m_own) add_up();
      total += cta - share;  // (of the numbers that the borders are made of)
    }
  }
  if (bad || !(m < INFINITY) || m == -INFINITY) {  // not finite, or nothing to draw from
    if (rank == 0 && tid == 0) {
      if (bad || m != -INFINITY) set_status(a.status, DFLASH_DEV_NONFINITE);
      a.tokens[row] = -1;
      if (a.logprob) a.logprob[row] = -INFINITY;
      if (a.kept) a.kept[row] = 0;
    }
    return;
  }
  if (!owner) return;

  if (set.greedy) {
    for (int j = j0; j < j1; ++j)
      if (part[j].x == m) {
        atomicMin(&s_batch, j);
        break;
      }
    __syncthreads();
    if (warp == 0) {
      uint4 v[kLoads];
      const int b = b0 + s_batch;
      load(b, v);
      uint32_t id = 0xffffffffu;
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (K::value(K::bits(v[j], e)) == m) id = min(id, static_cast<uint32_t>(b * BATCH + (j * 32 + lane) * VEC + e - skip));
      id = __reduce_min_sync(0xffffffffu, id);
      if (lane == 0) {
        a.tokens[row] = static_cast<int32_t>(id);
        if (a.logprob) a.logprob[row] = 0.f;
        if (a.kept) a.kept[row] = 1;
      }
    }
    return;
  }

  // ---- the batch in which u lies, and the token in it
  const uint64_t at = static_cast<uint64_t>(static_cast<double>(set.u) * static_cast<double>(total));
  const float k = start(m);
  const float whole = static_cast<float>(total) * 0x1p-40f;
  const uint64_t off = units(whole * 0x1p-24f * (28.f + 1.4f * log2f(static_cast<float>(a.vocab) / whole)));
  // (k is off by 2^-4 at most, and what `none` leaves out is far below the largest value; else no border is far enough)
  const bool close = !(fabsf(m) * c < 0x1p20f);
  before += below;
  if (!close && before <= at && at < before + own) {  // (one thread, or none where the CTAs' sums differ: then the exact ones decide)
    uint64_t x = before;
    int j = j0;
    for (; j < j1 - 1; ++j) {
      const uint64_t y = of_batch(j);
      if (at < x + y) break;
      x += y;
    }
    s_batch = j;
    s_from = x;
  }
  __syncthreads();
  if (warp == 0 && s_batch != 0x7fffffff) {
    uint4 v[kLoads];
    const int b = b0 + s_batch;
    load(b, v);
    const float k_r = start(part[s_batch].x), factor = ex2_approx(k - k_r);  // as in the batch's sum
    uint64_t from = s_from;
    bool found = false;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const uint64_t w = units(K::quick_sum_from(v[j], c, k_r) * factor);
      const uint64_t x = warp_upto(w, lane) + from;
      const unsigned over = __ballot_sync(0xffffffffu, x > at);
      if (!found && over && lane == __ffs(over) - 1) {
        uint64_t y = x - w;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float value = K::value(K::bits(v[j], e));
          const uint64_t low = y;
          y += units(ex2_approx(fmaf(value, c, k_r)) * factor);
          // the first past u, further from both of its borders than the sums may be off
          if (low <= at && y > at && low + off <= at && y > at + off) {
            a.tokens[row] = b * BATCH + (j * 32 + lane) * VEC + e - skip;
            if (a.logprob) {  // (in these sums the largest weight is 2^(m c + k), about 1)
              const float most = ex2_approx(fmaf(m, c, k));
              const uint64_t w = units(most);
              a.logprob[row] = set.log_of(value, m, static_cast<float>(total > w ? total - w : 0) * 0x1p-40f / most);
            }
            if (a.kept) a.kept[row] = static_cast<int32_t>(all);
            s_done = 1;
          }
        }
      }
      found |= over != 0;
      from = __shfl_sync(0xffffffffu, x, 31);
    }
  }
  __syncthreads();
  if (!s_done && tid == 0) {
    a.tokens[row] = kUndecided - 16 - (close ? a.drop + 1 : drop_of(whole / ex2_approx(fmaf(m, c, k)), a.drop));
    // (what the second kernel need not find again, where there is a place for it)
    if (a.logprob && a.kept) a.logprob[row] = m, a.kept[row] = static_cast<int32_t>(all);
  }
}

// Rows that the sums left open: exact ones, by clusters of kRestCtas.  A CTA has a part of the row's batches, which it reads for
// the weights, and before that for the largest value and the tokens that are not masked, where the first kernel had no place to
// leave these.  (Batches of half the first kernel's size with loads ahead 91 us for 1000 rows, 93 without; CTAs of 512 threads, for which an SM
// has to be empty, 104.)
template <int TYPE>
__global__ void __launch_bounds__(kRestThreads, 2) sample_rest_kernel(const __grid_constant__ SampleArgs a) {
  using E = Elem<TYPE>;
  using K = Keys<TYPE>;
  constexpr int VEC = E::VEC, BATCH = 32 * kRestLoads * VEC;  // (not the first kernel's batches)
  __shared__ uint64_t part[(1 << 19) * 4 / (512 * kRestLoads) / kRestCtas + 2];  // of this CTA's batches
  __shared__ TableEntry table[32];
  __shared__ Scale s_scale;
  __shared__ uint64_t s_wide[kRestWarps], cta_wide[kRestCtas];
  __shared__ uint32_t s_key[kRestWarps], s_count[kRestWarps], cta_key[kRestCtas], cta_count[kRestCtas], s_open[4 * kRestWarps];
  __shared__ int s_batch, s_row, s_drop, s_told, s_told_drop;
  __shared__ uint64_t s_from;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x % kRestCtas, cluster = blockIdx.x / kRestCtas, clusters = gridDim.x / kRestCtas;
  if (tid < 32) table[tid] = kTable[tid];
  auto sync = [] {
    __syncwarp();  // (the barrier wants its warp's lanes together)
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  };
  auto put = [](void* to, uint32_t v, int r) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(to), r)), "r"(v) : "memory");
  };
  sync();  // every CTA runs before another writes to it
  pdl_wait();
  // The clusters begin at different rows, and a row belongs to the one that changes its mark.
  constexpr int LOOK = 4;  // rows of a thread at a time
  const int chunks = (a.n_rows + LOOK * kRestThreads - 1) / (LOOK * kRestThreads);
  int chunk = static_cast<int>(static_cast<long long>(chunks) * cluster / clusters), seen = 0;
  for (;;) {
    if (rank == 0) {
      int row = -1;
      while (seen < chunks && row < 0) {
        unsigned open[LOOK];
#pragma unroll
        for (int i = 0; i < LOOK; ++i) {
          const int mine = (chunk * LOOK + i) * kRestThreads + tid;
          open[i] = __ballot_sync(0xffffffffu, mine < a.n_rows && __ldcg(a.tokens + mine) <= kUndecided);
        }
        __syncthreads();  // s_row and s_open of the last round have been read
        if (lane < LOOK) s_open[lane * kRestWarps + warp] = lane == 0 ? open[0] : lane == 1 ? open[1] : lane == 2 ? open[2] : open[3];
        if (tid == 0) s_row = -1;
        __syncthreads();
        if (tid == 0) {
          for (int i = 0; i < LOOK * kRestWarps && s_row < 0; ++i) {
            const int w = (i + cluster) % (LOOK * kRestWarps);
            for (unsigned left = s_open[w]; left && s_row < 0; left &= left - 1) {
              const int r = chunk * LOOK * kRestThreads + w * 32 + __ffs(left) - 1;
              const int32_t mark = __ldcg(a.tokens + r);
              if (mark <= kUndecided && atomicCAS(a.tokens + r, mark, kClaimed) == mark) s_row = r, s_drop = kUndecided - 16 - mark;
            }
          }
        }
        __syncthreads();
        row = s_row;
        if (row < 0) {
          ++seen;
          chunk = chunk + 1 == chunks ? 0 : chunk + 1;
        }
      }
      if (tid < kRestCtas) put(&s_told, static_cast<uint32_t>(row), tid), put(&s_told_drop, static_cast<uint32_t>(s_drop), tid);
      __syncwarp();
    }
    sync();
    const int row = s_told;
    int drop = s_told_drop;  // more than a.drop: not known
    if (row < 0) return;
    {
        const Settings set(a, row);
        if (tid == 0) set.scale(s_scale, min(drop, a.drop));
        const uint8_t* src = a.logits + row * a.row_bytes;
        const int skip = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15) / E::BYTES;
        const uint4* frame = reinterpret_cast<const uint4*>(src - skip * E::BYTES);
        const int places = a.vocab + skip;
        const int batches = (places + BATCH - 1) / BATCH;
        const int b0 = batches * rank / kRestCtas, b1 = batches * (rank + 1) / kRestCtas;
        auto load = [&](int b, uint4 (&v)[kRestLoads]) { load_batch<TYPE, kRestLoads>(src, frame, skip, places, a.vocab, b, lane, v); };
        float m;
        uint32_t all;
        if (a.logprob && a.kept) {  // left there by the first kernel
          m = __ldcg(a.logprob + row), all = static_cast<uint32_t>(__ldcg(a.kept + row));
        } else {
          uint32_t tops = E::NOTHING, count = 0;
          for (int b = b0 + warp; b < b1; b += kRestWarps) {
            uint4 v[kRestLoads];
            load(b, v);
#pragma unroll
            for (int j = 0; j < kRestLoads; ++j) {
              tops = E::max_words(tops, E::max_words(E::max_words(v[j].x, v[j].y), E::max_words(v[j].z, v[j].w)));
              count += K::unmasked(v[j]);
            }
          }
          const uint32_t key = __reduce_max_sync(0xffffffffu, float_order_key(E::max_of(tops)));
          count = __reduce_add_sync(0xffffffffu, count);
          if (lane == 0) s_key[warp] = key, s_count[warp] = count;
          __syncthreads();
          if (tid < kRestCtas) {
            uint32_t x = 0, y = 0;
#pragma unroll
            for (int i = 0; i < kRestWarps; ++i) x = max(x, s_key[i]), y += s_count[i];
            put(&cta_key[rank], x, tid);
            put(&cta_count[rank], y, tid);
          }
          __syncwarp();
          sync();
          uint32_t top = 0;
          all = 0;
#pragma unroll
          for (int r = 0; r < kRestCtas; ++r) top = max(top, cta_key[r]), all += cta_count[r];
          m = float_from_order_key(top);
        }
        if (tid == 0) s_scale.m = m;
        __syncthreads();
        const Scale& scale = s_scale;
        const int mine = 2 * tid;
        uint64_t first, own, before, cta, whole, below;
        for (;;) {
          uint4 next[kRestLoads];
          if (b0 + warp < b1) load(b0 + warp, next);
          for (int b = b0 + warp; b < b1; b += kRestWarps) {
            uint4 v[kRestLoads];
#pragma unroll
            for (int j = 0; j < kRestLoads; ++j) v[j] = next[j];
            if (b + kRestWarps < b1) load(b + kRestWarps, next);
            uint64_t sum = 0;
            // (not unrolled, here and below: the weights of a batch in line are many KB of instructions that are fetched for each)
#pragma unroll 1
            for (int j = 0; j < kRestLoads; ++j) {
              sum += K::exact_sum(v[0], scale, table);
              v[0] = v[1];
            }
            static_assert(kRestLoads == 2, "pieces");
            sum = warp_sum(sum);
            if (lane == 0) part[b - b0] = sum;
          }
          __syncthreads();
          // a thread has two neighbours
          static_assert(sizeof(part) / 8 <= 2 * kRestThreads, "batches");
          first = mine < b1 - b0 ? part[mine] : 0;
          own = first + (mine + 1 < b1 - b0 ? part[mine + 1] : 0);
          const uint64_t upto = warp_upto(own, lane);
          if (lane == 31) s_wide[warp] = upto;
          __syncthreads();
          before = upto - own, cta = 0;
#pragma unroll
          for (int i = 0; i < kRestWarps; ++i) {
            if (i < warp) before += s_wide[i];
            cta += s_wide[i];
          }
          if (tid < kRestCtas)
            asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(mapa_shared(smem_u32(&cta_wide[rank]), tid)), "l"(cta) : "memory");
          __syncwarp();
          sync();
          whole = 0, below = 0;
#pragma unroll
          for (int r = 0; r < kRestCtas; ++r) {
            if (r < rank) below += cta_wide[r];
            whole += cta_wide[r];
          }
          if (drop <= a.drop) break;
          // what the weights come to is known now: with all the places that it allows
          drop = drop_of(static_cast<float>(whole) * exp2f(static_cast<float>(a.drop - kFixed)), a.drop);
          sync();
          if (tid == 0) s_scale.drop = drop;
          __syncthreads();
        }
        const uint64_t place = static_cast<uint64_t>(static_cast<double>(set.u) * static_cast<double>(whole));
        if (set.u < kSmallNumber) {
          if (rank == 0) draw_small<TYPE>(a, row, K::LOWEST, m, whole, drop, all, reinterpret_cast<double*>(s_wide));
        } else if (place >= below && place < below + cta) {  // (one CTA)
          before += below;
          if (before <= place && place < before + own) {  // (one thread)
            const bool second = place >= before + first;
            s_batch = b0 + mine + second, s_from = before + (second ? first : 0);
          }
          __syncthreads();
          if (warp == 0) {
            uint4 v[kRestLoads];
            const int b = s_batch;
            load(b, v);
            uint64_t from = s_from;
#pragma unroll 1
            for (int j = 0; j < kRestLoads; ++j) {
              const uint64_t w = K::exact_sum(v[0], scale, table), upto = warp_upto(w, lane);
              const unsigned over = __ballot_sync(0xffffffffu, from + upto > place);
              if (over) {  // (the same for the warp)
                const int who = __ffs(over) - 1;
                uint4 piece;
                piece.x = __shfl_sync(0xffffffffu, v[0].x, who);
                piece.y = __shfl_sync(0xffffffffu, v[0].y, who);
                piece.z = __shfl_sync(0xffffffffu, v[0].z, who);
                piece.w = __shfl_sync(0xffffffffu, v[0].w, who);
                const uint64_t start = from + __shfl_sync(0xffffffffu, upto - w, who);
                float value;
                if (K::exact_find(piece, start, place, scale, table, lane, value)) {
                  a.tokens[row] = b * BATCH + (j * 32 + who) * VEC + lane - skip;
                  if (a.logprob) a.logprob[row] = set.log_of(value, m, others_of(whole, drop));
                  if (a.kept) a.kept[row] = static_cast<int32_t>(all);
                }
                break;
              }
              from += __shfl_sync(0xffffffffu, upto, 31);
              v[0] = v[1];
            }
          }
        }
        __syncwarp();
        sync();  // (the arrays are free)
    }
  }
}

// CTAs per row: until every SM has two, each warp with a batch at least.
int splits_of(int n_rows, int vocab, int type, int sms) {
  const int batch = kBatchBytes / (type == DFLASH_T_FP32 ? 4 : 2);
  const int most = (vocab + batch * kWarps - 1) / (batch * kWarps);
  int s = 1;  // powers of two
  while (2 * s <= kMaxSplits && 2 * s <= most && static_cast<long long>(n_rows) * s < sms) s *= 2;
  return s;
}

template <int TYPE>
cudaError_t launch(const SampleArgs& a, int sms, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.n_rows) * a.splits);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kRingBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.splits;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.splits > 1 ? 1 : 0;
  cudaError_t e = cudaFuncSetAttribute(sample_plain_kernel<TYPE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
  if (e == cudaSuccess && a.splits > 8)  // beyond the portable size
    e = cudaFuncSetAttribute(sample_plain_kernel<TYPE>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, sample_plain_kernel<TYPE>, a);
  if (e != cudaSuccess) return e;
  const int most = 2 * sms / kRestCtas;  // two CTAs per SM
  cfg.blockDim = dim3(kRestThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.gridDim = dim3(static_cast<unsigned>(a.n_rows < most ? a.n_rows : most) * kRestCtas);
  attr[0].val.clusterDim.x = kRestCtas;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sample_rest_kernel<TYPE>, a);
}

}  // namespace

cudaError_t launch_sample_plain(SampleArgs a, int type, cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  a.splits = splits_of(a.n_rows, a.vocab, type, sms);
  return type == DFLASH_T_FP32 ? launch<DFLASH_T_FP32>(a, sms, st)
         : type == DFLASH_T_BF16 ? launch<DFLASH_T_BF16>(a, sms, st)
                                 : launch<DFLASH_T_FP16>(a, sms, st);
}

}  // namespace dflash
