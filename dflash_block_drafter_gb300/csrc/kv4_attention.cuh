// What the kernels of the 4-bit paged attention share: arguments, the plan
// that shares a call's work out over CTAs, and the merge of split segments.
//
// A sequence s with r rows over kv cells has, per kv head, G * r query rows
// (row m = token m / G, head of the group m % G) which read the same cells: a
// segment.  They are at most as many as a CTA takes, R (the host picks the kernel and
// its R by G * max_rows).  A segment walks its visible cells in steps.  It counts as its
// steps plus OV units, which stand for what it costs to begin and to end one;
// all segments' units laid end to end are shared out evenly over C CTAs, so that
// every CTA has about the same work whatever the lengths (counted by steps
// alone, a CTA of 200 short requests got 17 segments where the mean was 4, and took
// twice the mean's time).  A segment that lies inside one CTA
// is written out by it; one that crosses into others leaves a piece (running
// maximum, sum, unnormalised O in FP32) per CTA, and the merge kernel joins
// them.  A CTA's range can hold at most two pieces: of the segment that began
// before it (slot 2c) and of one that begins in it and goes on (slot 2c + 1).
//
// The lengths are on the device, so every CTA forms the plan itself (prefix
// sums over at most kKv4MaxSeq sequences).
//
// Attention over a shared prefix takes two passes of the same kernels.  In the first
// (kKv4Prefix) the sequences are groups of requests: all rows of a group read the cells
// of the group's prefix, in segments of as many whole tokens as a CTA takes,
// the segments of one kv head side by side.  It leaves each row's maximum, sum and
// unnormalised O in `pre`.  The second (kKv4Own) is the attention of each request
// over its own cells, which joins them with `pre` where a row is written.
#pragma once

#include "common.cuh"
#include "internal.h"
#include "kernels.h"
#include "kv4.cuh"

namespace dflash {

constexpr int kKv4MaxSeq = 1024;

// Bounded wait for a phase of an mbarrier, as mbar_wait; the hint lets the
// hardware hold the warp up to 20 us per try instead of having it spin, which
// would take issue slots from the warps that unpack.
__device__ __forceinline__ bool kv4_wait(uint64_t* bar, uint32_t parity) {
  const uint32_t at = smem_u32(bar);
  unsigned long long t0 = 0;
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(at), "r"(parity), "r"(20000u)
        : "memory");
    if (ok) return true;
    const unsigned long long now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > kWaitTimeoutNs) return false;
  }
}

// The constants that turn the codes of a word into FP16 code - 8 (an integer put into the
// mantissa of 1024, as Kim et al., "Who Says Elephants Can't Run", 2022, publish it for
// weights).  Held in registers that the compiler takes for unknown: as immediates, the
// AND and the OR of a code would be two instructions (and the FMA's second constant a
// move), a third of the unpacking's arithmetic.
struct Kv4Consts {
  uint32_t base, minus_72;
  __device__ __forceinline__ Kv4Consts() {
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(base));      // 1024: a code in its low mantissa bits is added
    asm volatile("mov.b32 %0, 0xd480d480;" : "=r"(minus_72));
  }
  // codes 0 and 4 of a word (of a word shifted by 8: 2 and 6)
  __device__ __forceinline__ uint32_t even(uint32_t w) const {
    uint32_t r;
    asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(r) : "r"(w), "r"(base));
    return hsub2_u32(r, 0x64086408u);  // - 1032
  }
  // codes 1 and 5 (3 and 7), which count 16
  __device__ __forceinline__ uint32_t odd(uint32_t w) const {
    uint32_t r;
    asm("lop3.b32 %0, %1, 0x00f000f0, %2, 0xea;" : "=r"(r) : "r"(w), "r"(base));
    return hfma2_u32(r, 0x2c002c00u, minus_72);  // / 16 - 72
  }
};

// N consecutive words (1, 2 or 4) of shared memory.
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    static_assert(N == 4, "words");
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  }
}

// P is 2^(score - reference).  A row's reference is put kKv4Lift below its largest score so
// far and stays until a score passes it by 2^kKv4Slack, so that few tiles pay for a
// rescaling.  P up to 2^15 stays inside FP16's range, and at the lift a cell's weight is
// off by FP16's smallest step (2^-25) only 2^-32 below the largest, so that a
// long tail below one dominating cell keeps its sum (with the reference at the largest
// score, 32767 cells 2^-25.5 below another were lost).
constexpr float kKv4Slack = 15.f, kKv4Lift = 7.f;

// A call, or the passes of one over a shared prefix (above).
enum Kv4Mode { kKv4Plain, kKv4Prefix, kKv4Own };

struct Kv4Job;

struct Kv4AttnArgs {
  const uint8_t* cache;
  int n_pages, page_shift, n_kv, G;
  const uint16_t* q;
  uint16_t* out;
  int bf16;
  long long q_stride, out_stride;  // elements between tokens
  int n_seq, max_rows, n_tokens;
  const int32_t* row_offsets;
  const int32_t* kv_len;
  const int32_t* table;
  int table_stride;
  int causal, window;
  float scale_log2;  // softmax scale * log2(e)
  float* part;       // pieces' O [2 C][R][D]
  float2* part_ml;   // [2 C][R]: maximum (log2 units) and sum
  Kv4Job* jobs;  // [C]
  int32_t* status;
  // over a shared prefix; in its first pass n_seq, kv_len and table are those of the groups
  const int32_t* group_offsets;  // [n_seq + 1] sequences
  int n_all;       // sequences
  int per_segment;  // tokens of a segment
  float* pre;       // [n_tokens, n_q heads, D]
  float2* pre_ml;   // [n_tokens, n_q heads]: maximum (log2 units) and sum
};

// What sequence s asks for.
struct Kv4Seq {
  int r0, rows, kv;  // first token, tokens, cells
  int base, hi;      // visible cells [lo, hi) of any row, base = lo down to a step
  int lo;
  int steps;
};

template <int STEP, int MODE>
__device__ __forceinline__ Kv4Seq kv4_seq(const Kv4AttnArgs& a, int s, bool report) {
  Kv4Seq q;
  if constexpr (MODE == kKv4Prefix) {
    const int g0 = a.group_offsets[s], g1 = a.group_offsets[s + 1];
    const bool apart = (s == 0 && g0 != 0) || (s == a.n_seq - 1 && g1 != a.n_all);  // sequences of no group
    const bool bad = g0 < 0 || g1 < g0 || g1 > a.n_all;
    q.r0 = bad ? 0 : a.row_offsets[g0];
    const int r1 = bad ? 0 : a.row_offsets[g1];
    q.rows = r1 - q.r0;
    if (q.r0 < 0 || r1 > a.n_tokens || r1 < q.r0) q.rows = -1;
    if (report && (bad || apart || q.rows < 0)) set_status(a.status, DFLASH_DEV_BAD_BLOCK);
    q.rows = max(q.rows, 0);
  } else {
    q.r0 = a.row_offsets[s];
    const int r1 = a.row_offsets[s + 1];
    q.rows = r1 - q.r0;
    if (q.r0 < 0 || r1 > a.n_tokens || r1 < q.r0 || q.rows > a.max_rows) {
      if (report) set_status(a.status, DFLASH_DEV_BAD_BLOCK);
      q.rows = 0;
    }
  }
  const long long cap = static_cast<long long>(a.table_stride) << a.page_shift;
  int kv = a.kv_len[s];
  if (kv > cap) {
    if (report) set_status(a.status, DFLASH_DEV_CAPACITY);
    kv = static_cast<int>(cap);
  }
  q.kv = max(kv, 0);
  q.hi = q.kv;
  q.lo = 0;
  if (a.window > 0) {  // the first row that any window reaches
    const int upto = a.causal ? q.kv - q.rows + 1 : q.kv;  // behind the first row's own position
    q.lo = min(upto > a.window ? upto - a.window : 0, q.hi);
  }
  q.base = q.lo - q.lo % STEP;
  // rows that see no cell take one masked step, which writes their zeros
  q.steps = q.rows == 0 ? 0 : max((q.hi - q.base + STEP - 1) / STEP, 1);
  return q;
}

// The token x / G of a query row x < 128: x * ceil(2^17 / G) >> 17 (off by less than
// x G / 2^17 / G, below the 1 / G that a quotient lies from the next integer).
__device__ __forceinline__ uint32_t kv4_per_token(int G) { return ((1u << 17) + G - 1) / G; }
__device__ __forceinline__ int kv4_token(int x, uint32_t per_g) { return static_cast<int>(static_cast<uint32_t>(x) * per_g >> 17); }

// Segments of a sequence.
template <int MODE>
__device__ __forceinline__ int kv4_segments(const Kv4AttnArgs& a, int rows) {
  if constexpr (MODE == kKv4Prefix) return a.n_kv * ((rows + a.per_segment - 1) / a.per_segment);
  return a.n_kv;
}

// Row of `pre` of a token's head x of kv head `head`.
__device__ __forceinline__ size_t kv4_pre_row(const Kv4AttnArgs& a, int token, int head, int x) {
  return static_cast<size_t>(token) * (a.n_kv * a.G) + head * a.G + x;
}
// What brings a row's own results (maximum m, sum l) and its prefix's together: factors of both O,
// normalised; the sum of weights in l.
__device__ __forceinline__ float2 kv4_join(float m, float& l, float2 pre) {
  const float top = fmaxf(m, pre.x), from = top == -INFINITY ? 0.f : top;
  const float f = ex2_approx(m - from), g = ex2_approx(pre.x - from);
  l = l * f + pre.y * g;
  const float inv = l > 0.f ? 1.f / l : 0.f;
  return make_float2(f * inv, g * inv);
}

// Visible cells [lo, hi) of token i of the sequence.
__device__ __forceinline__ int2 kv4_sees(const Kv4AttnArgs& a, const Kv4Seq& q, int i) {
  const int upto = a.causal ? q.kv - q.rows + i + 1 : q.kv;  // behind the row's own position
  return make_int2(a.window > 0 && upto > a.window ? upto - a.window : 0, max(upto, 0));
}

// Prefix sums of the sequences' units (over their segments) in
// `pre` [n_seq + 1] by the whole CTA; returns the total.
template <int STEP, int OV, int MODE>
__device__ __forceinline__ long long kv4_plan(const Kv4AttnArgs& a, long long* pre, long long* scratch, bool report) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = blockDim.x;
  long long carry = 0;
  for (int s0 = 0; s0 < a.n_seq; s0 += n) {
    const int s = s0 + tid;
    long long v = 0;
    if (s < a.n_seq) {
      const Kv4Seq q = kv4_seq<STEP, MODE>(a, s, report);
      if (q.rows > 0) v = static_cast<long long>(q.steps + OV) * kv4_segments<MODE>(a, q.rows);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) scratch[warp] = v;
    __syncthreads();
    long long below = carry;
    for (int w = 0; w < n / 32; ++w) {
      if (w < warp) below += scratch[w];
      carry += scratch[w];
    }
    if (s < a.n_seq) pre[s + 1] = below + v;
    __syncthreads();
  }
  if (tid == 0) pre[0] = 0;
  __syncthreads();
  return carry;
}

// CTAs that a call of T units uses, at most `most`, and the unit that CTA c begins with.
__device__ __forceinline__ int kv4_ctas(long long T, int most) { return T < most ? max(static_cast<int>(T), 1) : most; }
__device__ __forceinline__ long long kv4_start(long long T, int C, int c) { return T * c / C; }
// The CTA whose range holds unit x.
__device__ __forceinline__ int kv4_owner(long long T, int C, long long x) {
  int c = static_cast<int>(x * C / T);
  while (kv4_start(T, C, c + 1) <= x) ++c;
  while (kv4_start(T, C, c) > x) --c;
  return c;
}

// A segment's part in a CTA: tiles [k0, k0 + n) of a sequence and kv head (n 0: no
// more parts).
struct Kv4Part {
  Kv4Seq q;
  int s, head, rows, k0, n;  // rows: query rows
  long long end, next;  // units: the segment's end; where this part ends
  // over a prefix, where q is the segment's: its number in the group, and the group's tokens
  int segment, r0, tokens;
};
// The first part with a tile in [at, x_end).  `hint`: the part before it, which ended at
// `at` (or a zeroed one for a CTA's first part, which may begin anywhere in a segment).
template <int STEP, int OV, int MODE>
__device__ __forceinline__ Kv4Part kv4_part(const Kv4AttnArgs& a, const long long* pre, long long at, long long x_end,
                                            const Kv4Part& hint) {
  Kv4Part p = hint;
  p.n = 0;
  p.next = x_end;
  if (at >= x_end) return p;
  constexpr bool PREFIX = MODE == kKv4Prefix;
  int& segment = PREFIX ? p.segment : p.head;
  const bool first = hint.n == 0;
  if (first || ++segment == kv4_segments<MODE>(a, PREFIX ? p.tokens : 1)) {  // another sequence
    int lo = 0, hi = a.n_seq - 1;
    if (!first && pre[p.s + 1] <= at && at < pre[p.s + 2]) lo = hi = p.s + 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid + 1] > at) hi = mid;
      else lo = mid + 1;
    }
    p.s = lo;
    p.q = kv4_seq<STEP, MODE>(a, lo, false);
    segment = 0;
    if (PREFIX) p.r0 = p.q.r0, p.tokens = p.q.rows;
  }
  const int units = p.q.steps + OV;
  long long begin = at;
  if (first) {
    const long long rel = at - pre[p.s];
    segment = rel >> 32 ? static_cast<int>(rel / units) : static_cast<int>(static_cast<uint32_t>(rel) / static_cast<uint32_t>(units));
    begin = pre[p.s] + static_cast<long long>(segment) * units;
  }
  p.end = begin + units;
  p.next = p.end < x_end ? p.end : x_end;
  p.k0 = max(static_cast<int>(at - begin) - OV, 0);
  p.n = max(static_cast<int>(p.next - begin) - OV, 0) - p.k0;  // 0: the range ends before the segment's first tile
  if constexpr (PREFIX) {
    const int of_head = (p.tokens + a.per_segment - 1) / a.per_segment;
    p.head = segment / of_head;
    const int skip = (segment - p.head * of_head) * a.per_segment;
    p.q.r0 = p.r0 + skip;
    p.q.rows = min(p.tokens - skip, a.per_segment);
  }
  p.rows = p.q.rows * a.G;
  return p;
}

// What a split segment's first CTA leaves for the merge kernel.
struct Kv4Job {
  int r0, head, n_rows;  // n_rows 0: no segment that goes on begins in this CTA
  int last;              // CTA of the last piece; the others lie between
};

// Joins the pieces of split segments: o = sum_i 2^(m_i - m) O_i /
// sum_i 2^(m_i - m) l_i.  Blocks (j, y): the j-th split segment, found by
// counting the records.  A warp has a row, a lane D / 32 channels of it.  With up to
// kFewPieces pieces the 8 warps of the blocks y take a row each; with more, the 8
// warps of a block share a row's pieces and join through shared memory, so that a
// segment of 150 pieces costs a warp 19 of them, four or eight in flight, not 150
// in turn.
constexpr int kMergeThreads = 256;
// (Over a prefix, whose segments of 128 rows have 10 to 20 pieces each, 16.  With 8, 16 and 32: 16 blocks of 8 over 32768 shared cells 122, 119 and
// 119 us, over 8192 83, 79 and 79; 64 tokens over 32768 126, 124 and 124; 8 blocks over 131072, 38 pieces each, 181, 182 and 180.)
template <int MODE>
constexpr int kFewPieces = MODE == kKv4Prefix ? 16 : 8;

template <int D, int R, int MODE>
__global__ void __launch_bounds__(kMergeThreads) kv4_merge_kernel(const Kv4AttnArgs a, int most) {
  constexpr int E = D / 32, WARPS = kMergeThreads / 32, U = D == 256 ? 4 : 8;
  __shared__ int s_count[WARPS];
  __shared__ int s_cta;
  __shared__ float acc[WARPS][D];
  __shared__ float2 accl[WARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) s_cta = -1;
  if constexpr (MODE == kKv4Prefix) pdl_launch_dependents();  // (the pass over the own cells)
  pdl_wait();
  int before = 0;  // split segments of earlier CTAs
  for (int c0 = 0; c0 < most; c0 += kMergeThreads) {
    const int c = c0 + tid;
    const bool is = c < most && __ldcg(&a.jobs[c].n_rows) > 0;
    const unsigned m = __ballot_sync(0xffffffffu, is);
    if (lane == 0) s_count[warp] = __popc(m);
    __syncthreads();
    int n = before + __popc(m & ((1u << lane) - 1));
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) n += s_count[w];
      before += s_count[w];
    }
    if (is && n == static_cast<int>(blockIdx.x)) s_cta = c;
    __syncthreads();
    if (s_cta >= 0) break;
  }
  const int c = s_cta;
  if (c < 0) return;
  const int4 j0 = __ldcg(reinterpret_cast<const int4*>(a.jobs + c));  // r0, head, rows, last
  const int n = j0.w - c + 1;
  const bool few = n <= kFewPieces<MODE>;
  const int i0 = few ? 0 : warp, step = few ? 1 : WARPS;
  const int m0 = few ? blockIdx.y * WARPS + warp : blockIdx.y, m_step = gridDim.y * (few ? WARPS : 1);
  for (int m = m0; m < j0.z; m += m_step) {
    float o[E], l = 0.f, top = -INFINITY;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int i = i0; i < n; i += step * U) {
      float2 ml[U];
      float v[U][E];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = i + u * step;
        ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int e = 0; e < E; ++e) v[u][e] = 0.f;
        if (k < n) {
          const size_t at = static_cast<size_t>(2 * (c + k) + (k == 0)) * R + m;
          ml[u] = __ldcg(a.part_ml + at);
#pragma unroll
          for (int e = 0; e < E; e += (E < 4 ? 2 : 4)) {  // 64 or 128 channels of the row a load
            if constexpr (E < 4) {
              const float2 x = __ldcg(reinterpret_cast<const float2*>(a.part + at * D) + lane);
              v[u][0] = x.x, v[u][1] = x.y;
            } else {
              const float4 x = __ldcg(reinterpret_cast<const float4*>(a.part + at * D) + (e >> 2) * 32 + lane);
              v[u][e] = x.x, v[u][e + 1] = x.y, v[u][e + 2] = x.z, v[u][e + 3] = x.w;
            }
          }
        }
      }
      float t = top;
#pragma unroll
      for (int u = 0; u < U; ++u) t = fmaxf(t, ml[u].x);
      const float from = t == -INFINITY ? 0.f : t, f = ex2_approx(top - from);
      l *= f;
      top = t;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float w = ex2_approx(ml[u].x - from);
        l = fmaf(w, ml[u].y, l);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(w, v[u][e], o[e]);
      }
    }
    if (!few) {  // the warps' results: every warp adds up D / 8 channels
      __syncthreads();  // the last row's have been read
#pragma unroll
      for (int e = 0; e < E; ++e) acc[warp][e * 32 + lane] = o[e];
      if (lane == 0) accl[warp] = make_float2(top, l);
      __syncthreads();
      if (warp > 0) continue;
      float t = -INFINITY;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) t = fmaxf(t, accl[w].x);
      const float from = t == -INFINITY ? 0.f : t;
      top = t;
      l = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float f = ex2_approx(accl[w].x - from);
        l = fmaf(f, accl[w].y, l);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(f, acc[w][e * 32 + lane], o[e]);
      }
    }
    float inv = l > 0.f ? 1.f / l : 0.f;
    if constexpr (MODE != kKv4Plain) {
      const size_t at = kv4_pre_row(a, j0.x + m / a.G, j0.y, m % a.G);
      float* pre = a.pre + at * D;
      float2 f = make_float2(1.f, 0.f);
      if constexpr (MODE == kKv4Own) f = kv4_join(top, l, __ldcg(a.pre_ml + at));
      else if (lane == 0) __stcg(a.pre_ml + at, make_float2(top, l));
#pragma unroll
      for (int e = 0; e < E; e += (E < 4 ? 2 : 4)) {
        if constexpr (E < 4) {
          float2* x = reinterpret_cast<float2*>(pre) + lane;
          if constexpr (MODE == kKv4Prefix) {
            __stcg(x, make_float2(o[0], o[1]));
          } else {
            const float2 y = __ldcg(x);
            o[0] = o[0] * f.x + y.x * f.y, o[1] = o[1] * f.x + y.y * f.y;
          }
        } else {
          float4* x = reinterpret_cast<float4*>(pre) + (e >> 2) * 32 + lane;
          if constexpr (MODE == kKv4Prefix) {
            __stcg(x, make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]));
          } else {
            const float4 y = __ldcg(x);
            o[e] = o[e] * f.x + y.x * f.y, o[e + 1] = o[e + 1] * f.x + y.y * f.y;
            o[e + 2] = o[e + 2] * f.x + y.z * f.y, o[e + 3] = o[e + 3] * f.x + y.w * f.y;
          }
        }
      }
      inv = 1.f;
    }
    if (!(l < INFINITY) && lane == 0) set_status(a.status, DFLASH_DEV_NONFINITE);
    if constexpr (MODE == kKv4Prefix) continue;
    uint16_t* dst = a.out + (j0.x + m / a.G) * a.out_stride + (j0.y * a.G + m % a.G) * D;
    auto pack = [&](float x, float y) { return a.bf16 ? pack_bf16x2(x * inv, y * inv) : pack_f16x2(x * inv, y * inv); };
    if constexpr (E < 4) {
      reinterpret_cast<uint32_t*>(dst)[lane] = pack(o[0], o[1]);
    } else {
#pragma unroll
      for (int e = 0; e < E; e += 4)
        reinterpret_cast<uint2*>(dst)[(e >> 2) * 32 + lane] = make_uint2(pack(o[e], o[e + 1]), pack(o[e + 2], o[e + 3]));
    }
  }
}

// Launches a kernel; `early`: it may begin while the one before still ends.
template <typename... P, typename... A>
cudaError_t kv4_launch(void (*kernel)(P...), bool early, dim3 grid, int threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Launches the merge behind an attention kernel of `most` CTAs, of which at
// most `jobs` segments can be split.
template <int D, int R, int MODE>
cudaError_t launch_kv4_merge(const Kv4AttnArgs& a, int most, int jobs, cudaStream_t st) {
  // few segments: one block per row, which many pieces want; many: at least one warp per row
  const int y = 1536 / jobs, few = (R + 7) / 8;
  return kv4_launch(kv4_merge_kernel<D, R, MODE>, true, dim3(jobs, y < few ? few : y < R ? y : R), kMergeThreads, 0, st, a, most);
}

// What the host knows of a call: its kernel, CTAs and split segments at most.
struct Kv4Shape {
  bool tc;    // the tcgen05 kernel: up to 128 query rows a segment
  int nt;     // else: 8-row tiles of them
  int most, jobs;
  int rows() const { return tc ? 128 : 8 * nt; }
};
// Checks of what both kinds of call have, and the shape of one over the requests' own cells
// (kv4_attention.cu).
int kv4_check_call(const dflash_kv4_cache* c, int n_q_heads, int n_seq, int max_rows, int table_stride);
cudaError_t kv4_shape_of(const dflash_kv4_cache* c, int n_q_heads, int n_seq, int max_rows, int table_stride, Kv4Shape* out);
// CTAs of the tcgen05 kernel for so many segments.
cudaError_t kv4_tc_shape(const dflash_kv4_cache* c, long long segments, int table_stride, Kv4Shape* out);
// Workspace of a pass: its jobs and pieces.
inline size_t kv4_pass_bytes(const dflash_kv4_cache* c, const Kv4Shape& s) {
  return s.most * (sizeof(Kv4Job) + 2 * size_t(s.rows()) * (c->head_dim * 4 + 8));
}
inline void kv4_set_workspace(Kv4AttnArgs& a, const dflash_kv4_cache* c, const Kv4Shape& s, void* workspace) {
  a.jobs = static_cast<Kv4Job*>(workspace);
  a.part = reinterpret_cast<float*>(a.jobs + s.most);
  a.part_ml = reinterpret_cast<float2*>(a.part + static_cast<size_t>(2 * s.most) * s.rows() * c->head_dim);
}

// The tcgen05 kernel (kv4_attention_tc.cuh): up to 128 rows, tiles of 64 cells at 256 channels, else of
// 128, one CTA per SM; of a plain call (kv4_attention_tc.cu) and of the passes of one over a shared prefix
// (kv4_prefix_attention_tc.cu).
cudaError_t launch_kv4_attn_tc(int d, const Kv4AttnArgs& a, int most, int jobs, cudaStream_t st);
cudaError_t launch_kv4_attn_tc_prefix(int d, const Kv4AttnArgs& a, int most, int jobs, cudaStream_t st);
cudaError_t launch_kv4_attn_tc_own(int d, const Kv4AttnArgs& a, int most, int jobs, cudaStream_t st);

}  // namespace dflash
