// Attention over the 4-bit paged K/V cache (dflash_kv4_attention in
// include/dflash.h): few query rows per kv head.
//
//   o_r = sum_j p_rj v_j / sum_j p_rj,   p_rj = 2^(s_rj - m_r),
//   s_rj = scale log2(e) q_r . k_j,      k, v = d (code - 8) per 32 channels.
//
// A call reads 1.125 bytes per channel of a cell (K and V), so at the memory's
// rate every scheduler has about 95 cycles for each 1024 codes: the unpacking
// has to be lean.  The products run on the warp-level matrix instruction with
// the cells as its M = 16 and 8 query rows as its N, so that single tokens
// waste few rows.
//
// S^T = K Q^T.  A lane's code word holds 8 channels.  `word & 0x000f000f` is
// already a pair of FP16 numbers: a code c in the low bits of an FP16 pattern
// is the subnormal c 2^-24, which the tensor cores take exactly (c 2^-20 for
// the mask 0x00f000f0), so unpacking K is 4 ANDs and a shift per word.  Q
// carries the other factor (FP16 rows scaled by a power of two, so nothing of
// BF16 is lost), the -8 of the codes is the accumulator's start value
// -8 2^-24 sum(q) of the 32-channel block, and the block's scale multiplies the
// finished FP32 sum: K enters the scores without any rounding.
// O^T = V^T P^T.  Two cells' words are interleaved (prmt) into pairs along the
// cells, turned into code - 8 (1024 + c, minus 1032) and multiplied by the
// cells' scales in FP16: one rounding of 2^-12 at most relative to the value.
// P goes through movmatrix from the accumulator layout to the B operand's and is
// rounded to FP16 (2^-12 relative at most, 2^-25 absolute; the sums are FP32 of
// the unrounded p).
//
// Work: 4 warps per CTA, each walks every fourth step of 32 cells of the
// CTA's range with its own maximum, sum and O in registers; bulk copies of
// whole groups (K, V and scales together) run a ring of stages ahead per warp.
// At a segment's end the warps' results are joined through the ring's memory.
#include <cstddef>

#include "kv4_attention.cuh"

namespace dflash {
namespace {

constexpr int kStep = 32;     // cells of a step: two groups
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kLeast = 4;     // steps that a CTA takes at least: one per warp

template <int D, int NT>
struct Geo {
  static constexpr int R = 8 * NT;                 // rows of a row group
  static constexpr int STAGE = 2 * Kv4<D>::GROUP_BYTES;
  static constexpr int STAGES = D == 256 ? 2 : D == 128 ? 4 : 8;
  static constexpr int RING = kWarps * STAGES * STAGE;
  static constexpr int QF = NT * (D / 32) * 512;   // Q fragments
  static constexpr int QS = NT * (D / 32) * 8 * 4; // accumulator start values
  static constexpr int SMEM = RING + QF + QS;
  static_assert(kWarps * R * D * 4 <= RING, "the warps' O fit the ring");
};

__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t bits) { return (v & mask) | bits; }

// D = A B + C for one 16 x 8 tile with a start value.
__device__ __forceinline__ void mma_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, float c0, float c1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}

__device__ __forceinline__ uint32_t movmatrix_t(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// N consecutive bytes (4, 8 or 16 a load) from shared memory.
template <int N>
__device__ __forceinline__ void load_words(uint32_t addr, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = lds32(addr);
  } else if constexpr (N == 2) {
    const uint2 v = lds64(addr);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    static_assert(N == 4, "words");
    const uint4 v = lds128(addr);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 2) kv4_attn_kernel(const Kv4AttnArgs a) {
  using F = Kv4<D>;
  using G = Geo<D, NT>;
  constexpr int R = G::R, B = F::BLOCKS, U = D / 64, ST = G::STAGES;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* ring = smem;
  uint8_t* qf = smem + G::RING;                                // [NT][B][32 lanes][16 B]
  float* qstart = reinterpret_cast<float*>(qf + G::QF);        // [NT][B][8 rows]
  __shared__ long long pre[kKv4MaxSeq + 1];
  __shared__ long long scratch[kWarps];
  __shared__ uint64_t bars[kWarps][ST];
  __shared__ float s_factor[R];
  __shared__ float2 s_ml[kWarps][R];
  __shared__ int2 s_sees[R];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  if (tid == 0) {
    for (int w = 0; w < kWarps; ++w)
      for (int i = 0; i < ST; ++i) mbar_init(&bars[w][i], 1);
    fence_barrier_init();
  }
  const long long T = kv4_plan<kStep, R>(a, pre, scratch, blockIdx.x == 0);
  const int C = kv4_ctas(T, gridDim.x, kLeast);
  const int c = blockIdx.x;
  pdl_launch_dependents();
  if (c >= C || T == 0) return;
  long long x = kv4_start(T, C, c);
  const long long x_end = kv4_start(T, C, c + 1);

  const int groups_of_page = 1 << (a.page_shift - 4);
  const int cell_g = (g & 1) ? 7 - (g >> 1) : g >> 1;  // cell of S^T's row g (and 8 + cell_g of row g + 8)
  uint8_t* my_ring = ring + warp * (ST * G::STAGE);
  uint64_t* my_bar = bars[warp];
  uint32_t phases = 0;  // bit i: parity of the next fill of the warp's stage i
  bool ok = true;

  while (x < x_end) {
    const int s = kv4_find(pre, a.n_seq, x);
    const Kv4Seq q = kv4_seq<kStep, R>(a, s, false);
    const long long rel = x - pre[s];
    const int unit = static_cast<int>(rel / q.steps);
    const int k0 = static_cast<int>(rel - static_cast<long long>(unit) * q.steps);
    const int k1 = static_cast<int>(min(static_cast<long long>(q.steps), k0 + (x_end - x)));
    const int head = unit / q.groups, row0 = unit % q.groups * R;
    const int n_rows = min(R, q.rows * a.G - row0);
    x += k1 - k0;

    // ---- copies: step k's groups go to stage i of the warp's ring
    const int32_t* pages = a.table + static_cast<long long>(s) * a.table_stride;
    // lanes look up the groups of 16 of the warp's steps at a time
    int my_page = 0, look0 = -1;
    auto issue = [&](int i) {  // the warp's i-th step
      const int k = k0 + warp + i * kWarps;
      if ((i >> 4) != look0) {
        look0 = i >> 4;
        const int kk = k0 + warp + ((look0 << 4) + (lane >> 1)) * kWarps;
        const int pos = q.base + kk * kStep + (lane & 1) * 16;
        my_page = -1;
        if (kk < k1 && pos < q.hi) {
          int page = pages[pos >> a.page_shift];
          if (page < 0 || page >= a.n_pages) {
            set_status(a.status, DFLASH_DEV_CAPACITY);
            page = 0;
          }
          my_page = page;
        }
      }
      const int p0 = __shfl_sync(0xffffffffu, my_page, (i & 15) * 2);
      const int p1 = __shfl_sync(0xffffffffu, my_page, (i & 15) * 2 + 1);
      if (lane == 0) {
        const int st = i % ST;
        uint8_t* dst = my_ring + st * G::STAGE;
        const int grp = ((q.base + k * kStep) >> 4) & (groups_of_page - 1);
        const int grp1 = ((q.base + k * kStep + 16) >> 4) & (groups_of_page - 1);
        mbar_arrive_expect_tx(&my_bar[st], ((p0 >= 0) + (p1 >= 0)) * F::GROUP_BYTES);
        if (p0 >= 0)
          bulk_g2s(dst, a.cache + ((static_cast<size_t>(p0) * a.n_kv + head) * groups_of_page + grp) * F::GROUP_BYTES,
                   F::GROUP_BYTES, &my_bar[st]);
        if (p1 >= 0)
          bulk_g2s(dst + F::GROUP_BYTES,
                   a.cache + ((static_cast<size_t>(p1) * a.n_kv + head) * groups_of_page + grp1) * F::GROUP_BYTES,
                   F::GROUP_BYTES, &my_bar[st]);
      }
    };
    const int mine = ok && k1 - k0 > warp ? (k1 - k0 - warp + kWarps - 1) / kWarps : 0;  // the warp's steps
    // the ring was last read (and written, by the join) through the generic proxy
    fence_proxy_async_smem();
    __syncthreads();
    for (int i = 0; i < min(mine, ST); ++i) issue(i);

    // ---- Q: 8 threads a row find its maximum, scale it and lay out the fragments
    for (int m = tid >> 3; m < R; m += kThreads / 8) {
      constexpr int E = D / 8;  // channels of a thread, consecutive
      const int part = tid & 7;
      float v[E];
      float top = 0.f;
      const int row = row0 + m;
      if (m < n_rows) {
        const uint16_t* src = a.q + (q.r0 + row / a.G) * a.q_stride + (head * a.G + row % a.G) * D + part * E;
#pragma unroll
        for (int e = 0; e < E; e += 8) {
          const uint4 raw = *reinterpret_cast<const uint4*>(src + e);
          const uint32_t pr[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t h = (j & 1) ? pr[j >> 1] >> 16 : pr[j >> 1] & 0xffffu;
            v[e + j] = a.bf16 ? __uint_as_float(h << 16) : __half2float(__ushort_as_half(static_cast<uint16_t>(h)));
            top = fmaxf(top, fabsf(v[e + j]));
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = 0.f;
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      // power of two that brings the row's maximum into [2^12, 2^13)
      const int ex = static_cast<int>(__float_as_uint(top) >> 23);
      const int up = top > 0.f ? min(12 + 127 - ex, 120) : 0;
      const float f = ldexpf(1.f, up);
      if (part == 0) {
        s_factor[m] = ldexpf(a.scale_log2, 24 - up);
        s_sees[m] = m < n_rows ? kv4_sees(a, q, row / a.G) : make_int2(0, 0);
      }
      // element e of block b, quad tt: word 4b + tt, nibble e; even nibbles as
      // they are, odd ones / 16 (their codes are 16 times as large)
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < E; e += 8) {
        const int w = (part * E + e) >> 3, b = w >> 2, tt = w & 3;
        __half h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          h[j] = __float2half_rn(v[e + j] * ((j & 1) ? f * 0.0625f : f));
          sum += __half2float(h[j]) * ((j & 1) ? 16.f : 1.f);
        }
        auto pair = [&](int lo, int hi) {
          const __half2 p = __halves2half2(h[lo], h[hi]);
          return *reinterpret_cast<const uint32_t*>(&p);
        };
        *reinterpret_cast<uint4*>(qf + (((m >> 3) * B + b) * 32 + (m & 7) * 4 + tt) * 16) =
            make_uint4(pair(0, 4), pair(1, 5), pair(2, 6), pair(3, 7));
        if constexpr (E == 32) {
          if (e == 24) {
            qstart[((m >> 3) * B + b) * 8 + (m & 7)] = sum * (-8.f / 16777216.f);
            sum = 0.f;
          }
        }
      }
      if constexpr (E < 32) {  // 32 / E threads share a block
#pragma unroll
        for (int o = 1; o < 32 / E; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (part % (32 / E) == 0) {
          const int b = part * E / 32;
          qstart[((m >> 3) * B + b) * 8 + (m & 7)] = sum * (-8.f / 16777216.f);
        }
      }
    }
    __syncthreads();

    float o[U][4][NT][4];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[u][i][n][e] = 0.f;
    float m_run[NT][2], l_run[NT][2], fac[NT][2];
    int2 sees[NT][2];
    int all_lo = 0, all_hi = 0x7fffffff;  // cells that every row sees
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m_run[n][e] = -INFINITY;
        l_run[n][e] = 0.f;
        fac[n][e] = s_factor[n * 8 + 2 * t + e];
        sees[n][e] = s_sees[n * 8 + 2 * t + e];
        if (n * 8 + 2 * t + e < n_rows) {
          all_lo = max(all_lo, sees[n][e].x);
          all_hi = min(all_hi, sees[n][e].y);
        }
      }
#pragma unroll
    for (int w = 1; w < 4; w <<= 1) {
      all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, w));
      all_hi = min(all_hi, __shfl_xor_sync(0xffffffffu, all_hi, w));
    }

    for (int i = 0; i < mine; ++i) {
      const int st = i % ST;
      ok = __all_sync(0xffffffffu, mbar_wait(&my_bar[st], (phases >> st) & 1));
      if (!ok) {
        // give up: nothing more is issued; what is in flight lands before the CTA ends
        for (int j = i; j < min(mine, i + ST); ++j) mbar_wait(&my_bar[j % ST], (phases >> (j % ST)) & 1);
        if (lane == 0) set_status(a.status, DFLASH_DEV_TIMEOUT);
        break;
      }
      phases ^= 1u << st;
      const uint32_t base = smem_u32(my_ring + st * G::STAGE);
      const int pos0 = q.base + (k0 + warp + i * kWarps) * kStep;
      const bool edge = pos0 < all_lo || pos0 + kStep > all_hi;
      float sc[2][NT][4];
      // ---- S^T
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const uint32_t gb = base + mt * F::GROUP_BYTES;
        // the lane's words and scales of cells cell_g and 8 + cell_g
        uint32_t wa[B], wb[B];
#pragma unroll
        for (int h = 0; h < (B + 3) / 4; ++h) {
          constexpr int N = B < 4 ? B : 4;
          uint32_t tmp[N];
          const uint32_t at = gb + cell_g * F::ROW + 4 * ((t * B + 4 * h) ^ F::k_swap(cell_g));
          load_words<N>(at, tmp);
#pragma unroll
          for (int e = 0; e < N; ++e) wa[4 * h + e] = tmp[e];
          // cell 8 + cell_g: k_swap goes by bit 2 of the cell, the same
          load_words<N>(at + 8 * F::ROW, tmp);
#pragma unroll
          for (int e = 0; e < N; ++e) wb[4 * h + e] = tmp[e];
        }
        uint32_t da[B / 2], db[B / 2];
        load_words<B / 2>(gb + F::K_SCALES + cell_g * F::SROW, da);
        load_words<B / 2>(gb + F::K_SCALES + (cell_g + 8) * F::SROW, db);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[mt][n][e] = 0.f;
#pragma unroll
        for (int b = 0; b < B; ++b) {
          const __half2 ha = *reinterpret_cast<const __half2*>(&da[b >> 1]);
          const __half2 hb = *reinterpret_cast<const __half2*>(&db[b >> 1]);
          const float fa = (b & 1) ? __high2float(ha) : __low2float(ha);
          const float fb = (b & 1) ? __high2float(hb) : __low2float(hb);
          const uint32_t va = wa[b] >> 8, vb = wb[b] >> 8;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint4 bq = *reinterpret_cast<const uint4*>(qf + ((n * B + b) * 32 + lane) * 16);
            const float2 start = *reinterpret_cast<const float2*>(qstart + (n * B + b) * 8 + 2 * t);
            float acc[4];
            mma_from(acc, wa[b] & 0x000f000fu, wb[b] & 0x000f000fu, wa[b] & 0x00f000f0u, wb[b] & 0x00f000f0u, bq.x,
                     bq.y, start.x, start.y);
            mma_f16_16816(acc, va & 0x000f000fu, vb & 0x000f000fu, va & 0x00f000f0u, vb & 0x00f000f0u, bq.z, bq.w);
            sc[mt][n][0] = fmaf(fa, acc[0], sc[mt][n][0]);
            sc[mt][n][1] = fmaf(fa, acc[1], sc[mt][n][1]);
            sc[mt][n][2] = fmaf(fb, acc[2], sc[mt][n][2]);
            sc[mt][n][3] = fmaf(fb, acc[3], sc[mt][n][3]);
          }
        }
      }
      // ---- softmax: maximum over the step's cells, P in the B operand's layout
      uint32_t pb[2][NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float v = sc[mt][n][e] * fac[n][e & 1];
            if (edge) {
              const int pos = pos0 + mt * 16 + cell_g + (e >> 1) * 8;
              if (pos < sees[n][e & 1].x || pos >= sees[n][e & 1].y) v = -INFINITY;
            }
            sc[mt][n][e] = v;
            top[e & 1] = fmaxf(top[e & 1], v);
          }
        float from[2], alpha[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], w));
          const float m_new = fmaxf(m_run[n][e], top[e]);
          from[e] = m_new == -INFINITY ? 0.f : m_new;
          alpha[e] = ex2_approx(m_run[n][e] - from[e]);
          m_run[n][e] = m_new;
          l_run[n][e] *= alpha[e];
        }
        if (__any_sync(0xffffffffu, alpha[0] < 1.f || alpha[1] < 1.f)) {
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[u][j][n][e] *= alpha[e & 1];
        }
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = ex2_approx(sc[mt][n][e] - from[e & 1]);
            l_run[n][e & 1] += p[e];
          }
          pb[mt][n][0] = movmatrix_t(pack_f16x2(p[0], p[1]));
          pb[mt][n][1] = movmatrix_t(pack_f16x2(p[2], p[3]));
        }
      }
      // ---- O^T: cells t, 7 - t and 8 + t, 15 - t of each group
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const uint32_t gb = base + mt * F::GROUP_BYTES;
        uint32_t vw[4][U];
        uint32_t vs[4][(U + 1) / 2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int cell = (k & 1 ? 7 - t : t) + (k >> 1) * 8;
          load_words<U>(gb + F::V_CODES + cell * F::ROW + 4 * U * (g ^ F::v_swap(cell)), vw[k]);
          const uint32_t at = gb + F::V_SCALES + cell * F::SROW + (g >> 2) * (U * 2);
          if constexpr (U == 1) {
            uint16_t h;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(at));
            vs[k][0] = h;
          } else {
            load_words<U / 2>(at, vs[k]);
          }
          if (edge) {  // cells that no row sees may hold anything: no weight times NaN
            const int pos = pos0 + mt * 16 + cell;
            if (pos < q.lo || pos >= q.hi) {
#pragma unroll
              for (int e = 0; e < (U + 1) / 2; ++e) vs[k][e] = 0;
            }
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t sel = (u & 1) ? 0x7632u : 0x5410u;
          const uint32_t d0 = prmt(vs[0][u >> 1], vs[1][u >> 1], sel);
          const uint32_t d1 = prmt(vs[2][u >> 1], vs[3][u >> 1], sel);
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // channels 64u + 8g + 2j, + 1
            const uint32_t half = (j >> 1) ? 0x7632u : 0x5410u;
            uint32_t lo = prmt(vw[0][u], vw[1][u], half), hi = prmt(vw[2][u], vw[3][u], half);
            if (j & 1) {
              lo >>= 8;
              hi >>= 8;
            }
            constexpr uint32_t MINUS_1032 = 0xe408e408u, SIXTEENTH = 0x2c002c00u, MINUS_72 = 0xd480d480u;
            const uint32_t a0 = hmul2_u32(hfma2_u32(and_or(lo, 0x000f000fu, 0x64006400u), 0x3c003c00u, MINUS_1032), d0);
            const uint32_t a1 = hmul2_u32(hfma2_u32(and_or(lo, 0x00f000f0u, 0x64006400u), SIXTEENTH, MINUS_72), d0);
            const uint32_t a2 = hmul2_u32(hfma2_u32(and_or(hi, 0x000f000fu, 0x64006400u), 0x3c003c00u, MINUS_1032), d1);
            const uint32_t a3 = hmul2_u32(hfma2_u32(and_or(hi, 0x00f000f0u, 0x64006400u), SIXTEENTH, MINUS_72), d1);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16_16816(o[u][j][n], a0, a1, a2, a3, pb[mt][n][0], pb[mt][n][1]);
          }
        }
      }
      __syncwarp();
      if (i + ST < mine) issue(i + ST);
    }
    // ---- join the warps: factors to the common maximum, then sums through the ring's memory
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l_run[n][e] += __shfl_xor_sync(0xffffffffu, l_run[n][e], w);
        if (g == 0) s_ml[warp][n * 8 + 2 * t + e] = make_float2(m_run[n][e], l_run[n][e]);
      }
    __syncthreads();
    float* buf = reinterpret_cast<float*>(ring);  // [warp][row][D]
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int m = n * 8 + 2 * t + e;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_ml[w][m].x);
        const float f = top == -INFINITY ? 0.f : ex2_approx(m_run[n][e] - top);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float* dst = buf + (warp * R + m) * D + 64 * u + 8 * g;
          *reinterpret_cast<float4*>(dst) =
              make_float4(o[u][0][n][e] * f, o[u][0][n][2 + e] * f, o[u][1][n][e] * f, o[u][1][n][2 + e] * f);
          *reinterpret_cast<float4*>(dst + 4) =
              make_float4(o[u][2][n][e] * f, o[u][2][n][2 + e] * f, o[u][3][n][e] * f, o[u][3][n][2 + e] * f);
        }
      }
    __syncthreads();
    const bool whole = k0 == 0 && k1 == q.steps;
    const int slot = 2 * c + (k0 == 0 ? 1 : 0);
    for (int i = tid; i < n_rows * (D / 4); i += kThreads) {
      const int m = i / (D / 4), col = i % (D / 4) * 4;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_ml[w][m].x);
      const float from = top == -INFINITY ? 0.f : top;
      float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
      float l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 v = *reinterpret_cast<const float4*>(buf + (w * R + m) * D + col);
        r.x += v.x;
        r.y += v.y;
        r.z += v.z;
        r.w += v.w;
        l = fmaf(s_ml[w][m].y, ex2_approx(s_ml[w][m].x - from), l);
      }
      if (whole) {
        const float inv = l > 0.f ? 1.f / l : 0.f;
        if (!(l < INFINITY)) set_status(a.status, DFLASH_DEV_NONFINITE);
        const int row = row0 + m;
        uint16_t* dst = a.out + (q.r0 + row / a.G) * a.out_stride + (head * a.G + row % a.G) * D + col;
        *reinterpret_cast<uint2*>(dst) =
            a.bf16 ? make_uint2(pack_bf16x2(r.x * inv, r.y * inv), pack_bf16x2(r.z * inv, r.w * inv))
                   : make_uint2(pack_f16x2(r.x * inv, r.y * inv), pack_f16x2(r.z * inv, r.w * inv));
      } else {
        __stcg(reinterpret_cast<float4*>(a.part + (static_cast<size_t>(slot) * R + m) * D + col), r);
        if (col == 0) __stcg(a.part_ml + static_cast<size_t>(slot) * R + m, make_float2(top, l));
      }
    }
  }
}


template <int D, int NT>
cudaError_t launch_attn(const Kv4AttnArgs& a, int most, cudaStream_t st) {
  using G = Geo<D, NT>;
  cudaError_t e = cudaFuncSetAttribute(kv4_attn_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM);
  if (e != cudaSuccess) return e;
  kv4_attn_kernel<D, NT><<<most, kThreads, G::SMEM, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || most == 1) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(most, G::R);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_merge_kernel<D, kStep, G::R>, a, most, kLeast);
}

// Rows per kv head that a call can have choose the width of the row groups.
struct Shape {
  int nt, most;
};
cudaError_t shape_of(const dflash_kv4_cache* c, int n_q_heads, int n_seq, int max_rows, int table_stride, Shape* out) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int rows = n_q_heads / c->n_kv_heads * max_rows;
  out->nt = rows <= 8 ? 1 : 2;
  const long long groups = (rows + 8 * out->nt - 1) / (8 * out->nt);
  const long long steps = (static_cast<long long>(table_stride) * c->page_size + kStep - 1) / kStep + 1;
  const long long ctas = (static_cast<long long>(n_seq) * c->n_kv_heads * groups * steps + kLeast - 1) / kLeast;
  out->most = static_cast<int>(ctas < 2 * sms ? ctas : 2 * sms);
  return cudaSuccess;
}

int check_call(const dflash_kv4_cache* c, int n_q_heads, int n_seq, int max_rows, int table_stride) {
  if (const int e = dflash_kv4_check(c)) return e;
  if (n_seq < 1 || table_stride < 1 || n_q_heads < 1 || n_q_heads % c->n_kv_heads) return DFLASH_ERR_INVALID_ARG;
  if (max_rows < 1 || max_rows > DFLASH_MAX_BLOCK) return DFLASH_ERR_INVALID_ARG;
  if (n_seq > kKv4MaxSeq) return DFLASH_ERR_CAPACITY;
  if (n_q_heads / c->n_kv_heads * max_rows > 128) return DFLASH_ERR_UNSUPPORTED;
  return DFLASH_OK;
}

size_t bytes_of(const dflash_kv4_cache* c, const Shape& s) {
  return static_cast<size_t>(2 * s.most) * 8 * s.nt * (c->head_dim * 4 + 8);
}

}  // namespace
}  // namespace dflash

using namespace dflash;

extern "C" {

size_t dflash_kv4_attention_workspace(const dflash_kv4_cache* c, int32_t n_q_heads, int32_t n_seq, int32_t max_rows,
                                      int32_t table_stride) {
  Shape s;
  if (check_call(c, n_q_heads, n_seq, max_rows, table_stride) != DFLASH_OK ||
      shape_of(c, n_q_heads, n_seq, max_rows, table_stride, &s) != cudaSuccess)
    return 0;
  return bytes_of(c, s);
}

int dflash_kv4_attention(const dflash_kv4_cache* c, const void* q, void* out, int32_t type, int64_t q_stride,
                         int64_t out_stride, int32_t n_tokens, int32_t n_q_heads, int32_t n_seq, int32_t max_rows,
                         const int32_t* row_offsets, const int32_t* kv_len, const int32_t* table, int32_t table_stride,
                         int32_t causal, int32_t window, float scale, void* workspace, size_t workspace_bytes,
                         int32_t* dev_status, dflash_stream_t stream) {
  if (const int e = check_call(c, n_q_heads, n_seq, max_rows, table_stride)) return e;
  if (type != DFLASH_T_BF16 && type != DFLASH_T_FP16) return DFLASH_ERR_UNSUPPORTED;
  const int64_t width = static_cast<int64_t>(n_q_heads) * c->head_dim;
  if (n_tokens < 0 || window < 0 || !(scale > 0.f) || !(scale < INFINITY)) return DFLASH_ERR_INVALID_ARG;
  if (!row_offsets || !kv_len || !table) return DFLASH_ERR_INVALID_ARG;
  if (n_tokens == 0) return DFLASH_OK;
  if (!q || !out || reinterpret_cast<uintptr_t>(q) % 16 || reinterpret_cast<uintptr_t>(out) % 16 || q_stride < width ||
      out_stride < width || q_stride % 8 || out_stride % 8)
    return DFLASH_ERR_INVALID_ARG;
  Shape s;
  cudaError_t e = shape_of(c, n_q_heads, n_seq, max_rows, table_stride, &s);
  if (e != cudaSuccess) return cuda_status(e, "kv4 attention");
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16) return DFLASH_ERR_INVALID_ARG;
  if (workspace_bytes < bytes_of(c, s)) return DFLASH_ERR_CAPACITY;
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
  a.part = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part + static_cast<size_t>(2 * s.most) * 8 * s.nt * c->head_dim);
  a.status = dev_status;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  switch (c->head_dim) {
    case 64: e = s.nt == 1 ? launch_attn<64, 1>(a, s.most, st) : launch_attn<64, 2>(a, s.most, st); break;
    case 128: e = s.nt == 1 ? launch_attn<128, 1>(a, s.most, st) : launch_attn<128, 2>(a, s.most, st); break;
    default: e = s.nt == 1 ? launch_attn<256, 1>(a, s.most, st) : launch_attn<256, 2>(a, s.most, st); break;
  }
  return cuda_status(e, "kv4 attention");
}

}  // extern "C"
