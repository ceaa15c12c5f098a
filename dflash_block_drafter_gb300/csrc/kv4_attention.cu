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
// carries the other factor: FP16 rows scaled by the power of two that brings their
// largest value into [2^15, 2^16), so that a value is off by 2^-36 of the row's
// largest at most.  A block's scale multiplies the finished FP32 sum of its 32
// channels.  The -8 of the codes is one more product, of a cell's scales with -8
// times the blocks' sums of q, each held as two FP16 terms: 22 bits, or as many as
// FP16's smallest step leaves, 2^-19 of the row's largest value.  K itself enters the
// scores without any rounding.
// O^T = V^T P^T.  Two cells' words are interleaved (prmt) into pairs along the
// cells, turned into code - 8 (1024 + c, minus 1032) and multiplied by the
// cells' scales in FP16: one rounding of 2^-11 at most relative to the value.
// P goes through movmatrix from the accumulator layout to the B operand's and is
// rounded to FP16 (2^-11 relative at most, 2^-32 of the largest weight absolute; the
// sums are FP32 of the unrounded p).
//
// Work: the 4 warps of a CTA take a tile of 128 cells together.  For S^T
// each warp has its own 32 cells and all channels; P goes through shared memory; for
// O^T each warp has its own quarter of the channels and all cells.  So O is 16
// registers per 8 rows at most, two or three CTAs fit an SM, and a segment ends
// without joining warps.  One barrier per tile orders P, the ring's stages and the
// vote on the maximum: the reference of a row's weights moves seldom (kKv4Slack), so
// that the first tile and few others pay for a rescaling.  Bulk copies of whole groups
// (K, V and scales together) run one or two tiles ahead, into the CTA's next segment too.
//
// (FP16 for P and V: the tensor cores' next wider type, TF32, has the same 11 bits at
// half the rate; more bits would mean two terms each, twice the products.)
//
// Measured: 16 single tokens of 24 / 2 heads of 256 over 2048 .. 32768 cells 55 us for
// 162 MB (2.9 TB/s), 200 of 32 / 8 heads of 128 over 1 .. 2047 cells 78 us for 224 MB, 64
// blocks of 8 rows of 32 / 8 heads of 128 over 512 .. 8192 cells 182 us for 358 MB.
// The chains of unpacking and products of the two or three warps per scheduler bound
// it (about half of the issue slots are used), not the copies: one per tile instead of
// four, or deeper rings, change nothing; eight warps on a tile, four per scheduler,
// with 128 registers each take 64 and 104 us.
#include <cstddef>

#include "kv4_attention.cuh"

namespace dflash {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kOverhead = 2;  // a segment's beginning and end, in tiles

constexpr int kPlanBytes(int n_seq) { return (n_seq + 1) * 8; }

template <int D, int NT>
struct Geo {
  static constexpr int R = 8 * NT;                 // query rows of a segment, at most
  static constexpr int MT = 2;                     // 16-cell groups of a warp in a tile
  static constexpr int GROUPS = kWarps * MT;
  static constexpr int TILE = 16 * GROUPS;         // cells of a tile
  static constexpr int STAGE = GROUPS * Kv4<D>::GROUP_BYTES;
  static constexpr int STAGES = D == 256 ? 2 : 3;
  // CTAs per SM: three, or two where three leave a thread too few registers.  Measured with
  // two and three on 64 blocks of 8 rows over 512 .. 8192 cells, 8 kv heads: 32 rows of
  // 128 channels 183 and 220 us (508 bytes of spill loads), 24 rows 160 and 153; 32 rows of
  // 64 channels 139 and 128, 24 rows 122 and 110.  (256 channels: shared memory for two.)
  static constexpr int PER_SM = D == 256 || (D == 128 && NT == 4) ? 2 : 3;
  static constexpr int RING = STAGES * STAGE;
  static constexpr int QF = NT * (D / 32) * 512;   // Q fragments
  static constexpr int QS = NT * 256;              // fragments of the blocks' sums
  static constexpr int P = GROUPS * NT * 256;      // P fragments of a tile, double-buffered
  static constexpr int SMEM = RING + QF + QS + 2 * P;
  static constexpr int JT = D / 64;                // 16-channel tiles of O^T that a warp owns
};

// D = A B and D += A B for one 16 x 8 tile.  Not volatile, like the plain loads
// below: the compiler may run a group's loads and unpacking under another's products.
__device__ __forceinline__ void mma_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ void mma_add(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix_t(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, (Geo<D, NT>::PER_SM)) kv4_attn_kernel(const Kv4AttnArgs a) {
  using F = Kv4<D>;
  using G = Geo<D, NT>;
  constexpr int R = G::R, B = F::BLOCKS, U = D / 64, ST = G::STAGES, MT = G::MT, TILE = G::TILE, JT = G::JT;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* ring = smem;
  uint8_t* qf = smem + G::RING;                                // [NT][B][32 lanes][16 B]
  __half* qsum = reinterpret_cast<__half*>(qf + G::QF);         // [NT][32 lanes][2 terms][2]
  uint8_t* pf = qf + G::QF + G::QS;                            // [2][GROUPS][NT][32 lanes][8 B]
  long long* pre = reinterpret_cast<long long*>(pf + 2 * G::P);  // [n_seq + 1]
  __shared__ long long scratch[kWarps];
  __shared__ uint64_t full[ST];
  __shared__ float s_factor[R];
  __shared__ float s_max[kWarps][R], s_sum[kWarps][R];
  __shared__ int2 s_sees[R];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) mbar_init(&full[i], kWarps);
    fence_barrier_init();
  }
  const long long T = kv4_plan<TILE, kOverhead>(a, pre, scratch, blockIdx.x == 0);
  const int C = kv4_ctas(T, gridDim.x);
  const int c = blockIdx.x;
  pdl_launch_dependents();
  if (c >= C || T == 0) {
    if (tid == 0) a.jobs[c].n_rows = 0;
    return;
  }
  const long long x_end = kv4_start(T, C, c + 1);

  const int groups_of_page = 1 << (a.page_shift - 4);
  // Word of the V chunk of channel group g that this lane takes, and its first pair of
  // channels there.  The word differs by g, so that the 8 groups of 4 cells, exchanged as
  // Kv4::v_swap says, lie in 32 different banks (the same word for all g: 4 ways of
  // conflicts at D 256, 2 at 128).
  const int u = (warp * JT / 4) ^ (D == 256 ? g >> 1 : D == 128 ? g >> 2 : 0), j0 = warp * JT % 4;
  const int cell_g = (g & 1) ? 7 - (g >> 1) : g >> 1;  // cell of S^T's row g (and 8 + cell_g of row g + 8)
  const Kv4Consts kc;
  const uint32_t per_g = kv4_per_token(a.G);
  uint32_t fills = 0;  // tiles that the ring has taken in earlier segments
  bool ok = true, job = false;

  // the lanes look up the pages of this warp's groups, 32 / MT tiles at a time (groups
  // that no row sees have no page: those before a window may have been given back)
  auto look_up = [&](const Kv4Part& p, int from) {
    const int i = from + lane / MT;
    const int pos = p.q.base + (p.k0 + i) * TILE + (warp * MT + lane % MT) * 16;
    if (i >= p.n || pos + 16 <= p.q.lo || pos >= p.q.hi) return -1;
    int page = a.table[static_cast<long long>(p.s) * a.table_stride + (pos >> a.page_shift)];
    if (page < 0 || page >= a.n_pages) {
      set_status(a.status, DFLASH_DEV_CAPACITY);
      page = 0;
    }
    return page;
  };
  // copies this warp's groups of tile i of a part as the ring's fill `fill`
  auto issue = [&](const Kv4Part& p, int i, uint32_t fill, int pages) {
    const int st = fill % ST;
    int page[MT], bytes = 0;
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      page[j] = __shfl_sync(0xffffffffu, pages, i % (32 / MT) * MT + j);
      bytes += page[j] >= 0 ? F::GROUP_BYTES : 0;
    }
    if (lane == 0) {
      mbar_arrive_expect_tx(&full[st], bytes);
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const int gi = warp * MT + j;
        const int grp = ((p.q.base + (p.k0 + i) * TILE + gi * 16) >> 4) & (groups_of_page - 1);
        if (page[j] >= 0)
          bulk_g2s(ring + st * G::STAGE + gi * F::GROUP_BYTES,
                   a.cache + ((static_cast<size_t>(page[j]) * a.n_kv + p.head) * groups_of_page + grp) * F::GROUP_BYTES,
                   F::GROUP_BYTES, &full[st]);
      }
    }
  };

  Kv4Part cur = kv4_part<TILE, kOverhead>(a, pre, kv4_start(T, C, c), x_end, Kv4Part{});
  int pages = look_up(cur, 0);
  int issued = 0;  // tiles of the current part that are on their way
  for (; issued < min(cur.n, ST); ++issued) issue(cur, issued, issued, pages);
  while (cur.n > 0) {
    const Kv4Seq q = cur.q;
    const int k0 = cur.k0, k1 = cur.k0 + cur.n, head = cur.head;
    const int n_rows = cur.rows;
    const int n = ok ? cur.n : 0;  // tiles
    // the next part's first tiles follow this one's last without a gap
    const Kv4Part next = kv4_part<TILE, kOverhead>(a, pre, cur.next, x_end, cur);
    int next_pages = look_up(next, 0);
    int next_issued = 0;
    __syncthreads();  // the last segment is done with Q and P

    // ---- Q: 8 threads a row find its maximum, scale it and lay out the fragments
    for (int m = tid >> 3; m < R; m += kThreads / 8) {
      constexpr int E = D / 8;  // channels of a thread, consecutive
      const int part = tid & 7;
      float v[E];
      float top = 0.f;
      if (m < n_rows) {
        const uint16_t* src = a.q + q.r0 * a.q_stride + kv4_token(m, per_g) * (a.q_stride - a.G * D) + (head * a.G + m) * D + part * E;
#pragma unroll
        for (int e = 0; e < E; e += 8) {
          const uint4 raw = *reinterpret_cast<const uint4*>(src + e);
          const uint32_t pr[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (a.bf16) {
              v[e + 2 * j] = __uint_as_float(pr[j] << 16);
              v[e + 2 * j + 1] = __uint_as_float(pr[j] & 0xffff0000u);
            } else {
              const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&pr[j]));
              v[e + 2 * j] = x.x;
              v[e + 2 * j + 1] = x.y;
            }
            top = fmaxf(top, fmaxf(fabsf(v[e + 2 * j]), fabsf(v[e + 2 * j + 1])));
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = 0.f;
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      // power of two that brings the row's maximum into [2^15, 2^16) (a BF16 or FP16 value's
      // bits reach FP16's largest there, 65504, and do not pass it)
      const int ex = static_cast<int>(__float_as_uint(top) >> 23);
      const int up = top > 0.f ? min(15 + 127 - ex, 120) : 0;
      auto power = [](int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); };
      const float f = power(up);
      if (part == 0) {
        // (beyond 2^100 any two scores that differ are too far apart to share weight)
        s_factor[m] = fminf(a.scale_log2 * power(-up) * 0x1p24f, 0x1p100f);
        s_sees[m] = m < n_rows ? kv4_sees(a, q, kv4_token(m, per_g)) : make_int2(0, 0);
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
      }
      // -8 2^-24 times the block's sum, in two terms: term h of block b is row
      // 8 h + b of the product's B operand, held by lane (m % 8, b / 2)
      if constexpr (E < 32) {  // 32 / E threads share a block
#pragma unroll
        for (int o = 1; o < 32 / E; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      }
      __half* at = qsum + ((m >> 3) * 32 + (m & 7) * 4) * 4;
      if (part % (32 / E) == 0) {
        const int b = part * E / 32;
        const float v8 = sum * (-8.f / 16777216.f);
        const __half hi = __float2half_rn(v8);
        at[(b >> 1) * 4 + (b & 1)] = hi;
        at[(b >> 1) * 4 + 2 + (b & 1)] = __float2half_rn(v8 - __half2float(hi));
      } else {  // rows of no block
        const int b = B + part - part * E / 32 - 1;
        at[(b >> 1) * 4 + (b & 1)] = at[(b >> 1) * 4 + 2 + (b & 1)] = __ushort_as_half(0);
      }
    }
    __syncthreads();

    float o[JT][NT][4];
#pragma unroll
    for (int j = 0; j < JT; ++j)
#pragma unroll
      for (int n2 = 0; n2 < NT; ++n2)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][n2][e] = 0.f;
    // of rows 8 n2 + 2t + e: reference, sum over this lane's cells, factor
    float m_ref[NT][2], l_run[NT][2], fac[NT][2];
    int all_lo = 0, all_hi = 0x7fffffff;  // cells that every row sees
#pragma unroll
    for (int n2 = 0; n2 < NT; ++n2)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int m = n2 * 8 + 2 * t + e;
        m_ref[n2][e] = -INFINITY;
        l_run[n2][e] = 0.f;
        fac[n2][e] = s_factor[m];
        if (m < n_rows) {
          all_lo = max(all_lo, s_sees[m].x);
          all_hi = min(all_hi, s_sees[m].y);
        }
      }
#pragma unroll
    for (int w = 1; w < 4; w <<= 1) {
      all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, w));
      all_hi = min(all_hi, __shfl_xor_sync(0xffffffffu, all_hi, w));
    }

    for (int i = 0; i < n; ++i) {
      const uint32_t fill = fills + i;
      const int st = fill % ST;
      const bool late = !kv4_wait(&full[st], (fill / ST) & 1);
      const uint8_t* base = ring + st * G::STAGE;
      const int pos0 = q.base + (k0 + i) * TILE;
      const bool edge = pos0 < all_lo || pos0 + TILE > all_hi;
      // the lane's words and scales of cells cell_g and 8 + cell_g
      uint32_t wa[MT][B], wb[MT][B], da[MT][B / 2], db[MT][B / 2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const uint8_t* gb = base + (warp * MT + mt) * F::GROUP_BYTES;
#pragma unroll
        for (int h = 0; h < (B + 3) / 4; ++h) {
          constexpr int N = B < 4 ? B : 4;
          uint32_t tmp[N];
          const uint8_t* at = gb + cell_g * F::ROW + 4 * ((t * B + 4 * h) ^ F::k_swap(cell_g));
          load_words<N>(at, tmp);
#pragma unroll
          for (int e = 0; e < N; ++e) wa[mt][4 * h + e] = tmp[e];
          // cell 8 + cell_g: k_swap goes by bit 2 of the cell, the same
          load_words<N>(at + 8 * F::ROW, tmp);
#pragma unroll
          for (int e = 0; e < N; ++e) wb[mt][4 * h + e] = tmp[e];
        }
        load_words<B / 2>(gb + F::K_SCALES + cell_g * F::SROW, da[mt]);
        load_words<B / 2>(gb + F::K_SCALES + (cell_g + 8) * F::SROW, db[mt]);
      }
      // ---- S^T of this warp's cells, from the codes' -8 (scales of blocks 2t, 2t + 1)
      float sc[MT][NT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const uint8_t* at = base + (warp * MT + mt) * F::GROUP_BYTES + F::K_SCALES + cell_g * F::SROW + 4 * t;
        uint32_t s0 = 0, s1 = 0;
        if (2 * t < B) {
          s0 = *reinterpret_cast<const uint32_t*>(at);
          s1 = *reinterpret_cast<const uint32_t*>(at + 8 * F::SROW);
        }
#pragma unroll
        for (int n2 = 0; n2 < NT; ++n2) {
          const uint2 qs = *reinterpret_cast<const uint2*>(qsum + (n2 * 32 + lane) * 4);
          mma_zero(sc[mt][n2], s0, s1, s0, s1, qs.x, qs.y);
        }
      }
#pragma unroll
      for (int b = 0; b < B; ++b) {
#pragma unroll
        for (int n2 = 0; n2 < NT; ++n2) {
          const uint4 bq = *reinterpret_cast<const uint4*>(qf + ((n2 * B + b) * 32 + lane) * 16);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const __half2 ha = *reinterpret_cast<const __half2*>(&da[mt][b >> 1]);
            const __half2 hb = *reinterpret_cast<const __half2*>(&db[mt][b >> 1]);
            const float fa = (b & 1) ? __high2float(ha) : __low2float(ha);
            const float fb = (b & 1) ? __high2float(hb) : __low2float(hb);
            const uint32_t ua = wa[mt][b], ub = wb[mt][b], va = ua >> 8, vb = ub >> 8;
            float acc[4];
            mma_zero(acc, ua & 0x000f000fu, ub & 0x000f000fu, ua & 0x00f000f0u, ub & 0x00f000f0u, bq.x, bq.y);
            mma_add(acc, va & 0x000f000fu, vb & 0x000f000fu, va & 0x00f000f0u, vb & 0x00f000f0u, bq.z, bq.w);
            sc[mt][n2][0] = fmaf(fa, acc[0], sc[mt][n2][0]);
            sc[mt][n2][1] = fmaf(fa, acc[1], sc[mt][n2][1]);
            sc[mt][n2][2] = fmaf(fb, acc[2], sc[mt][n2][2]);
            sc[mt][n2][3] = fmaf(fb, acc[3], sc[mt][n2][3]);
          }
        }
      }
      // ---- scores in log2 units; does any pass its row's reference by too much?
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n2 = 0; n2 < NT; ++n2)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[mt][n2][e] *= fac[n2][e & 1];
      if (edge) {
        // cells that a row does not see
#pragma unroll
        for (int n2 = 0; n2 < NT; ++n2)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int2 sees = s_sees[n2 * 8 + 2 * t + (e & 1)];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              const int pos = pos0 + (warp * MT + mt) * 16 + cell_g + (e >> 1) * 8;
              if (pos < sees.x || pos >= sees.y) sc[mt][n2][e] = -INFINITY;
            }
          }
        // and cells that none sees may hold anything: no weight times NaN, so
        // their V scales become 0 (the barrier below orders it before the reads)
        for (int j = lane; j < MT * 16 * (F::SROW / 4); j += 32) {
          const int cell = j / (F::SROW / 4), pos = pos0 + warp * MT * 16 + cell;
          if (pos < q.lo || pos >= q.hi)
            *reinterpret_cast<uint32_t*>(ring + st * G::STAGE + (warp * MT + cell / 16) * F::GROUP_BYTES + F::V_SCALES +
                                         (cell % 16) * F::SROW + j % (F::SROW / 4) * 4) = 0;
        }
        fence_proxy_async_smem();  // the stage's next copy comes after these writes
      }
      bool over = false;
#pragma unroll
      for (int n2 = 0; n2 < NT; ++n2)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = fmaxf(sc[0][n2][e], sc[0][n2][2 + e]);
#pragma unroll
          for (int mt = 1; mt < MT; ++mt) v = fmaxf(v, fmaxf(sc[mt][n2][e], sc[mt][n2][2 + e]));
          over |= v > m_ref[n2][e] + kKv4Slack;
        }
      uint8_t* pt = pf + (i & 1) * G::P;
      auto write_p = [&](float (&sum)[NT][2]) {
#pragma unroll
        for (int n2 = 0; n2 < NT; ++n2) {
          const float f0 = m_ref[n2][0] == -INFINITY ? 0.f : m_ref[n2][0];
          const float f1 = m_ref[n2][1] == -INFINITY ? 0.f : m_ref[n2][1];
          sum[n2][0] = sum[n2][1] = 0.f;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const float p0 = ex2_approx(sc[mt][n2][0] - f0), p1 = ex2_approx(sc[mt][n2][1] - f1);
            const float p2 = ex2_approx(sc[mt][n2][2] - f0), p3 = ex2_approx(sc[mt][n2][3] - f1);
            sum[n2][0] += p0 + p2;
            sum[n2][1] += p1 + p3;
            *reinterpret_cast<uint2*>(pt + (((warp * MT + mt) * NT + n2) * 32 + lane) * 8) =
                make_uint2(movmatrix_t(pack_f16x2(p0, p1)), movmatrix_t(pack_f16x2(p2, p3)));
          }
        }
      };
      float sum[NT][2];
      write_p(sum);
      if (__syncthreads_or(over || late)) {
        if (__syncthreads_or(late)) {
          // a copy did not come in time: nothing more is issued or computed; what
          // is in flight lands before the CTA ends
          for (int j = i; j < issued + next_issued; ++j) kv4_wait(&full[(fills + j) % ST], ((fills + j) / ST) & 1);
          if (tid == 0) set_status(a.status, DFLASH_DEV_TIMEOUT);
          ok = false;
          break;
        }
        // new references: the rows' maxima so far over all warps
        float top[NT][2];
#pragma unroll
        for (int n2 = 0; n2 < NT; ++n2)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = -INFINITY;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) v = fmaxf(v, fmaxf(sc[mt][n2][e], sc[mt][n2][2 + e]));
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, w));
            top[n2][e] = v;
            if (g == 0) s_max[warp][n2 * 8 + 2 * t + e] = v;
          }
        __syncthreads();
#pragma unroll
        for (int n2 = 0; n2 < NT; ++n2)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = m_ref[n2][e];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v = fmaxf(v, s_max[w][n2 * 8 + 2 * t + e] - kKv4Lift);
            const float alpha = v == -INFINITY ? 0.f : ex2_approx(m_ref[n2][e] - v);
            m_ref[n2][e] = v;
            l_run[n2][e] *= alpha;
#pragma unroll
            for (int j = 0; j < JT; ++j) {
              o[j][n2][e] *= alpha;
              o[j][n2][2 + e] *= alpha;
            }
          }
        write_p(sum);
        __syncthreads();
      }
#pragma unroll
      for (int n2 = 0; n2 < NT; ++n2)
#pragma unroll
        for (int e = 0; e < 2; ++e) l_run[n2][e] += sum[n2][e];
      // every warp has finished the tile before: its stage takes a new one
      if (i > 0) {
        if (issued < n) {
          if (issued % (32 / MT) == 0) pages = look_up(cur, issued);
          issue(cur, issued, fills + issued, pages);
          ++issued;
        } else if (next_issued < min(next.n, 32 / MT)) {
          issue(next, next_issued, fills + n + next_issued, next_pages);
          ++next_issued;
        }
      }
      // ---- O^T: cells t, 7 - t and 8 + t, 15 - t of each group, this warp's channels
#pragma unroll
      for (int gi = 0; gi < G::GROUPS; ++gi) {
        const uint8_t* gb = base + gi * F::GROUP_BYTES;
        uint32_t vw[4], vs[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int cell = (k & 1 ? 7 - t : t) + (k >> 1) * 8;
          vw[k] = *reinterpret_cast<const uint32_t*>(gb + F::V_CODES + cell * F::ROW + 4 * (U * (g ^ F::v_swap(cell)) + u));
          vs[k] = *reinterpret_cast<const uint16_t*>(gb + F::V_SCALES + cell * F::SROW + ((g >> 2) * U + u) * 2);
        }
        const uint32_t d0 = prmt(vs[0], vs[1], 0x5410), d1 = prmt(vs[2], vs[3], 0x5410);
        uint2 pb[NT];
#pragma unroll
        for (int n2 = 0; n2 < NT; ++n2)
          pb[n2] = *reinterpret_cast<const uint2*>(pt + ((gi * NT + n2) * 32 + lane) * 8);
        uint32_t lo[2], hi[2];
        if constexpr (JT == 4) {
          lo[0] = prmt(vw[0], vw[1], 0x5410), hi[0] = prmt(vw[2], vw[3], 0x5410);
          lo[1] = prmt(vw[0], vw[1], 0x7632), hi[1] = prmt(vw[2], vw[3], 0x7632);
        } else {
          const uint32_t sel = j0 >= 2 ? 0x7632u : 0x5410u;
          lo[0] = prmt(vw[0], vw[1], sel), hi[0] = prmt(vw[2], vw[3], sel);
          if (JT == 1 && (j0 & 1)) lo[0] >>= 8, hi[0] >>= 8;
        }
#pragma unroll
        for (int j = 0; j < JT; ++j) {  // channels 64u + 8g + 2 (j0 + j), + 1
          const uint32_t l = (j & 1) ? lo[j >> 1] >> 8 : lo[j >> 1], h = (j & 1) ? hi[j >> 1] >> 8 : hi[j >> 1];
          const uint32_t a0 = hmul2_u32(kc.even(l), d0), a1 = hmul2_u32(kc.odd(l), d0);
          const uint32_t a2 = hmul2_u32(kc.even(h), d1), a3 = hmul2_u32(kc.odd(h), d1);
#pragma unroll
          for (int n2 = 0; n2 < NT; ++n2) mma_add(o[j][n2], a0, a1, a2, a3, pb[n2].x, pb[n2].y);
        }
      }
    }
    fills += n;
    // (the last tile's stage is free once every warp is behind the barrier below)
    // ---- the rows' sums over all warps
#pragma unroll
    for (int n2 = 0; n2 < NT; ++n2)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l_run[n2][e] += __shfl_xor_sync(0xffffffffu, l_run[n2][e], w);
        if (g == 0) s_sum[warp][n2 * 8 + 2 * t + e] = l_run[n2][e];
      }
    __syncthreads();
    if (ok) {
      for (; next_issued < min(next.n, ST); ++next_issued) issue(next, next_issued, fills + next_issued, next_pages);
    }
    const bool whole = k0 == 0 && k1 == q.steps;
    const int slot = 2 * c + (k0 == 0 ? 1 : 0);
    const int col = 64 * u + 8 * g + 2 * j0;
#pragma unroll
    for (int n2 = 0; n2 < NT; ++n2)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int m = n2 * 8 + 2 * t + e;
        if (m >= n_rows) continue;
        float l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) l += s_sum[w][m];
        float f = 1.f;
        if (whole) {
          f = l > 0.f ? 1.f / l : 0.f;
          if (!(l < INFINITY)) set_status(a.status, DFLASH_DEV_NONFINITE);
          uint16_t* dst = a.out + q.r0 * a.out_stride + kv4_token(m, per_g) * (a.out_stride - a.G * D) + (head * a.G + m) * D + col;
          uint32_t w[JT];
#pragma unroll
          for (int j = 0; j < JT; ++j)
            w[j] = a.bf16 ? pack_bf16x2(o[j][n2][e] * f, o[j][n2][2 + e] * f) : pack_f16x2(o[j][n2][e] * f, o[j][n2][2 + e] * f);
          if constexpr (JT == 4) *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
          else if constexpr (JT == 2) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
          else *reinterpret_cast<uint32_t*>(dst) = w[0];
        } else {
          float* dst = a.part + (static_cast<size_t>(slot) * R + m) * D + col;
#pragma unroll
          for (int j = 0; j < JT; ++j) __stcg(reinterpret_cast<float2*>(dst) + j, make_float2(o[j][n2][e], o[j][n2][2 + e]));
          if (warp == 0 && g == 0) __stcg(a.part_ml + static_cast<size_t>(slot) * R + m, make_float2(m_ref[n2][e], l));
        }
      }
    if (!whole && k0 == 0) {  // the segment goes on in the next CTAs
      job = true;
      if (tid == 0) {
        a.jobs[c] = Kv4Job{q.r0, head, n_rows, kv4_owner(T, C, cur.end - 1)};
      }
    }
    cur = next;
    pages = next_pages;
    issued = next_issued;
  }
  if (!job && tid == 0) a.jobs[c].n_rows = 0;
}

template <int D, int NT>
cudaError_t launch_attn(const Kv4AttnArgs& a, int most, int jobs, cudaStream_t st) {
  using G = Geo<D, NT>;
  cudaError_t e = cudaFuncSetAttribute(kv4_attn_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       G::SMEM + kPlanBytes(kKv4MaxSeq));
  if (e != cudaSuccess) return e;
  kv4_attn_kernel<D, NT><<<most, kThreads, G::SMEM + kPlanBytes(a.n_seq), st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || most == 1) return e;
  return launch_kv4_merge<D, G::R>(a, most, jobs, st);
}

// Shared memory of an SM, and what a CTA takes of it besides its dynamic part
// (its static arrays and the system's 1 KB).
constexpr int kSmemOfSm = 228 * 1024, kStaticSmem = 2560;
struct CtaCost {
  int smem, per_sm;
};
CtaCost cost_of(int d, int nt) {
  switch (d * 8 + nt) {
#define DFLASH_KV4_COST(D, NT) \
  case D * 8 + NT: return {Geo<D, NT>::SMEM, Geo<D, NT>::PER_SM};
#define DFLASH_KV4_COSTS(D) \
  DFLASH_KV4_COST(D, 1) DFLASH_KV4_COST(D, 2) DFLASH_KV4_COST(D, 3) DFLASH_KV4_COST(D, 4)
    DFLASH_KV4_COSTS(64)
    DFLASH_KV4_COSTS(128)
    DFLASH_KV4_COSTS(256)
#undef DFLASH_KV4_COSTS
#undef DFLASH_KV4_COST
  }
  return {kSmemOfSm, 1};
}

// What the host knows of a call: its kernel, CTAs and split segments at most.
struct Shape {
  bool tc;    // the tcgen05 kernel: up to 128 query rows a segment
  int nt;     // else: 8-row tiles of them
  int most, jobs;
  int rows() const { return tc ? 128 : 8 * nt; }
};
// More rows per kv head than this go to the tcgen05 kernel.  Measured, here and there:
//   16 sequences of 2048 .. 32768 cells, 2 kv heads of 256: 12 rows 58 and 98 us, 24 rows
//   81 and 100, 32 rows 91 and 101 (floor 25);
//   64 of 512 .. 8192 cells, 8 kv heads of 128: 24 rows 154 and 255, 32 rows 182 and 255
//   (floor 53); of 64: 24 rows 110 and 164, 32 rows 128 and 164 (floor 26).
// Beyond, a kernel of this kind would unpack every cell once per 32 rows.
constexpr int kTcRows = 32;
cudaError_t shape_of(const dflash_kv4_cache* c, int n_q_heads, int n_seq, int max_rows, int table_stride, Shape* out) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int rows = n_q_heads / c->n_kv_heads * max_rows;
  out->tc = rows > kTcRows;
  if (out->tc) {
    out->nt = 0;
    const long long segments = static_cast<long long>(n_seq) * c->n_kv_heads;
    const int tile = c->head_dim == 256 ? 64 : 128;
    const long long tiles = (static_cast<long long>(table_stride) * c->page_size + tile - 1) / tile + 1;
    out->most = static_cast<int>(segments * tiles < sms ? segments * tiles : sms);
    out->jobs = static_cast<int>(segments < out->most ? segments : out->most);
    return cudaSuccess;
  }
  out->nt = (rows + 7) / 8;
  const int tile = 128;
  const long long segments = static_cast<long long>(n_seq) * c->n_kv_heads;
  // (a window may begin anywhere in a tile)
  const long long tiles = (static_cast<long long>(table_stride) * c->page_size + tile - 1) / tile + 1;
  const long long ctas = segments * (tiles + kOverhead);
  // one wave of CTAs: every one of them has the same share
  const CtaCost cost = cost_of(c->head_dim, out->nt);
  const int fit = kSmemOfSm / (cost.smem + kPlanBytes(n_seq) + kStaticSmem);
  const int per_sm = fit < cost.per_sm ? fit : cost.per_sm;
  out->most = static_cast<int>(ctas < per_sm * sms ? ctas : per_sm * sms);
  out->jobs = static_cast<int>(segments < out->most ? segments : out->most);
  return cudaSuccess;
}

int check_call(const dflash_kv4_cache* c, int n_q_heads, int n_seq, int max_rows, int table_stride) {
  if (const int e = dflash_kv4_check(c)) return e;
  if (n_seq < 1 || table_stride < 1 || n_q_heads < 1 || n_q_heads % c->n_kv_heads) return DFLASH_ERR_INVALID_ARG;
  if (max_rows < 1 || max_rows > DFLASH_MAX_BLOCK) return DFLASH_ERR_INVALID_ARG;
  // (positions up to a tile behind the table's last stay within 31 bits)
  if (n_seq > kKv4MaxSeq || static_cast<long long>(table_stride) * c->page_size > 0x7fffff00ll) return DFLASH_ERR_CAPACITY;
  if (n_q_heads / c->n_kv_heads * max_rows > 128) return DFLASH_ERR_UNSUPPORTED;
  return DFLASH_OK;
}

size_t bytes_of(const dflash_kv4_cache* c, const Shape& s) {
  return s.most * (sizeof(Kv4Job) + 2 * size_t(s.rows()) * (c->head_dim * 4 + 8));
}

template <int D>
cudaError_t launch_nt(const Kv4AttnArgs& a, const Shape& s, cudaStream_t st) {
  switch (s.nt) {
    case 1: return launch_attn<D, 1>(a, s.most, s.jobs, st);
    case 2: return launch_attn<D, 2>(a, s.most, s.jobs, st);
    case 3: return launch_attn<D, 3>(a, s.most, s.jobs, st);
    default: return launch_attn<D, 4>(a, s.most, s.jobs, st);
  }
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
  // (2^127: its product with log2(e) is still finite)
  if (n_tokens < 0 || window < 0 || !(scale > 0.f) || !(scale <= 0x1p127f)) return DFLASH_ERR_INVALID_ARG;
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
  a.jobs = static_cast<Kv4Job*>(workspace);
  a.part = reinterpret_cast<float*>(a.jobs + s.most);
  a.part_ml = reinterpret_cast<float2*>(a.part + static_cast<size_t>(2 * s.most) * s.rows() * c->head_dim);
  a.status = dev_status;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (s.tc) {
    e = launch_kv4_attn_tc(c->head_dim, a, s.most, s.jobs, st);
  } else {
    switch (c->head_dim) {
      case 64: e = launch_nt<64>(a, s, st); break;
      case 128: e = launch_nt<128>(a, s, st); break;
      default: e = launch_nt<256>(a, s, st); break;
    }
  }
  return cuda_status(e, "kv4 attention");
}

}  // extern "C"
