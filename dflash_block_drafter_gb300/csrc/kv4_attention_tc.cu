// Attention over the 4-bit paged K/V cache for many query rows per kv head
// (blocks of several tokens over wide groups), on the tcgen05 tensor cores.
//
// One CTA per SM takes tiles of 64 cells for up to 128 query rows:
//   warp 0        copies the tiles' packed groups into a ring (bulk copies);
//   warps 10..17  unpack a tile once for all rows: K and V as FP16
//                 d (code - 8), in the 128-byte-swizzled layouts the MMAs read,
//                 double-buffered;
//   warp 1        issues S = Q K^T (M 128, N 64) and O += P V (M 128, N = D);
//   warps 2..9    softmax: a thread has one row (TMEM lane) and 32 of the
//                 tile's 64 cells.
// Q and P are the MMAs' A operands in tensor memory (FP16 pairs), so shared
// memory carries only K and V: per tile and D = 256 64 KB written and read
// (about 1000 cycles of its bandwidth, as many as the MMAs take), against 790
// cycles for the tile's bytes from HBM.  P lies over the S it came from; the columns are
// S0 | S1 | O | Q = 64 + 64 + D + D / 2.
//
// The 8 channels of a code word lie in the order 0 4 1 5 2 6 3 7, in which
// masking the word yields pairs: Q's columns are stored in the same order,
// and O's are read back in it.
// Roundings: K, V and P to FP16 (2^-11 relative each, P 2^-25 absolute), Q exact (rows
// scaled by a power of two); scores, sums and O in FP32.  Scores are taken
// relative to a reference that moves only when a row passes it by 2^8.
#include "kv4_attention.cuh"

namespace dflash {
namespace {

constexpr int kTile = 64;       // cells of a tile
constexpr int kGroups = 4;
constexpr int kRows = 128;
constexpr int kSoftWarps = 8, kUnpackWarps = 8;
constexpr int kThreads = 32 * (2 + kSoftWarps + kUnpackWarps);
constexpr int kSoftThreads = 32 * kSoftWarps;
constexpr int kPacked = 4;      // stages of the packed ring
constexpr int kTmemCols = 512;
constexpr float kSlack = 8.f;   // log2 units by which a score may pass the reference

template <int D>
struct Geo {
  static constexpr int STAGE = kGroups * Kv4<D>::GROUP_BYTES;
  static constexpr int BUF = kTile * D * 2;  // one unpacked K or V tile
  static constexpr int RED = (2 * 2 * kRows + 2 * kRows) * 4;
  static constexpr int SMEM = 1024 + 4 * BUF + kPacked * STAGE + RED;
  static constexpr int S_COL = 0, O_COL = 2 * kTile, Q_COL = O_COL + D;
};

// D[tmem] (+)= A[tmem] * B[smem desc], kind::f16, one CTA.
__device__ __forceinline__ void umma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&w)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "r"(w[8]), "r"(w[9]),
      "r"(w[10]), "r"(w[11]), "r"(w[12]), "r"(w[13]), "r"(w[14]), "r"(w[15])
      : "memory");
}

// One code word times its block's scale (twice in d): 8 FP16 in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ uint4 unpack(uint32_t w, uint32_t d) {
  constexpr uint32_t ONE = 0x3c003c00u, MINUS_1032 = 0xe408e408u, SIXTEENTH = 0x2c002c00u, MINUS_72 = 0xd480d480u;
  constexpr uint32_t BASE = 0x64006400u;  // 1024: the code lies in the low mantissa bits
  const uint32_t v = w >> 8;
  uint4 r;
  r.x = hmul2_u32(hfma2_u32((w & 0x000f000fu) | BASE, ONE, MINUS_1032), d);
  r.y = hmul2_u32(hfma2_u32((w & 0x00f000f0u) | BASE, SIXTEENTH, MINUS_72), d);
  r.z = hmul2_u32(hfma2_u32((v & 0x000f000fu) | BASE, ONE, MINUS_1032), d);
  r.w = hmul2_u32(hfma2_u32((v & 0x00f000f0u) | BASE, SIXTEENTH, MINUS_72), d);
  return r;
}

// N consecutive words (1, 2 or 4) of shared memory, and N consecutive FP16 as N pairs of equals.
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  }
}
template <int N>
__device__ __forceinline__ void load_scales(const uint8_t* p, uint32_t (&d)[N]) {
  if constexpr (N == 1) {
    const uint32_t h = *reinterpret_cast<const uint16_t*>(p);
    d[0] = prmt(h, h, 0x1010u);
  } else {
    uint32_t w[N / 2];
    load_words<N / 2>(p, w);
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = prmt(w[i >> 1], w[i >> 1], (i & 1) ? 0x3232u : 0x1010u);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv4_attn_tc_kernel(const Kv4AttnArgs a) {
  using F = Kv4<D>;
  using G = Geo<D>;
  constexpr int R = kRows, NP = kPacked, U = D / 64, B = D / 32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* kbuf = smem;                       // [2][D / 64 boxes][64 cells][128 B]
  uint8_t* vbuf = kbuf + 2 * G::BUF;          // [2]
  uint8_t* ring = vbuf + 2 * G::BUF;          // [NP] packed tiles
  float* red_max = reinterpret_cast<float*>(ring + NP * G::STAGE);  // [2][2 halves][128 rows]
  float* red_sum = red_max + 2 * 2 * R;                             // [2 halves][128 rows]
  long long* pre = reinterpret_cast<long long*>(red_sum + 2 * R);   // [n_seq + 1]
  __shared__ long long scratch[kThreads / 32];
  __shared__ uint64_t pfull[NP], pfree[NP], kready[2], kfree[2], vready[2], vfree[2], sfull[2], pready[2], qready, ofree, mdone;
  __shared__ uint32_t s_tmem;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < NP; ++i) {
      mbar_init(&pfull[i], 1);
      mbar_init(&pfree[i], kUnpackWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&kready[i], kUnpackWarps);
      mbar_init(&kfree[i], 1);
      mbar_init(&vready[i], kUnpackWarps);
      mbar_init(&vfree[i], 1);
      mbar_init(&sfull[i], 1);
      mbar_init(&pready[i], kSoftWarps);
    }
    mbar_init(&qready, kSoftWarps);
    mbar_init(&ofree, kSoftWarps);
    mbar_init(&mdone, 1);
    fence_barrier_init();
  }
  const long long T = kv4_plan<kTile, R>(a, pre, scratch, blockIdx.x == 0);
  const int C = kv4_ctas(T, gridDim.x, 1);
  const int c = blockIdx.x;
  pdl_launch_dependents();
  if (c >= C || T == 0) {
    if (tid == 0) a.jobs[c].n_rows = 0;
    return;
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const long long x_begin = kv4_start(T, C, c), x_end = kv4_start(T, C, c + 1);
  bool ok = true;

  // a segment's part in this CTA: tiles [k0, k0 + n) of a sequence, kv head and row group
  struct Part {
    Kv4Seq q;
    int s, head, row0, k0, n, rows;
  };
  auto part_at = [&](long long at) {
    Part p{};
    if (at >= x_end) return p;
    p.s = kv4_find(pre, a.n_seq, at);
    p.q = kv4_seq<kTile, R>(a, p.s, false);
    const long long rel = at - pre[p.s];
    const int unit = static_cast<int>(rel / p.q.steps);
    p.k0 = static_cast<int>(rel - static_cast<long long>(unit) * p.q.steps);
    p.n = static_cast<int>(min(static_cast<long long>(p.q.steps - p.k0), x_end - at));
    p.head = unit / p.q.groups;
    p.row0 = unit % p.q.groups * R;
    p.rows = min(R, p.q.rows * a.G - p.row0);
    return p;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const int groups_of_page = 1 << (a.page_shift - 4);
    uint32_t g = 0;  // tiles over all parts
    for (long long x = x_begin; x < x_end && ok;) {
      const Part p = part_at(x);
      x += p.n;
      int page = -1;
      for (int i = 0; i < p.n && ok; ++i, ++g) {
        if (i % 8 == 0) {  // the lanes look up the groups of 8 tiles
          const int ii = i + (lane >> 2);
          const int pos = p.q.base + (p.k0 + ii) * kTile + (lane & 3) * 16;
          page = -1;
          if (ii < p.n && pos < p.q.hi) {
            page = a.table[static_cast<long long>(p.s) * a.table_stride + (pos >> a.page_shift)];
            if (page < 0 || page >= a.n_pages) {
              set_status(a.status, DFLASH_DEV_CAPACITY);
              page = 0;
            }
          }
        }
        const int st = g % NP;
        if (g >= NP) ok = __all_sync(0xffffffffu, mbar_wait(&pfree[st], (g / NP - 1) & 1));
        if (!ok) break;
        const int mine = __shfl_sync(0xffffffffu, page, (i % 8) * 4 + (lane & 3));
        const unsigned have = __ballot_sync(0xffffffffu, lane < kGroups && mine >= 0);
        if (lane == 0) mbar_arrive_expect_tx(&pfull[st], __popc(have) * F::GROUP_BYTES);
        __syncwarp();
        if (lane < kGroups && mine >= 0) {
          const int grp = ((p.q.base + (p.k0 + i) * kTile + lane * 16) >> 4) & (groups_of_page - 1);
          bulk_g2s(ring + st * G::STAGE + lane * F::GROUP_BYTES,
                   a.cache + ((static_cast<size_t>(mine) * a.n_kv + p.head) * groups_of_page + grp) * F::GROUP_BYTES,
                   F::GROUP_BYTES, &pfull[st]);
        }
      }
    }
    // every copy lands before the CTA ends
    for (uint32_t i = g < NP ? 0 : g - NP; i < g; ++i)
      if (!mbar_wait(&pfull[i % NP], (i / NP) & 1)) ok = false;
    if (!ok && lane == 0) set_status(a.status, DFLASH_DEV_TIMEOUT);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc_qk = umma_idesc_f16(128, kTile, false, false);
      constexpr uint32_t idesc_pv = umma_idesc_f16(128, D, false, true);
      const uint32_t k_s = smem_u32(kbuf), v_s = smem_u32(vbuf);
      // S[g % 2] = Q K_g^T, once K_g is there and P of tile g - 2, which lies in the same columns, has been used
      auto issue_qk = [&](uint32_t g) -> bool {
        if (!mbar_wait(&kready[g & 1], (g >> 1) & 1)) return false;
        if (g >= 2 && !mbar_wait(&vfree[g & 1], ((g >> 1) - 1) & 1)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t db = umma_desc_sw128(k_s + (g & 1) * G::BUF + (kk >> 2) * (kTile * 128) + (kk & 3) * 32, 16, 1024);
          umma_f16_ta(tmem + G::S_COL + (g & 1) * kTile, tmem + G::Q_COL + kk * 8, db, idesc_qk, kk > 0);
        }
        umma_commit(&sfull[g & 1]);
        umma_commit(&kfree[g & 1]);
        return true;
      };
      uint32_t g = 0, part = 0;
      for (long long x = x_begin; x < x_end && ok; ++part) {
        const int n = part_at(x).n;
        x += n;
        if (!mbar_wait(&qready, part & 1)) ok = false;
        if (ok && !issue_qk(g)) ok = false;
        for (int i = 0; i < n && ok; ++i, ++g) {
          if (i + 1 < n && !issue_qk(g + 1)) ok = false;
          if (ok && i == 0 && part > 0 && !mbar_wait(&ofree, (part - 1) & 1)) ok = false;
          if (!ok || !mbar_wait(&vready[g & 1], (g >> 1) & 1) || !mbar_wait(&pready[g & 1], (g >> 1) & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk) {
            const uint64_t db = umma_desc_sw128(v_s + (g & 1) * G::BUF + kk * 2048, kTile * 128, 1024);
            umma_f16_ta(tmem + G::O_COL, tmem + G::S_COL + (g & 1) * kTile + kk * 8, db, idesc_pv, (i > 0 || kk > 0) ? 1u : 0u);
          }
          umma_commit(&vfree[g & 1]);
        }
      }
      // tensor memory may only be freed once every issued MMA has finished
      umma_commit(&mdone);
      if (!mbar_wait(&mdone, 0)) ok = false;
      if (!ok) set_status(a.status, DFLASH_DEV_TIMEOUT);
    }
  } else if (warp < 2 + kSoftWarps) {
    // ------------------------------------------------------------ softmax
    const int q4 = warp & 3, cs = (warp - 2) >> 2;  // TMEM lane quarter, half of the tile's cells (and of O's columns)
    const int m = q4 * 32 + lane;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
    uint32_t g = 0;
    for (long long x = x_begin; x < x_end;) {
      const Part p = part_at(x);
      x += p.n;
      const bool mine = m < p.rows, live = q4 * 32 < p.rows;  // the row; any row of the quarter
      const int row = p.row0 + m;
      const int2 sees = mine ? kv4_sees(a, p.q, row / a.G) : make_int2(0, 0);
      int all_lo = mine ? sees.x : 0, all_hi = mine ? sees.y : 0x7fffffff;  // cells that every row of the quarter sees
#pragma unroll
      for (int w = 1; w < 32; w <<= 1) {
        all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, w));
        all_hi = min(all_hi, __shfl_xor_sync(0xffffffffu, all_hi, w));
      }
      // ---- Q into tensor memory: half cs of the row's channels
      const uint16_t* src = a.q + (p.q.r0 + row / a.G) * a.q_stride + (p.head * a.G + row % a.G) * D + cs * (D / 2);
      auto value = [&](uint32_t h) { return a.bf16 ? __uint_as_float(h << 16) : __half2float(__ushort_as_half(static_cast<uint16_t>(h))); };
      float top = 0.f;
      if (mine) {
#pragma unroll 4
        for (int e = 0; e < D / 2; e += 8) {
          const uint4 r = *reinterpret_cast<const uint4*>(src + e);
          const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) top = fmaxf(top, fmaxf(fabsf(value(w[j] & 0xffffu)), fabsf(value(w[j] >> 16))));
        }
      }
      red_sum[cs * R + m] = top;
      named_bar_sync(1, kSoftThreads);
      top = fmaxf(red_sum[m], red_sum[R + m]);
      // power of two that brings the row's maximum into [2^12, 2^13)
      const int up = top > 0.f ? min(12 + 127 - static_cast<int>(__float_as_uint(top) >> 23), 120) : 0;
      const float f = ldexpf(1.f, up), factor = fmaxf(ldexpf(a.scale_log2, -up), 1.17549435e-38f);
      if (live) {
#pragma unroll 1
        for (int e = 0; e < D / 2; e += 32) {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint4 r = make_uint4(0, 0, 0, 0);
            if (mine) r = *reinterpret_cast<const uint4*>(src + e + 8 * k);
            const uint32_t v[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // channels i and i + 4
              const uint32_t lo = (i & 1) ? v[i >> 1] >> 16 : v[i >> 1] & 0xffffu;
              const uint32_t hi = (i & 1) ? v[2 + (i >> 1)] >> 16 : v[2 + (i >> 1)] & 0xffffu;
              w[4 * k + i] = pack_f16x2(value(lo) * f, value(hi) * f);
            }
          }
          tmem_st16(lane_addr + G::Q_COL + (cs * (D / 2) + e) / 2, w);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&qready);
      // ---- tiles
      float m_ref = -INFINITY, l = 0.f;
      for (int i = 0; i < p.n; ++i, ++g) {
        const int b = g & 1;
        const uint32_t s_addr = lane_addr + G::S_COL + b * kTile;
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&sfull[b], (g >> 1) & 1));
        tc_fence_after();
        const int pos0 = p.q.base + (p.k0 + i) * kTile + cs * 32;
        uint32_t r[32];
        float mx = -INFINITY;
        const bool edge = pos0 < all_lo || pos0 + 32 > all_hi;
        if (live) {
          tmem_ld32(s_addr + cs * 32, r);
          tmem_wait_ld();
          tmem_reg_fence(r);
          if (edge) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (pos0 + e < sees.x || pos0 + e >= sees.y) r[e] = 0xff800000u;  // -infinity
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) mx = fmaxf(mx, __uint_as_float(r[e]));
          mx *= factor;  // positive: the order stays
        }
        red_max[b * 2 * R + cs * R + m] = mx;
        named_bar_sync(1, kSoftThreads);  // also: every half's S has been read
        if (live) {
          mx = fmaxf(red_max[b * 2 * R + m], red_max[b * 2 * R + R + m]);
          float alpha = 1.f;
          if (mx > m_ref + kSlack) {
            alpha = ex2_approx(m_ref - mx);
            m_ref = mx;
            l *= alpha;
          }
          if (i > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
            // the products so far, once they are all in O: half cs of the columns
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&vfree[b ^ 1], ((g - 1) >> 1) & 1));
            tc_fence_after();
#pragma unroll 1
            for (int h = 0; h < D / 2; h += 32) {
              uint32_t o[32];
              const uint32_t at = lane_addr + G::O_COL + cs * (D / 2) + h;
              tmem_ld32(at, o);
              tmem_wait_ld();
              tmem_reg_fence(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(at, o);
            }
            tmem_wait_st();
          }
          const float from = m_ref == -INFINITY ? 0.f : m_ref;
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float p0 = ex2_approx(fmaf(__uint_as_float(r[e]), factor, -from));
            const float p1 = ex2_approx(fmaf(__uint_as_float(r[e + 1]), factor, -from));
            l += p0 + p1;
            w[e >> 1] = pack_f16x2(p0, p1);
          }
          tmem_st16(s_addr + cs * 16, w);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pready[b]);
      }
      // ---- O of the part
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&vfree[(g - 1) & 1], ((g - 1) >> 1) & 1));
      tc_fence_after();
      red_sum[cs * R + m] = l;
      named_bar_sync(1, kSoftThreads);
      l = red_sum[m] + red_sum[R + m];
      const bool whole = p.k0 == 0 && p.n == p.q.steps;
      const int slot = 2 * c + (p.k0 == 0 ? 1 : 0);
      if (live) {
        const float inv = whole ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
        if (whole && mine && !(l < INFINITY)) set_status(a.status, DFLASH_DEV_NONFINITE);
#pragma unroll 1
        for (int h = 0; h < D / 2; h += 32) {
          uint32_t o[32];
          const int col = cs * (D / 2) + h;
          tmem_ld32(lane_addr + G::O_COL + col, o);
          tmem_wait_ld();
          tmem_reg_fence(o);
          if (mine) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // 8 channels, stored as 0 4 1 5 2 6 3 7
              float v[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) v[(e >> 1) + 4 * (e & 1)] = __uint_as_float(o[8 * k + e]) * inv;
              if (whole) {
                uint16_t* dst = a.out + (p.q.r0 + row / a.G) * a.out_stride + (p.head * a.G + row % a.G) * D + col + 8 * k;
                *reinterpret_cast<uint4*>(dst) =
                    a.bf16 ? make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]))
                           : make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]), pack_f16x2(v[6], v[7]));
              } else {
                float* dst = a.part + (static_cast<size_t>(slot) * R + m) * D + col + 8 * k;
                __stcg(reinterpret_cast<float4*>(dst), make_float4(v[0], v[1], v[2], v[3]));
                __stcg(reinterpret_cast<float4*>(dst) + 1, make_float4(v[4], v[5], v[6], v[7]));
              }
            }
          }
          __syncwarp();
        }
        if (!whole && mine && cs == 0) __stcg(a.part_ml + static_cast<size_t>(slot) * R + m, make_float2(m_ref, l));
      }
      tc_fence_before();
      named_bar_sync(1, kSoftThreads);  // red_sum has been read
      if (lane == 0) mbar_arrive(&ofree);
      if (warp == 2 && lane == 0 && x >= x_end) {
        // the last part: does its segment begin here and go on in the next CTAs?
        Kv4Job r{p.q.r0, p.row0, p.head, 0, 0, {0, 0, 0}};
        if (!whole && p.k0 == 0) {
          r.n_rows = p.rows;
          r.last = kv4_owner(T, C, x - p.n + p.q.steps - 1);
        }
        a.jobs[c] = r;
      }
    }
    if (!ok && lane == 0) set_status(a.status, DFLASH_DEV_TIMEOUT);
  } else {
    // ------------------------------------------------------------ unpacking
    const int w8 = warp - 2 - kSoftWarps;
    const int t = lane & 3;
    uint32_t g = 0;
    for (long long x = x_begin; x < x_end && ok;) {
      const Part p = part_at(x);
      x += p.n;
      for (int i = 0; i < p.n && ok; ++i, ++g) {
        const int st = g % NP, b = g & 1;
        const uint8_t* packed = ring + st * G::STAGE;
        const int pos0 = p.q.base + (p.k0 + i) * kTile;
        const bool edge = pos0 < p.q.lo || pos0 + kTile > p.q.hi;
        // cells that no row sees may hold anything: they become zeros
        auto hidden = [&](int cell) { return edge && (pos0 + cell < p.q.lo || pos0 + cell >= p.q.hi); };
        bool here = mbar_wait(&pfull[st], (g / NP) & 1);
        if (g >= 2) here = here && mbar_wait(&kfree[b], ((g >> 1) - 1) & 1);
        if (!__all_sync(0xffffffffu, here)) {
          ok = false;
          break;
        }
        // K: 8 lanes take the four quads t of two cells whose rows lie in
        // different banks, both as codes and, swizzled, as FP16
        uint8_t* kb = kbuf + b * G::BUF;
        constexpr int KW = B < 4 ? B : 4;  // words of a lane: blocks KW h ..
#pragma unroll
        for (int it = 0; it < (D == 256 ? 2 : 1); ++it) {
          int cell, h = 0;
          if constexpr (D == 256) {
            const int q = it * 32 + w8 * 4 + (lane >> 3);
            h = q & 1;
            cell = ((q >> 3) << 3) + ((q >> 1) & 3) + ((lane >> 2) & 1) * 4;
          } else if constexpr (D == 128) {
            const int q = w8 * 4 + (lane >> 3);
            cell = ((q >> 2) << 3) + ((q & 3) ^ (((lane >> 2) & 1) * 5));
          } else {
            const int q = w8 * 2 + (lane >> 4), k = (lane >> 2) & 3;
            cell = ((q >> 1) << 3) + ((q & 1) ^ ((k & 1) * 5) ^ ((k >> 1) * 2));
          }
          const uint8_t* grp = packed + (cell >> 4) * F::GROUP_BYTES;
          const int cg = cell & 15;
          uint32_t w[KW], d[KW];
          load_words<KW>(grp + F::K_CODES + cg * F::ROW + 4 * ((t * B + 4 * h) ^ F::k_swap(cg)), w);
          load_scales<KW>(grp + F::K_SCALES + cg * F::SROW + 8 * h, d);
          const bool zero = hidden(cell);
#pragma unroll
          for (int j = 0; j < KW; ++j) {
            const int blk = 4 * h + j;  // word 4 blk + t: box blk / 2, chunk 4 (blk % 2) + t
            const uint4 v = unpack(w[j], zero ? 0u : d[j]);
            *reinterpret_cast<uint4*>(kb + (blk >> 1) * (kTile * 128) + cell * 128 + (((4 * (blk & 1) + t) ^ (cell & 7)) << 4)) = v;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&kready[b]);
        // V: 8 lanes take the 8 channel groups of one cell
        if (g >= 2 && !__all_sync(0xffffffffu, mbar_wait(&vfree[b], ((g >> 1) - 1) & 1))) {
          ok = false;
          break;
        }
        uint8_t* vb = vbuf + b * G::BUF;
        const int ch = lane & 7;
#pragma unroll
        for (int it = 0; it < 2; ++it) {
          const int cell = it * 32 + w8 * 4 + (lane >> 3), cg = cell & 15;
          const uint8_t* grp = packed + (cell >> 4) * F::GROUP_BYTES;
          uint32_t w[U], d[U];
          load_words<U>(grp + F::V_CODES + cg * F::ROW + 4 * U * (ch ^ F::v_swap(cg)), w);
          load_scales<U>(grp + F::V_SCALES + cg * F::SROW + 2 * U * (ch >> 2), d);
          const bool zero = hidden(cell);
#pragma unroll
          for (int u = 0; u < U; ++u)  // word 8u + ch: box u, chunk ch
            *reinterpret_cast<uint4*>(vb + u * (kTile * 128) + cell * 128 + ((ch ^ (cell & 7)) << 4)) = unpack(w[u], zero ? 0u : d[u]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&vready[b]);
          mbar_arrive(&pfree[st]);
        }
      }
    }
    if (!ok && lane == 0) set_status(a.status, DFLASH_DEV_TIMEOUT);
  }
  // every warp whole again before the CTA-wide barrier, then the tensor memory goes
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D>
cudaError_t launch(const Kv4AttnArgs& a, int most, int jobs, cudaStream_t st) {
  using G = Geo<D>;
  cudaError_t e = cudaFuncSetAttribute(kv4_attn_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       G::SMEM + 8 * (kKv4MaxSeq + 1));
  if (e != cudaSuccess) return e;
  kv4_attn_tc_kernel<D><<<most, kThreads, G::SMEM + 8 * (a.n_seq + 1), st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || most == 1) return e;
  return launch_kv4_merge<D, kRows>(a, most, jobs, st);
}

}  // namespace

cudaError_t launch_kv4_attn_tc(int d, const Kv4AttnArgs& a, int most, int jobs, cudaStream_t st) {
  switch (d) {
    case 64: return launch<64>(a, most, jobs, st);
    case 128: return launch<128>(a, most, jobs, st);
    default: return launch<256>(a, most, jobs, st);
  }
}

}  // namespace dflash
