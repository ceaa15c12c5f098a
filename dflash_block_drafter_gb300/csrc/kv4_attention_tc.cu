// Attention over the 4-bit paged K/V cache for many query rows per kv head
// (blocks of several tokens over wide groups), on the tcgen05 tensor cores.
//
// One CTA per SM takes tiles of T cells (64 at D = 256, else 128: a tile costs
// about as much in hand-overs as in work) for up to 128 query rows:
//   warp 0        issues S = Q K^T (M 128, N = T), warp 2 O += P V (M 128, N = D):
//                 two warps, because a wait and the issue of a tile's MMAs
//                 take one warp as long as the MMAs themselves;
//   warps 1, 3    copy the tiles' packed K and V into rings (bulk copies): V's stages
//                 are held longer, and one warp's copies took as long as a tile;
//   warps 4..11   softmax: a thread has one row (TMEM lane) of every other
//                 tile: warps 4..7 the even ones, 8..11 the odd ones, so that the
//                 waits and fences of one tile lie under the arithmetic of the next;
//   warps 12..19  unpack K, warps 20..27 unpack V, once for all rows: FP16
//                 d (code - 8) in the 128-byte-swizzled layouts the MMAs read,
//                 double-buffered; four warps each for the even and the odd tiles.
// Q and P are the MMAs' A operands in tensor memory (FP16 pairs), P over the S it
// came from, so that shared memory carries little more than K and V: per tile and D =
// 256 64 KB written and read (1000 cycles), as much as the MMAs take, against 790
// cycles for the tile's bytes from HBM.  There are three S where they fit, because the
// chain from one S over the softmax and P V to the next in its place takes the longest.
// Columns: S | O | Q = 3 * 64 + 256 + 64 at D = 256 (half of Q: its channels from 128
// on are an operand in shared memory), 2 * 128 + 128 + 64 at D = 128, 3 * 128 + 64 + 32.
//
// The 8 channels of a code word lie in the order 0 4 1 5 2 6 3 7, in which
// masking the word yields pairs: Q's columns are stored in the same order,
// and O's are read back in it.
// Roundings: K, V and P to FP16 (2^-11 relative each, P 2^-32 of the row's largest weight
// absolute), Q by 2^-27 of a row's largest value at most (BF16 rows are scaled by a
// power of two, FP16 exact); scores, sums and O in FP32.  (FP16: the tensor cores' next
// wider type, TF32, has the same 11 bits at half the rate.)  The two softmax warps of a
// quarter of the rows hand a row's reference to each other tile by tile.
//
// Measured: a block of 8 tokens of 24 / 2 heads of 256 over 262144 cells 91 us (568
// TFLOP/s, 1.6 TB/s), 16 blocks of 2 .. 8 over 2048 .. 32768 cells 87 us; 64 blocks of 8 of
// 40 / 8 heads over 512 .. 8192 cells 259 us at 128 channels, 170 at 64.  No unit is full
// (issue 48 %, ALU 38 %, tensor pipe 37 %): a tile takes about 1900 cycles for its way
// through eight barriers, and the first product waits 9 to 10 us for the plan and Q.
// At 72 registers at launch 438, 398 and 402 bytes of spill stores (256, 128, 64 channels).
#include "kv4_attention.cuh"

namespace dflash {
namespace {

constexpr int kRows = 128;
constexpr int kOverhead = 8;   // a segment's beginning and end, in tiles
constexpr int kSoftWarps = 8, kUnpackWarps = 8;  // (unpacking: K and V each)
constexpr int kQkWarp = 0, kCopyKWarp = 1, kPvWarp = 2, kCopyVWarp = 3;
constexpr int kSoftWarp0 = 4, kUnpackWarp0 = kSoftWarp0 + kSoftWarps;
constexpr int kThreads = 32 * (kSoftWarps + 2 * kUnpackWarps + 4);  // whole warpgroups
constexpr int kSoftThreads = 32 * kSoftWarps;
// Registers a thread: 72 at launch (64512 in all), then 104, 64 and 40 by role:
// 256 * 104 + 512 * 64 + 128 * 40 = 64512.
constexpr int kSoftRegs = 104, kUnpackRegs = 64, kOtherRegs = 40;
static_assert(kThreads * 72 <= 65536 && kSoftThreads * kSoftRegs + 64 * kUnpackWarps * kUnpackRegs + 128 * kOtherRegs <= kThreads * 72,
              "the roles' registers come out of the launch's");
constexpr int kTmemCols = 512;

template <int D>
struct Geo {
  static constexpr int TILE = D == 256 ? 64 : 128;           // cells of a tile
  static constexpr int GROUPS = TILE / 16;
  static constexpr int SCORES = D == 128 ? 2 : 3;            // S buffers
  static constexpr int PACKED = D == 256 ? 3 : D == 128 ? 4 : 6;  // stages of the packed rings
  static constexpr int HALF = Kv4<D>::GROUP_BYTES / 2;       // K or V of a group: codes, then scales
  static constexpr int STAGE = GROUPS * HALF;
  static_assert(Kv4<D>::V_CODES == HALF && Kv4<D>::V_SCALES == HALF + Kv4<D>::K_SCALES, "halves");
  static constexpr int BUF = TILE * D * 2;                   // one unpacked K or V tile
  static constexpr int RED = 3 * kRows * 4;
  static constexpr int QT = D == 256 ? 128 : D;              // channels of Q in tensor memory
  static constexpr int QBUF = kRows * (D - QT) * 2;          // the others, [64-channel boxes][128 rows][128 B]
  static constexpr int SMEM = 1024 + 4 * BUF + QBUF + 2 * PACKED * STAGE + RED;
  static constexpr int S_COL = 0, O_COL = SCORES * TILE, Q_COL = O_COL + D;
  static_assert(Q_COL + QT / 2 <= kTmemCols, "columns");
};

// D[tmem] (+)= A * B[smem desc], kind::f16, one CTA; A in tensor memory (ta) or
// by a descriptor too (sa).  A descriptor comes in two words: only its low one, the address, changes between the
// MMAs of a tile, so that a warp that computes it as a whole keeps it in
// uniform registers and issues an MMA in a few instructions (with one lane's
// 64-bit descriptors the issue, not the tensor cores, took the time).
__device__ __forceinline__ void umma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void umma_f16_sa(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 a, {%1, %2};\n\t"
      "mov.b64 b, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&w)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "r"(w[8]), "r"(w[9]),
      "r"(w[10]), "r"(w[11]), "r"(w[12]), "r"(w[13]), "r"(w[14]), "r"(w[15])
      : "memory");
}

// One code word times its block's scale (twice in d): 8 FP16 in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ uint4 unpack(uint32_t w, uint32_t d, const Kv4Consts& k) {
  const uint32_t v = w >> 8;
  uint4 r;
  r.x = hmul2_u32(k.even(w), d);
  r.y = hmul2_u32(k.odd(w), d);
  r.z = hmul2_u32(k.even(v), d);
  r.w = hmul2_u32(k.odd(v), d);
  return r;
}

// N consecutive FP16 of shared memory as N pairs of equals.
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
  constexpr int R = kRows, NP = G::PACKED, U = D / 64, B = D / 32, kTile = G::TILE, kScores = G::SCORES, kGroups = G::GROUPS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* kbuf = smem;                       // [2][D / 64 boxes][T cells][128 B]
  uint8_t* vbuf = kbuf + 2 * G::BUF;          // [2]
  uint8_t* qbuf = vbuf + 2 * G::BUF;          // Q's channels from QT on
  uint8_t* kring = qbuf + G::QBUF;            // [NP] packed tiles of K
  uint8_t* vring = kring + NP * G::STAGE;     // and of V
  float* s_ref = reinterpret_cast<float*>(vring + NP * G::STAGE);   // [128 rows] references of the scores
  float* red_sum = s_ref + R;                                       // [2][128 rows]
  long long* pre = reinterpret_cast<long long*>(red_sum + 2 * R);   // [n_seq + 1]
  __shared__ long long scratch[kThreads / 32];
  __shared__ uint64_t kpfull[NP], kpfree[NP], vpfull[NP], vpfree[NP], kready[2], kfree[2], vready[2], vfree[2], sfull[kScores], sfree[kScores], pready[kScores], qready, odone, ofree, done[2];
  __shared__ uint32_t s_tmem;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < NP; ++i) {
      mbar_init(&kpfull[i], 1);
      mbar_init(&kpfree[i], kUnpackWarps / 2);
      mbar_init(&vpfull[i], 1);
      mbar_init(&vpfree[i], kUnpackWarps / 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&kready[i], kUnpackWarps / 2);
      mbar_init(&kfree[i], 1);
      mbar_init(&vready[i], kUnpackWarps / 2);
      mbar_init(&vfree[i], 1);
      mbar_init(&done[i], 1);
    }
    for (int i = 0; i < kScores; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&sfree[i], 1);
      mbar_init(&pready[i], kSoftWarps / 2);
    }
    mbar_init(&qready, kSoftWarps);
    mbar_init(&odone, 1);
    mbar_init(&ofree, kSoftWarps);
    fence_barrier_init();
  }
  const long long T = kv4_plan<kTile, kOverhead>(a, pre, scratch, blockIdx.x == 0);
  const int C = kv4_ctas(T, gridDim.x);
  const int c = blockIdx.x;
  pdl_launch_dependents();
  if (c >= C || T == 0) {
    if (tid == 0) a.jobs[c].n_rows = 0;
    return;
  }
  if (warp == kQkWarp) {
    tmem_alloc(&s_tmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const long long x_begin = kv4_start(T, C, c), x_end = kv4_start(T, C, c + 1);
  bool ok = true;

  const Kv4Part none{};
  auto part_at = [&](long long at, const Kv4Part& before) { return kv4_part<kTile, kOverhead>(a, pre, at, x_end, before); };

  if (warp < kSoftWarp0) fewer_registers<kOtherRegs>();
  if (warp == kCopyKWarp || warp == kCopyVWarp) {
    // ------------------------------------------------------------ producers
    const bool v_side = warp == kCopyVWarp;
    uint64_t* pfull = v_side ? vpfull : kpfull;
    uint64_t* pfree = v_side ? vpfree : kpfree;
    uint8_t* ring = v_side ? vring : kring;
    const int groups_of_page = 1 << (a.page_shift - 4);
    uint32_t g = 0;  // tiles over all parts
    for (Kv4Part p = part_at(x_begin, none); p.n > 0 && ok; p = part_at(p.next, p)) {
      // a lane holds the address of its group of its tile of WIN (0: nothing to copy, for
      // groups that no row sees: those before a window may have been given back), and
      // that of the WIN tiles after them
      constexpr int WIN = 32 / kGroups;
      const int lane_tile = lane / kGroups, lane_group = lane % kGroups;
      auto look_up = [&](int from) -> const uint8_t* {
        const int i = from + lane_tile;
        const int pos = p.q.base + (p.k0 + i) * kTile + lane_group * 16;
        if (i >= p.n || pos + 16 <= p.q.lo || pos >= p.q.hi) return nullptr;
        int page = a.table[static_cast<long long>(p.s) * a.table_stride + (pos >> a.page_shift)];
        if (page < 0 || page >= a.n_pages) {
          set_status(a.status, DFLASH_DEV_CAPACITY);
          page = 0;
        }
        const int grp = (pos >> 4) & (groups_of_page - 1);
        return a.cache + ((static_cast<size_t>(page) * a.n_kv + p.head) * groups_of_page + grp) * F::GROUP_BYTES +
               (v_side ? F::V_CODES : F::K_CODES);
      };
      const uint8_t *from = nullptr, *later = look_up(0);
      // the ring is too short for HBM's latency: L2 is asked for each tile WIN - 1 tiles
      // before it is copied, and at a part's beginning for those looked up that the ring
      // does not take (at 256 channels; in the CTA's first part only once Q is there,
      // whose loads would have to wait behind them)
      constexpr bool BEHIND = WIN > NP;
      if (BEHIND && g > 0 && lane_tile >= NP && later) bulk_prefetch_l2_plain(later, G::HALF);
      unsigned have = 0;
      for (int i = 0; i < p.n && ok; ++i, ++g) {
        const int t = i % WIN, st = g % NP;
        if (t == 0) {
          from = later;
          have = __ballot_sync(0xffffffffu, from != nullptr);
          later = look_up(i + WIN);
        }
        if (g >= NP) ok = __all_sync(0xffffffffu, kv4_wait(&pfree[st], (g / NP - 1) & 1));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&pfull[st], __popc(have >> (t * kGroups) & ((1u << kGroups) - 1)) * G::HALF);
        __syncwarp();
        if (lane_tile == t && from) bulk_g2s(ring + st * G::STAGE + lane_group * G::HALF, from, G::HALF, &pfull[st]);
        // (tiles of this part are still to come, so that it cannot end, and `qready` not
        // go on to the next part's phase, before this warp has seen it)
        if (BEHIND && g == NP - 1 && i == NP - 1 && i + 1 < p.n) {
          ok = __all_sync(0xffffffffu, kv4_wait(&qready, 0));
          if (lane_tile >= NP && from) bulk_prefetch_l2_plain(from, G::HALF);
        }
        if (t > 0 && lane_tile == t - 1 && later) bulk_prefetch_l2_plain(later, G::HALF);
        if (t == 0 && i > 0 && lane_tile == WIN - 1 && from) bulk_prefetch_l2_plain(from, G::HALF);
      }
    }
    // every copy lands before the CTA ends
    for (uint32_t i = g < NP ? 0 : g - NP; i < g; ++i)
      if (!kv4_wait(&pfull[i % NP], (i / NP) & 1)) ok = false;
    if (!ok && lane == 0) set_status(a.status, DFLASH_DEV_TIMEOUT);
  } else if (warp == kQkWarp) {
    // ------------------------------------------------------------ S = Q K^T
    // (the whole warp waits and computes, one lane issues)
    constexpr uint32_t idesc = umma_idesc_f16(128, kTile, false, false);
    const uint64_t kd = umma_desc_sw128(smem_u32(kbuf), 16, 1024);
    const uint32_t k_lo = static_cast<uint32_t>(kd), k_hi = static_cast<uint32_t>(kd >> 32);
    const uint64_t qd = umma_desc_sw128(smem_u32(qbuf), 16, 1024);
    const uint32_t q_lo = static_cast<uint32_t>(qd), q_hi = static_cast<uint32_t>(qd >> 32);
    const bool one = elect_one();
    uint32_t g = 0, part = 0;
    for (Kv4Part p = part_at(x_begin, none); p.n > 0 && ok; p = part_at(p.next, p), ++part) {
      const int n = p.n;
      ok = __all_sync(0xffffffffu, kv4_wait(&qready, part & 1));
      for (int i = 0; i < n && ok; ++i, ++g) {
        const uint32_t b = g & 1, sb = g % kScores, turn = g / kScores;
        bool here = kv4_wait(&kready[b], (g >> 1) & 1);
        if (turn > 0) here = here && kv4_wait(&sfree[sb], (turn - 1) & 1);  // P of the tile that had this S
        ok = __all_sync(0xffffffffu, here);
        if (!ok) break;
        tc_fence_after();
        const uint32_t lo = k_lo + b * (G::BUF >> 4), to = tmem + G::S_COL + sb * kTile;
        if (one) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t k_at = lo + (((kk >> 2) * (kTile * 128) + (kk & 3) * 32) >> 4);
            if (kk * 16 < G::QT) {
              umma_f16_ta(to, tmem + G::Q_COL + kk * 8, k_at, k_hi, idesc, kk > 0);
            } else {
              constexpr int K0 = G::QT / 16;
              umma_f16_sa(to, q_lo + ((((kk - K0) >> 2) * (kRows * 128) + (kk & 3) * 32) >> 4), q_hi, k_at, k_hi, idesc, 1);
            }
          }
          umma_commit(&sfull[sb]);
          umma_commit(&kfree[b]);
        }
        __syncwarp();
      }
    }
    // tensor memory may only be freed once every issued MMA has finished
    if (one) umma_commit(&done[0]);
    __syncwarp();
    if (!__all_sync(0xffffffffu, kv4_wait(&done[0], 0))) ok = false;
    if (!ok && lane == 0) set_status(a.status, DFLASH_DEV_TIMEOUT);
  } else if (warp == kPvWarp) {
    // ------------------------------------------------------------ O += P V
    constexpr uint32_t idesc = umma_idesc_f16(128, D, false, true);
    const uint64_t vd = umma_desc_sw128(smem_u32(vbuf), kTile * 128, 1024);
    const uint32_t v_lo = static_cast<uint32_t>(vd), v_hi = static_cast<uint32_t>(vd >> 32);
    const bool one = elect_one();
    uint32_t g = 0, part = 0;
    for (Kv4Part p = part_at(x_begin, none); p.n > 0 && ok; p = part_at(p.next, p), ++part) {
      const int n = p.n;
      // O of the part before has been read
      if (part > 0) ok = __all_sync(0xffffffffu, kv4_wait(&ofree, (part - 1) & 1));
      for (int i = 0; i < n && ok; ++i, ++g) {
        const uint32_t b = g & 1, sb = g % kScores;
        const bool here = kv4_wait(&vready[b], (g >> 1) & 1) && kv4_wait(&pready[sb], (g / kScores) & 1);
        ok = __all_sync(0xffffffffu, here);
        if (!ok) break;
        tc_fence_after();
        const uint32_t lo = v_lo + b * (G::BUF >> 4), from = tmem + G::S_COL + sb * kTile, more = i > 0;
        if (one) {
          umma_f16_ta(tmem + G::O_COL, from, lo, v_hi, idesc, more);
#pragma unroll
          for (int kk = 1; kk < kTile / 16; ++kk)
            umma_f16_ta(tmem + G::O_COL, from + kk * 8, lo + kk * (2048 >> 4), v_hi, idesc, 1);
          umma_commit(&vfree[b]);
          umma_commit(&sfree[sb]);
          if (i == n - 1) umma_commit(&odone);  // (a barrier of its own: vfree may be two phases behind then)
        }
        __syncwarp();
      }
    }
    if (one) umma_commit(&done[1]);
    __syncwarp();
    if (!__all_sync(0xffffffffu, kv4_wait(&done[1], 0))) ok = false;
    if (!ok && lane == 0) set_status(a.status, DFLASH_DEV_TIMEOUT);
  } else if (warp >= kSoftWarp0 && warp < kUnpackWarp0) {
    // ------------------------------------------------------------ softmax
    more_registers<kSoftRegs>();
    const int q4 = warp & 3, cs = (warp - kSoftWarp0) >> 2;  // TMEM lane quarter; tiles by parity, and half of Q's and O's columns
    const int m = q4 * 32 + lane;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
    uint32_t g = 0, part = 0;
    Kv4Job job{};  // the segment that begins here and goes on in the next CTAs, if one does
    for (Kv4Part p = part_at(x_begin, none); p.n > 0; p = part_at(p.next, p)) {
      const uint32_t per_g = kv4_per_token(a.G);
      const bool mine = m < p.rows, live = q4 * 32 < p.rows;  // the row; any row of the quarter
      const int2 sees = mine ? kv4_sees(a, p.q, kv4_token(m, per_g)) : make_int2(0, 0);
      int all_lo = mine ? sees.x : 0, all_hi = mine ? sees.y : 0x7fffffff;  // cells that every row of the quarter sees
#pragma unroll
      for (int w = 1; w < 32; w <<= 1) {
        all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, w));
        all_hi = min(all_hi, __shfl_xor_sync(0xffffffffu, all_hi, w));
      }
      // ---- Q into tensor memory: half cs of the row's channels
      // (Nothing else runs until Q is there, and an instruction of a chain costs several
      // cycles: FP16 rows are taken as they are, magnitudes compared as pairs of bits,
      // powers of two made of bits, the token of a row found by a multiplication.)
      const uint16_t* src = a.q + p.q.r0 * a.q_stride + kv4_token(m, per_g) * (a.q_stride - a.G * D) +
                            (p.head * a.G + m) * D + cs * (D / 2);
      // BF16 rows are scaled into FP16's range: by 2^8 where their largest magnitude is
      // in [2^-6, 2^7) (what falls below FP16's smallest value is 2^-27 of that, at most), so
      // that one pass over Q does; else by the power that brings it into [2^12, 2^13).
      auto power = [](int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); };
      int up = a.bf16 ? 8 : 0;
      for (bool again = false;; again = true) {
        uint32_t top = 0;
        if (live) {
          const float f = power(up);
#pragma unroll 1
          for (int e = 0; e < D / 2; e += 32) {
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint4 r = make_uint4(0, 0, 0, 0);
              if (mine) r = *reinterpret_cast<const uint4*>(src + e + 8 * k);
              if (a.bf16) {  // channels i and i + 4
                auto pair = [&](uint32_t lo, uint32_t hi) { return pack_f16x2(__uint_as_float(lo) * f, __uint_as_float(hi) * f); };
                w[4 * k] = pair(r.x << 16, r.z << 16), w[4 * k + 1] = pair(r.x & 0xffff0000u, r.z & 0xffff0000u);
                w[4 * k + 2] = pair(r.y << 16, r.w << 16), w[4 * k + 3] = pair(r.y & 0xffff0000u, r.w & 0xffff0000u);
              } else {
                w[4 * k] = prmt(r.x, r.z, 0x5410u), w[4 * k + 1] = prmt(r.x, r.z, 0x7632u);
                w[4 * k + 2] = prmt(r.y, r.w, 0x5410u), w[4 * k + 3] = prmt(r.y, r.w, 0x7632u);
              }
              top = __vmaxu2(top, __vmaxu2(__vmaxu2(r.x & 0x7fff7fffu, r.y & 0x7fff7fffu), __vmaxu2(r.z & 0x7fff7fffu, r.w & 0x7fff7fffu)));
            }
            if (cs * (D / 2) < G::QT) {
              tmem_st16(lane_addr + G::Q_COL + (cs * (D / 2) + e) / 2, w);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                *reinterpret_cast<uint4*>(qbuf + (e >> 6) * (kRows * 128) + m * 128 + (((((e & 63) >> 3) + k) ^ (m & 7)) << 4)) =
                    make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
            }
          }
          tmem_wait_st();
        }
        // A row with an infinity or a NaN is reported here already: below, where the sum of its
        // weights shows them, a score of -infinity passes for a cell that the row does not see.
        if (!again && sees.x < sees.y && max(top & 0xffffu, top >> 16) >= (a.bf16 ? 0x7f80u : 0x7c00u)) set_status(a.status, DFLASH_DEV_NONFINITE);
        if (again || !a.bf16) break;
        red_sum[cs * R + m] = __uint_as_float(top);
        named_bar_sync(1, kSoftThreads);
        top = __vmaxu2(__float_as_uint(red_sum[m]), __float_as_uint(red_sum[R + m]));
        const int ex = static_cast<int>(max(top & 0xffffu, top >> 16) >> 7);
        const bool other = top && (ex < 127 - 6 || ex > 127 + 6);
        if (!__any_sync(0xffffffffu, other)) break;
        if (other) up = min(12 + 127 - ex, 120);
      }
      // (beyond 2^80 any two scores that differ are too far apart to share weight)
      const float factor = fminf(fmaxf(a.scale_log2 * power(-up), 1.17549435e-38f), 0x1p80f);
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&qready);
      // ---- tiles of this warp's parity
      float m_ref = -INFINITY, l = 0.f;  // l in units of 2^m_ref
      const uint32_t g_end = g + p.n, g_first = g;
      for (g += (g ^ cs) & 1; g < g_end; g += 2) {
        const int b = cs, sb = g % kScores, i = g - g_first;
        const uint32_t s_addr = lane_addr + G::S_COL + sb * kTile;
        if (ok) ok = __all_sync(0xffffffffu, kv4_wait(&sfull[sb], (g / kScores) & 1));
        tc_fence_after();
        const int pos0 = p.q.base + (p.k0 + i) * kTile;
        // 64 cells at a time (S of a tile of 128 is read twice: for the maximum, and
        // again for P, which by then may lie over the half before)
        constexpr int HALVES = kTile / 64;
        uint32_t r[2][32];
        auto read_s = [&](int half) {
          tmem_ld32(s_addr + half * 64, r[0]);
          tmem_ld32(s_addr + half * 64 + 32, r[1]);
          tmem_wait_ld();
          tmem_reg_fence(r[0]);
          tmem_reg_fence(r[1]);
          const int pos = pos0 + half * 64;
          if (pos < all_lo || pos + 64 > all_hi) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (pos + 32 * h + e < sees.x || pos + 32 * h + e >= sees.y) r[h][e] = 0xff800000u;  // -infinity
          }
        };
        float mx = -INFINITY;
        if (live) {
#pragma unroll
          for (int half = 0; half < HALVES; ++half) {
            read_s(half);
#pragma unroll
            for (int e = 0; e < 32; ++e) mx = max3(mx, __uint_as_float(r[0][e]), __uint_as_float(r[1][e]));
          }
          mx *= factor;  // positive: the order stays
        }
        // the reference that the tile before left (barrier 2 + 2 q4 + parity)
        if (g > 0) named_bar_sync(2 + 2 * q4 + b, 64);
        if (live) {
          const float was = i > 0 ? s_ref[m] : -INFINITY;
          const bool over = mx > was + kKv4Slack;
          const float ref = over ? mx - kKv4Lift : was;
          if (i == 0 || __any_sync(0xffffffffu, over)) {
            s_ref[m] = ref;
            if (i > 0) {
              // the products so far, once they are all in O (that this tile has its S
              // says that P V of tile g - 3 is done: the parity means tile g - 1)
              if (ok) ok = __all_sync(0xffffffffu, kv4_wait(&vfree[b ^ 1], ((g - 1) >> 1) & 1));
              tc_fence_after();
              const float alpha = over ? ex2_approx(was - ref) : 1.f;
#pragma unroll 1
              for (int h = 0; h < D; h += 16) {
                uint32_t o[16];
                const uint32_t at = lane_addr + G::O_COL + h;
                tmem_ld16(at, o);
                tmem_wait_ld();
                tmem_reg_fence(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st16(at, o);
              }
              tmem_wait_st();
            }
          }
          if (ref > m_ref) {
            l *= ex2_approx(m_ref - ref);
            m_ref = ref;
          }
        }
        __syncwarp();
        named_bar_arrive(2 + 2 * q4 + (b ^ 1), 64);
        if (live) {
          const float from = m_ref == -INFINITY ? 0.f : m_ref;
          const uint64_t factor2 = pack2(factor, factor), from2 = pack2(-from, -from);
          uint64_t sum2 = pack2(0.f, 0.f);
#pragma unroll
          for (int half = 0; half < HALVES; ++half) {
            if (HALVES > 1) read_s(half);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                float x0, x1;
                unpack2(fma2(pack2(__uint_as_float(r[h][e]), __uint_as_float(r[h][e + 1])), factor2, from2), x0, x1);
                const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                sum2 = add2(sum2, pack2(p0, p1));
                r[0][16 * h + (e >> 1)] = pack_f16x2(p0, p1);
              }
            tmem_st32(s_addr + half * 32, r[0]);
          }
          float s0, s1;
          unpack2(sum2, s0, s1);
          l += s0 + s1;
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pready[sb]);
      }
      g = g_end;
      // ---- O of the part
      if (ok) ok = __all_sync(0xffffffffu, kv4_wait(&odone, part & 1));
      ++part;
      tc_fence_after();
      named_bar_sync(1, kSoftThreads);  // the last reference
      if (live) {
        const float ref = s_ref[m];
        l = l > 0.f ? l * ex2_approx(m_ref - ref) : l;  // (not of a NaN; a parity without weight has 0)
        m_ref = ref;
      }
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
                uint16_t* dst = a.out + p.q.r0 * a.out_stride + kv4_token(m, per_g) * (a.out_stride - a.G * D) + (p.head * a.G + m) * D + col + 8 * k;
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
      if (!whole && p.k0 == 0) job = Kv4Job{p.q.r0, p.head, p.rows, kv4_owner(T, C, p.end - 1)};
    }
    if (warp == kSoftWarp0 && lane == 0) a.jobs[c] = job;
    if (!ok && lane == 0) set_status(a.status, DFLASH_DEV_TIMEOUT);
  } else if (warp >= kUnpackWarp0) {
    // ------------------------------------------------------------ unpacking
    fewer_registers<kUnpackRegs>();
    const bool v_side = warp >= kUnpackWarp0 + kUnpackWarps;
    const int w4 = warp & 3, b = ((warp - kUnpackWarp0) >> 2) & 1;  // of four warps; parity of its tiles
    uint64_t* ready = (v_side ? vready : kready) + b;
    uint64_t* free_ = (v_side ? vfree : kfree) + b;
    uint64_t* pfull = v_side ? vpfull : kpfull;
    uint64_t* pfree = v_side ? vpfree : kpfree;
    const uint8_t* ring = v_side ? vring : kring;
    const Kv4Consts kc;
    // A lane's first cell of a tile, its codes and scales there (in the packed
    // tile) and its first 16 bytes in the unpacked tile; the others lie whole
    // groups further.  K: 8 lanes take the four quads t of two cells whose
    // rows lie in different banks, both as codes and, swizzled, as FP16; a lane has
    // words of blocks 4h .. (word 4 blk + t goes to box blk / 2, chunk 4 (blk % 2) + t).
    // V: 8 lanes take the 8 channel groups of one cell (word 8u + ch: box u, chunk ch).
    constexpr int KW = B < 4 ? B : 4;           // words of a lane in a K row
    constexpr int KSTEP = D == 256 ? 16 : 32;   // cells between a lane's K rows
    int cell, codes, scales, first;
    if (v_side) {
      const int ch = lane & 7;
      cell = w4 * 4 + (lane >> 3);
      codes = cell * F::ROW + 4 * U * (ch ^ F::v_swap(cell));
      scales = F::K_SCALES + cell * F::SROW + 2 * U * (ch >> 2);
      first = cell * 128 + ((ch ^ (cell & 7)) << 4);
    } else {
      const int t = lane & 3;
      int h = 0;
      if constexpr (D == 256) {
        const int q = w4 * 4 + (lane >> 3);
        h = q & 1;
        cell = ((q >> 3) << 3) + ((q >> 1) & 3) + ((lane >> 2) & 1) * 4;
      } else if constexpr (D == 128) {
        const int q = w4 * 4 + (lane >> 3);
        cell = ((q >> 2) << 3) + ((q & 3) ^ (((lane >> 2) & 1) * 5));
      } else {
        const int q = w4 * 2 + (lane >> 4), k = (lane >> 2) & 3;
        cell = ((q >> 1) << 3) + ((q & 1) ^ ((k & 1) * 5) ^ ((k >> 1) * 2));
      }
      const int cg = cell & 15;
      codes = (cell >> 4) * G::HALF + cg * F::ROW + 4 * ((t * B + 4 * h) ^ F::k_swap(cg));
      scales = (cell >> 4) * G::HALF + F::K_SCALES + cg * F::SROW + 8 * h;
      first = 2 * h * (kTile * 128) + cell * 128 + ((t ^ (cell & 7)) << 4);
    }
    uint8_t* to = (v_side ? vbuf : kbuf) + b * G::BUF + first;
    uint8_t* to4 = (v_side ? vbuf : kbuf) + b * G::BUF + (first ^ 64);  // chunk + 4
    uint32_t g = 0;
    for (Kv4Part p = part_at(x_begin, none); p.n > 0 && ok; p = part_at(p.next, p)) {
      const uint32_t g_end = g + p.n, g_first = g;
      for (g += (g ^ b) & 1; g < g_end; g += 2) {
        const int st = g % NP;
        const uint8_t* packed = ring + st * G::STAGE;
        const int pos0 = p.q.base + (p.k0 + static_cast<int>(g - g_first)) * kTile;
        // cells that no row sees may hold anything: they become zeros
        const bool edge = pos0 < p.q.lo || pos0 + kTile > p.q.hi;
        auto hidden = [&](int off) { return pos0 + cell + off < p.q.lo || pos0 + cell + off >= p.q.hi; };
        // First the buffer: that tile g - 2 has been used says that the stage's
        // last tile, g - NP, has been unpacked (by the other parity's warps), so that
        // the parity below cannot be taken for that of an earlier phase.
        static_assert(NP >= 2, "see above");
        bool here = true;
        if (g >= 2) here = kv4_wait(free_, ((g >> 1) - 1) & 1);
        here = here && kv4_wait(&pfull[st], (g / NP) & 1);
        if (!__all_sync(0xffffffffu, here)) {
          ok = false;
          break;
        }
        if (!v_side) {
          constexpr int N = kTile / KSTEP;
          uint32_t w[N][KW], d[N][KW];
#pragma unroll
          for (int it = 0; it < N; ++it) {
            load_words<KW>(packed + codes + it * (KSTEP / 16) * G::HALF, w[it]);
            load_scales<KW>(packed + scales + it * (KSTEP / 16) * G::HALF, d[it]);
            if (edge && hidden(it * KSTEP))
              for (int j = 0; j < KW; ++j) d[it][j] = 0;
          }
#pragma unroll
          for (int it = 0; it < N; ++it)
#pragma unroll
            for (int j = 0; j < KW; ++j)
              *reinterpret_cast<uint4*>(((j & 1) ? to4 : to) + (j >> 1) * (kTile * 128) + it * KSTEP * 128) =
                  unpack(w[it][j], d[it][j], kc);
        } else {
          constexpr int N = kGroups;
          uint32_t w[N][U], d[N][U];
#pragma unroll
          for (int it = 0; it < N; ++it) {
            load_words<U>(packed + codes + it * G::HALF, w[it]);
            load_scales<U>(packed + scales + it * G::HALF, d[it]);
            if (edge && hidden(it * 16))
              for (int u = 0; u < U; ++u) d[it][u] = 0;
          }
#pragma unroll
          for (int it = 0; it < N; ++it)
#pragma unroll
            for (int u = 0; u < U; ++u)
              *reinterpret_cast<uint4*>(to + u * (kTile * 128) + it * 16 * 128) = unpack(w[it][u], d[it][u], kc);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(ready);
          mbar_arrive(&pfree[st]);
        }
      }
      g = g_end;
    }
    if (!ok && lane == 0) set_status(a.status, DFLASH_DEV_TIMEOUT);
  }
  // every warp whole again before the CTA-wide barrier, then the tensor memory goes
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kQkWarp) {
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
