// Per-head RMSNorm and position rotation of query and key rows in one pass
// (dflash_qk_norm_rope in include/dflash.h).
//
//   y_c = x_c w_c / sqrt(mean_c x_c^2 + eps)
//   z_j = y_j cos a_j - y_{j+h} sin a_j,  z_{j+h} = y_{j+h} cos a_j + y_j sin a_j
//   a_j = position (of j's axis) * frequency j,  j < h = rotary_dim / 2.
//
// A lane has 8 pairs of channels of a head, two 16-byte loads and stores h apart (of the
// channels that are not turned 16 neighbours), a warp 512 channels: two, four or eight heads.  So both channels of a
// pair are in one lane.  (With 8 neighbours in a lane and the partners by shuffles, a value took 0.6 instructions of a warp
// instead of 0.3, and 30001 rows of 32 / 8 heads of 128 144 us.)  Weights, cosines and sines of a row are folded into
// two factors per channel, z = (x A + x' B) / rms, once per row and for all of its heads.
// Everything is FP32, rounded once to the rows' type.  Heads whose squares leave its range, and all heads where a weight is very large or
// small, are scaled by powers of two first.  The bytes bound it: every value is read and written once.
//
// Measured, calls in a row: 30001 rows of 32 / 8 heads of 128 104 us, 5.9 TB/s (floor 90 us at the 6.8 TB/s of a copy; 307 MB read,
// issue slots at 50 %); 4097 rows of 16 / 16 heads of 64 with three axes 12 us (floor 5; rows still in L2).  Few rows are a launch: 8 rows 6 us.
#include "common.cuh"
#include "internal.h"
#include "kernels.h"

#include <cmath>

namespace dflash {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kUnroll = 4;   // steps of a warp whose loads are in flight
constexpr int kPerSm = 2;    // CTAs of an SM
constexpr int kMaxAxes = 4;

struct RopeSide {
  const uint16_t* x;
  uint16_t* out;
  long long stride, out_stride;  // elements between rows
  const float* weight;           // null: no norm
  int heads, steps;              // steps: of a warp over the heads
};

struct RopeArgs {
  RopeSide side[2];  // queries, keys
  int n_rows, splits;  // warps of a row
  float eps;
  const int32_t* positions;
  long long position_stride;
  int n_axes, half;
  const uint8_t* axes;
  const uint64_t* turns;
  int32_t* status;
};

// Two pieces of 8 channels as FP32.
template <bool BF16>
__device__ __forceinline__ void widen(const uint4 (&raw)[2], float (&x)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t w[4] = {raw[h].x, raw[h].y, raw[h].z, raw[h].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (BF16) {
        x[8 * h + 2 * k] = __uint_as_float(w[k] << 16);
        x[8 * h + 2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
        x[8 * h + 2 * k] = f.x;
        x[8 * h + 2 * k + 1] = f.y;
      }
    }
  }
}

// Sum of squares of a head's values times f, a power of two that keeps them in FP32's range.
template <bool BF16, int LANES>
__device__ __noinline__ float far_squares(uint4 a, uint4 b, float f) {
  const uint4 raw[2] = {a, b};
  float x[16], s = 0.f;
  widen<BF16>(raw, x);
#pragma unroll
  for (int i = 0; i < 16; ++i) s = fmaf(x[i] * f, x[i] * f, s);
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, kPerSm) qk_norm_rope_kernel(const RopeArgs a) {
  constexpr int LANES = D / 16, HEADS = 32 / LANES;  // lanes of a head, heads of a step of a warp
  constexpr uint32_t ONES = BF16 ? 0x3f803f80u : 0x3c003c00u;
  __shared__ __align__(16) float s_w[2][D];
  __shared__ uint64_t s_turns[D / 2];
  __shared__ uint8_t s_axis[D / 2];
  __shared__ __align__(16) float2 s_angle[kWarps][D / 2];  // (cos, sin) of each warp's row
  const int tid = threadIdx.x, lane = tid & 31;
  float2* angle = s_angle[tid >> 5];
  // weights (or an eps) whose products with values of heads that are neither `big` nor `low` below may leave FP32's range
  bool wide = a.eps > 1e38f;
  for (int i = tid; i < D; i += kThreads) {
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const float w = a.side[which].weight ? a.side[which].weight[i] : 1.f;
      wide |= !(fabsf(w) <= 0x1p62f) || (w != 0.f && fabsf(w) < 0x1p-30f);
      s_w[which][i] = w;
    }
    if (i < a.half) {
      s_turns[i] = a.turns[i];
      int axis = a.axes ? a.axes[i] : 0;
      if (axis >= a.n_axes) {
        if (blockIdx.x == 0) set_status(a.status, DFLASH_DEV_BAD_VALUE);
        axis = 0;
      }
      s_axis[i] = static_cast<uint8_t>(axis);
    }
  }
  wide = __syncthreads_or(wide);
  const float most = wide ? -1.f : 1e38f;  // of a sum of squares, for heads that need no care
  const int sub = lane / LANES, at = lane % LANES;
  const bool turned = at < a.half / 8;
  const int j0 = at * 8;                                        // frequencies of the lane's pairs
  const int ca = turned ? j0 : at * 16;                         // its channels (those behind the turned ones begin at 2 half)
  const int cb = turned ? j0 + a.half : ca + 8;
  const int steps = a.side[0].steps + a.side[1].steps;
  const long long units = static_cast<long long>(a.n_rows) * a.splits;
  for (long long unit = blockIdx.x * kWarps + (tid >> 5); unit < units; unit += gridDim.x * kWarps) {
    const long long row = a.splits == 1 ? unit : unit / a.splits;
    const int split = static_cast<int>(unit - row * a.splits);
    const int i0 = static_cast<int>(static_cast<long long>(steps) * split / a.splits);
    const int i1 = static_cast<int>(static_cast<long long>(steps) * (split + 1) / a.splits);
    if (a.half) {
      int pos[kMaxAxes];
      bool skip = false;
#pragma unroll
      for (int i = 0; i < kMaxAxes; ++i) {
        pos[i] = i < a.n_axes ? a.positions[i * a.position_stride + row] : 0;
        skip |= pos[i] < 0;
      }
      if (skip) continue;  // a row of the padded batch
      __syncwarp();        // the last row's angles have been read
      for (int j = lane; j < a.half; j += 32) {
        int p = pos[0];
        if (a.n_axes > 1) {
          const int axis = s_axis[j];
#pragma unroll
          for (int i = 1; i < kMaxAxes; ++i) p = axis == i ? pos[i] : p;
        }
        float2 t;
        rope_sincos(s_turns[j], p, t.y, t.x);
        angle[j] = t;
      }
      __syncwarp();
    }
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      // (chosen field by field: an index into the arguments would copy them to local memory)
      const RopeSide s = {which ? a.side[1].x : a.side[0].x, which ? a.side[1].out : a.side[0].out,
                          which ? a.side[1].stride : a.side[0].stride, which ? a.side[1].out_stride : a.side[0].out_stride,
                          which ? a.side[1].weight : a.side[0].weight, which ? a.side[1].heads : a.side[0].heads,
                          which ? a.side[1].steps : a.side[0].steps};
      const int b0 = which ? max(i0 - a.side[0].steps, 0) : min(i0, s.steps);
      const int b1 = which ? max(i1 - a.side[0].steps, 0) : min(i1, s.steps);
      if (b0 >= b1) continue;
      // z_a = (a aa + b ab) / rms, z_b = (b ba + a bb) / rms
      float aa[8], ab[8], ba[8], bb[8];
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float2 w = *reinterpret_cast<const float2*>(&s_w[which][ca + e]);
        const float2 v = *reinterpret_cast<const float2*>(&s_w[which][cb + e]);
        float4 t = make_float4(1.f, 0.f, 1.f, 0.f);  // cos, sin of two pairs
        if (turned) t = *reinterpret_cast<const float4*>(&angle[j0 + e]);
        aa[e] = w.x * t.x, aa[e + 1] = w.y * t.z;
        ab[e] = -v.x * t.y, ab[e + 1] = -v.y * t.w;
        ba[e] = v.x * t.x, ba[e + 1] = v.y * t.z;
        bb[e] = w.x * t.y, bb[e + 1] = w.y * t.w;
      }
      const uint16_t* src = s.x + row * s.stride + sub * D;
      uint16_t* dst = s.out + row * s.out_stride + sub * D;
      const bool norm = s.weight != nullptr;
#pragma unroll 1
      for (int i = b0; i < b1; i += kUnroll) {
        uint4 raw[kUnroll][2];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          raw[u][0] = raw[u][1] = make_uint4(ONES, ONES, ONES, ONES);  // (a head that there is not is an ordinary one)
          if (i + u < b1 && (i + u) * HEADS + sub < s.heads) {
            const uint16_t* from = src + (i + u) * (HEADS * D);
            raw[u][0] = __ldcs(reinterpret_cast<const uint4*>(from + ca));
            raw[u][1] = __ldcs(reinterpret_cast<const uint4*>(from + cb));
          }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          if (i + u >= b1) break;  // (the same for the warp)
          float x[16], ssq = 0.f, ssq2 = 0.f;
          widen<BF16>(raw[u], x);
#pragma unroll
          for (int e = 0; e < 16; e += 2) ssq = fmaf(x[e], x[e], ssq), ssq2 = fmaf(x[e + 1], x[e + 1], ssq2);
          ssq += ssq2;
#pragma unroll
          for (int o = 1; o < LANES; o <<= 1) ssq += __shfl_xor_sync(0xffffffffu, ssq, o);
          const float m = ssq * (1.f / D) + a.eps;
          float inv = norm ? rsqrtf(m) : 1.f;
          const bool low = norm && ssq < 1e-20f;
          if (__any_sync(0xffffffffu, !(ssq < most) || low)) {
            // The values are scaled by powers of two until the largest is about 1 (f, for their squares, and h), and 1 / rms is that of
            // the scaled ones, so that products with the weights leave the range only where results do.
            const bool big = !(ssq < 1e38f);
            const float f = big ? 0x1p-70f : low ? 0x1p90f : 0.5f;
            const float far = far_squares<BF16, LANES>(raw[u][0], raw[u][1], f);
            if (big && !(far < INFINITY) && at == 0) set_status(a.status, DFLASH_DEV_NONFINITE);
            if (norm && (!(ssq < most) || low)) {
              auto power = [](float v) { return __uint_as_float(__float_as_uint(v) & 0x7f800000u); };
              // 1 / rms of the values times g, the same power where the squares count
              const bool least = m < 1e-30f, same = big || least || !low;
              const float g = same ? f : 0.5f;
              const float r = rsqrtf((big || least ? far : 0.25f * ssq) * (1.f / D) + a.eps * g * g);
              const float back = same ? 1.f : 0x1p-91f;  // g / f
              // (2^100: beside an eps far above the squares, inv has its bits still)
              const float h = far > 0.f && far < INFINITY ? fminf(power(rsqrtf(far)), power(r) * 0x1p100f * back) : 1.f;
              inv = r < INFINITY ? r / h * back : 0.f;  // a head of zeros without eps stays one
#pragma unroll
              for (int e = 0; e < 16; ++e) x[e] = x[e] * f * h;
            }
          }
          uint32_t za[4], zb[4];
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float z0 = fmaf(x[8 + e], ab[e], x[e] * aa[e]) * inv, z1 = fmaf(x[9 + e], ab[e + 1], x[e + 1] * aa[e + 1]) * inv;
            const float y0 = fmaf(x[e], bb[e], x[8 + e] * ba[e]) * inv, y1 = fmaf(x[e + 1], bb[e + 1], x[9 + e] * ba[e + 1]) * inv;
            za[e / 2] = BF16 ? pack_bf16x2(z0, z1) : pack_f16x2(z0, z1);
            zb[e / 2] = BF16 ? pack_bf16x2(y0, y1) : pack_f16x2(y0, y1);
          }
          if ((i + u) * HEADS + sub < s.heads) {
            uint16_t* to = dst + (i + u) * (HEADS * D);
            __stcs(reinterpret_cast<uint4*>(to + ca), make_uint4(za[0], za[1], za[2], za[3]));
            __stcs(reinterpret_cast<uint4*>(to + cb), make_uint4(zb[0], zb[1], zb[2], zb[3]));
          }
        }
      }
    }
  }
}

template <int D>
cudaError_t launch(RopeArgs a, bool bf16, cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  constexpr int HEADS = 512 / D;
  for (RopeSide& s : a.side) s.steps = (s.heads + HEADS - 1) / HEADS;
  const int steps = a.side[0].steps + a.side[1].steps;
  // few rows: a row's heads are shared out until every SM has its warps
  const long long want = static_cast<long long>(sms) * 16;
  const int most = (steps + kUnroll - 1) / kUnroll;
  const long long by = (want + a.n_rows - 1) / a.n_rows;
  a.splits = static_cast<int>(by < most ? by : most);
  const long long blocks = (static_cast<long long>(a.n_rows) * a.splits + kWarps - 1) / kWarps;
  // One wave.  Measured on 30001 rows of 32 / 8 heads of 128 (floor 90 us): 104 us; CTAs of less loads, three or four
  // on an SM, 105 to 129; several waves 107 to 117.
  const unsigned grid = static_cast<unsigned>(blocks < 1ll * kPerSm * sms ? blocks : 1ll * kPerSm * sms);
  if (bf16) qk_norm_rope_kernel<D, true><<<grid, kThreads, 0, st>>>(a);
  else qk_norm_rope_kernel<D, false><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

bool bad_rows(const void* x, const void* out, int64_t stride, int64_t out_stride, int32_t heads, int32_t d) {
  if (heads == 0) return false;
  const int64_t width = static_cast<int64_t>(heads) * d;
  return !x || !out || reinterpret_cast<uintptr_t>(x) % 16 || reinterpret_cast<uintptr_t>(out) % 16 || stride < width ||
         out_stride < width || stride % 8 || out_stride % 8;
}

}  // namespace
}  // namespace dflash

using namespace dflash;

extern "C" {

int dflash_rope_turns(const double* inv_freq, int32_t n, uint64_t* turns) {
  if (n < 0 || (n > 0 && (!inv_freq || !turns))) return DFLASH_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n; ++i)
    if (!std::isfinite(inv_freq[i])) return DFLASH_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n; ++i) {
    const double t = inv_freq[i] / 6.283185307179586476925286766559;
    const double part = std::ldexp(t - std::floor(t), 64);  // whole turns are none
    turns[i] = part >= 18446744073709551615.0 ? 0 : static_cast<uint64_t>(part);
  }
  return DFLASH_OK;
}

int dflash_qk_norm_rope(const void* q, void* q_out, int64_t q_stride, int64_t q_out_stride, int32_t n_q_heads,
                        const void* k, void* k_out, int64_t k_stride, int64_t k_out_stride, int32_t n_k_heads,
                        int32_t head_dim, int32_t type, int32_t n_rows, const float* q_weight, const float* k_weight,
                        float eps, const int32_t* positions, int64_t position_stride, int32_t n_axes,
                        const uint8_t* axes, const uint64_t* turns, int32_t rotary_dim, int32_t* dev_status,
                        dflash_stream_t stream) {
  if (type != DFLASH_T_BF16 && type != DFLASH_T_FP16) return DFLASH_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return DFLASH_ERR_UNSUPPORTED;
  if (n_rows < 0 || n_q_heads < 0 || n_k_heads < 0 || rotary_dim < 0 || rotary_dim > head_dim || !(eps >= 0.f) ||
      !(eps < INFINITY))
    return DFLASH_ERR_INVALID_ARG;
  if (rotary_dim % 16) return DFLASH_ERR_UNSUPPORTED;
  if (n_q_heads > 65536 || n_k_heads > 65536) return DFLASH_ERR_CAPACITY;
  if (rotary_dim > 0) {
    if (n_axes < 1 || n_axes > kMaxAxes) return DFLASH_ERR_UNSUPPORTED;
    if (n_axes > 1 && (!axes || position_stride < n_rows)) return DFLASH_ERR_INVALID_ARG;
  }
  if (n_rows == 0 || n_q_heads + n_k_heads == 0) return DFLASH_OK;
  if (bad_rows(q, q_out, q_stride, q_out_stride, n_q_heads, head_dim) ||
      bad_rows(k, k_out, k_stride, k_out_stride, n_k_heads, head_dim) ||
      (rotary_dim > 0 && (!positions || !turns || reinterpret_cast<uintptr_t>(turns) % 8)))
    return DFLASH_ERR_INVALID_ARG;
  RopeArgs a{};
  a.side[0] = {static_cast<const uint16_t*>(q), static_cast<uint16_t*>(q_out), q_stride, q_out_stride, q_weight, n_q_heads, 0};
  a.side[1] = {static_cast<const uint16_t*>(k), static_cast<uint16_t*>(k_out), k_stride, k_out_stride, k_weight, n_k_heads, 0};
  a.n_rows = n_rows;
  a.eps = eps;
  a.positions = positions;
  a.position_stride = position_stride;
  a.n_axes = n_axes;
  a.half = rotary_dim / 2;
  a.axes = n_axes > 1 ? axes : nullptr;
  a.turns = turns;
  a.status = dev_status;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool bf16 = type == DFLASH_T_BF16;
  const cudaError_t e = head_dim == 64 ? launch<64>(a, bf16, st) : head_dim == 128 ? launch<128>(a, bf16, st) : launch<256>(a, bf16, st);
  return cuda_status(e, "qk norm rope");
}

}  // extern "C"
