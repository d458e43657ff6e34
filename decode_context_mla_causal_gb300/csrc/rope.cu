// Rotary positions of query and key heads.
//
// Pair (a, b) at position n turns by the angle 2 pi f n, f the pair's frequency in turns. f is
// given as a fraction of 2^64, so that n f modulo 2^64, an integer product, is the exact fraction
// of a turn at any position; its upper 32 bits, as a signed number of half turns in [-1, 1) rounded
// to fp32 (24 bits: off by at most 2^-25 half turns), go through sincospi, which needs no reduction
// (a 32-bit angle in radians is off by 0.06 at a million, and a 64-bit one costs the slow units).
//
// Memory-bound: 4 bytes moved per element, and few operations once cosine and sine of a row are
// shared by its heads: a CTA forms them for its rows in shared memory, then moves the heads, 32
// bytes (eight pairs) to a thread. 8192 rows of 128 heads, the 64 dims that turn of 192, and one
// head beside them: 49.6 us, 5.4 TB/s, floor 39.8. 32 rows are bound by the launch, 2.3 us.
#include <algorithm>
#include <cmath>

#include "common.cuh"

namespace dcpmla {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxPairs = 2048;  // of a CTA's rows
constexpr int kAhead = 2;         // units of a thread on their way: one or four 53 us, two 50.6

struct RopeSide {
  const uint16_t* x;
  uint16_t* out;
  int64_t x_row, x_head, out_row, out_head;
  int heads;
};
struct RopeParams {
  RopeSide a, b;
  const int32_t* positions;
  const uint64_t* table;
  float amplitude;
  int rows, rot_pairs, row_count, units, copies;  // units of eight pairs, of 8 dims that are copied
  FastDiv unit_div, head_div, pair_div;
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

template <bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
  // [row][pair]: cosine, sine; read two pairs at a time
  __shared__ __align__(16) float2 s_turn[kMaxPairs];
  const int row0 = blockIdx.x * p.row_count;
  const int rows = min(p.row_count, p.rows - row0);
  for (int i = threadIdx.x; i < rows * p.rot_pairs; i += kRopeThreads) {
    const int t = p.pair_div.div(i);
    const uint64_t turn = (uint64_t)(int64_t)p.positions[row0 + t] * p.table[i - t * p.rot_pairs];
    float s, c;
    sincospif((float)(int32_t)(turn >> 32) * (1.f / 2147483648.f), &s, &c);
    s_turn[i] = make_float2(c * p.amplitude, s * p.amplitude);
  }
  __syncthreads();
  const int per_head = p.units + p.copies;
  const int heads = p.a.heads + p.b.heads;
  const int all = rows * heads * per_head;
  const int step = gridDim.y * kRopeThreads;
  // kAhead units of a thread are on their way at a time
  for (int i0 = blockIdx.y * kRopeThreads + threadIdx.x; i0 < all; i0 += kAhead * step) {
    uint4 v[kAhead][2];
    uint16_t* to[kAhead];  // NULL: nothing to do
    int unit[kAhead], row[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = i0 + k * step;
      to[k] = nullptr;
      if (i >= all) continue;
      const int th = p.unit_div.div(i), u = i - th * per_head;
      const int t = p.head_div.div(th), h = th - t * heads;
      const bool first = h < p.a.heads;
      const int hh = first ? h : h - p.a.heads;
      const uint16_t* x = (first ? p.a.x : p.b.x) +
                          (int64_t)(row0 + t) * (first ? p.a.x_row : p.b.x_row) +
                          (int64_t)hh * (first ? p.a.x_head : p.b.x_head);
      uint16_t* out = (first ? p.a.out : p.b.out) +
                      (int64_t)(row0 + t) * (first ? p.a.out_row : p.b.out_row) +
                      (int64_t)hh * (first ? p.a.out_head : p.b.out_head);
      unit[k] = u, row[k] = t;
      if (u >= p.units) {
        if (x == out) continue;
        const int at = 2 * p.rot_pairs + 8 * (u - p.units);
        v[k][0] = *reinterpret_cast<const uint4*>(x + at);
        to[k] = out + at;
      } else {
        to[k] = out + (kInterleaved ? 16 * u : 8 * u);
        const uint16_t* from = x + (kInterleaved ? 16 * u : 8 * u);
        v[k][0] = *reinterpret_cast<const uint4*>(from);
        v[k][1] = *reinterpret_cast<const uint4*>(from + (kInterleaved ? 8 : p.rot_pairs));
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (to[k] == nullptr) continue;
      if (unit[k] >= p.units) {
        *reinterpret_cast<uint4*>(to[k]) = v[k][0];
        continue;
      }
      const uint32_t w[8] = {v[k][0].x, v[k][0].y, v[k][0].z, v[k][0].w,
                             v[k][1].x, v[k][1].y, v[k][1].z, v[k][1].w};
      uint32_t y[8];
      const float4* turns =
          reinterpret_cast<const float4*>(s_turn + row[k] * p.rot_pairs + 8 * unit[k]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 cs = turns[e];  // of two pairs
        if (kInterleaved) {
          y[2 * e] = pack2(lo_of(w[2 * e]) * cs.x - hi_of(w[2 * e]) * cs.y,
                           hi_of(w[2 * e]) * cs.x + lo_of(w[2 * e]) * cs.y);
          y[2 * e + 1] = pack2(lo_of(w[2 * e + 1]) * cs.z - hi_of(w[2 * e + 1]) * cs.w,
                               hi_of(w[2 * e + 1]) * cs.z + lo_of(w[2 * e + 1]) * cs.w);
        } else {
          const uint32_t a = w[e], b = w[4 + e];
          y[e] = pack2(lo_of(a) * cs.x - lo_of(b) * cs.y, hi_of(a) * cs.z - hi_of(b) * cs.w);
          y[4 + e] = pack2(lo_of(b) * cs.x + lo_of(a) * cs.y, hi_of(b) * cs.z + hi_of(a) * cs.w);
        }
      }
      *reinterpret_cast<uint4*>(to[k]) = make_uint4(y[0], y[1], y[2], y[3]);
      *reinterpret_cast<uint4*>(to[k] + (kInterleaved ? 8 : p.rot_pairs)) =
          make_uint4(y[4], y[5], y[6], y[7]);
    }
  }
}

}  // namespace

void rope_table(int rot_dim, double base, const dcp_rope_scaling* scaling, uint64_t* table,
                float* amplitude) {
  const int n = rot_dim / 2;
  const double two_pi = 6.283185307179586476925;
  double lo = 0.0, hi = 0.0, up = 1.0;
  const bool parts = scaling != nullptr && scaling->kind == DCP_ROPE_YARN;
  if (parts) {
    // the pair that turns `turns` times within the original length; the slow one may lie behind the
    // last pair, and the ramp then does not reach 1
    auto pair = [&](double turns) {
      return n * std::log(scaling->original_len / (turns * two_pi)) / std::log(base);
    };
    lo = std::fmax(0.0, std::floor(pair(scaling->beta_fast)));
    hi = std::fmin(rot_dim - 1.0, std::ceil(pair(scaling->beta_slow)));
    up = scaling->amplitude > 0.0 ? scaling->amplitude
         : scaling->factor > 1.0  ? 0.1 * std::log(scaling->factor) + 1.0
                                  : 1.0;
  }
  for (int i = 0; i < n; ++i) {
    const double f = std::pow(base, -(double)i / n);
    double g = f;
    if (parts) {
      const double r = std::fmin(1.0, std::fmax(0.0, (i - lo) / std::fmax(hi - lo, 0.001)));
      g = f * (1.0 - r) + f / scaling->factor * r;
    } else if (scaling != nullptr) {
      g = f / scaling->factor;
    }
    const double turns = g / two_pi;  // whole turns do not count
    table[i] = (uint64_t)std::floor(std::ldexp(turns - std::floor(turns), 64) + 0.5);
  }
  *amplitude = (float)up;
}

cudaError_t launch_rope(int rows, int dim, int rot_dim, bool interleaved, const int32_t* positions,
                        const uint64_t* table, float amplitude, const dcp_rope_heads& a,
                        const dcp_rope_heads* b, cudaStream_t stream) {
  RopeParams p;
  auto side = [](const dcp_rope_heads& h) {
    return RopeSide{static_cast<const uint16_t*>(h.x), static_cast<uint16_t*>(h.out), h.x_row,
                    h.x_head, h.out_row, h.out_head, h.heads};
  };
  p.a = side(a);
  p.b = b != nullptr ? side(*b) : RopeSide{};
  p.positions = positions;
  p.table = table;
  p.amplitude = amplitude;
  p.rows = rows;
  p.rot_pairs = rot_dim / 2;
  p.units = rot_dim / 16;
  const bool in_place = a.x == a.out && (b == nullptr || b->x == b->out);
  p.copies = in_place ? 0 : (dim - rot_dim) / 8;
  const int heads = p.a.heads + p.b.heads, per_head = p.units + p.copies;
  // Rows of a CTA: as many as it has threads for cosines and sines, fewer while that leaves
  // SMs without a CTA (two CTAs to an SM 50.6 us for 8192 rows, one or four the same, eight 54.5);
  // heads in several CTAs where the rows are few.
  const int most = std::max(1, kRopeThreads / p.rot_pairs);
  p.row_count = std::max(1, std::min(most, rows / (2 * kSms)));
  p.unit_div = FastDiv::by(per_head);
  p.head_div = FastDiv::by(heads);
  p.pair_div = FastDiv::by(p.rot_pairs);
  const int grid_x = (rows + p.row_count - 1) / p.row_count;
  const int64_t threads = (int64_t)p.row_count * heads * per_head;
  const int64_t want = (threads + kRopeThreads - 1) / kRopeThreads;
  const int grid_y = (int)std::max<int64_t>(1, std::min<int64_t>(want, 4 * kSms / std::max(1, grid_x)));
  const dim3 grid((unsigned)grid_x, (unsigned)grid_y);
  if (interleaved) rope_kernel<true><<<grid, kRopeThreads, 0, stream>>>(p);
  else rope_kernel<false><<<grid, kRopeThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace dcpmla
