// Rotary positions: pair i of a head's first rot_dim values is turned by
// position * freq[i] and multiplied by a gain,
//   (u, w) -> gain (u cos a - w sin a, u sin a + w cos a).
//
// What bounds it: every value is read once and written once, 4 bytes, and the
// angles are the same for all heads of a row.  So a block takes one row or two,
// computes their sines and cosines once into shared memory, and its threads each
// turn 16 values (two 16-byte pieces) at a time.  16384 rows of 48 heads of 128:
// 60.6 us, 6.6 TB/s, what a plain copy of them takes (one row a block: 62 to 69 us,
// four: 63, eight: 68; without the streaming hints 61 to 62; two units in flight
// a thread 67).
//
// Angles: a double's freq / 2 pi as a 64-bit fraction of a turn, times the
// position modulo 2^64, is the angle modulo a turn without any reduction: off
// by less than position * 2^-53 of its frequency and 2^-33 of a turn.  The
// signed fraction goes through sincospif.
#include <cmath>

#include "tv_kernels.cuh"
#include "tv_pages.cuh"

namespace tv {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxBlockRows = 2;
constexpr int kPairs = TV_ROPE_MAX_PAIRS;

struct RopeRows {
  const __nv_bfloat16* x;
  __nv_bfloat16* out;
  const int32_t* pos;
  int32_t* status;
  size_t x_stride, out_stride;
  int rows, heads, head_dim, rot, per;   // per: rows of a block
  float gain;
  uint64_t turn[kPairs];                 // of a position, in 2^-64
};

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pair_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A unit is 16 values of a head: pieces 8 j .. + 7 of the first and of the
// second half of what turns, or 16 neighbours.  Its sines and cosines are four
// 16-byte chunks of two pairs each; chunk c of unit j lies at c * units + j, so
// that the lanes of a warp, on neighbouring units, read neighbouring chunks.
template <bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeRows p) {
  __shared__ float4 s_turn[kMaxBlockRows][kPairs / 2];
  __shared__ int s_stop;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, row0 = blockIdx.x * p.per, nr = min(p.per, p.rows - row0);
  const int units = p.head_dim / 16, turning = p.rot / 16, pairs = p.rot / 2;
  if (tid == 0) s_stop = status_get(p.status);
  for (int i = tid; i < nr * pairs; i += kRopeThreads) {
    const int r = i / pairs, k = i % pairs;
    const int64_t a = (int64_t)((uint64_t)(int64_t)__ldg(p.pos + row0 + r) * p.turn[k]);
    float s, c;
    sincospif((float)(int32_t)(a >> 32) * 0x1p-31f, &s, &c);
    reinterpret_cast<float2*>(s_turn[r])[((k % 8 / 2) * turning + k / 8) * 2 + k % 2] = make_float2(c * p.gain, s * p.gain);
  }
  __syncthreads();
  if (s_stop != 0) return;
  const uint32_t per_row = (uint32_t)p.heads * units, all = per_row * nr;
  for (uint32_t i = tid; i < all; i += kRopeThreads) {
    const uint32_t r = i / per_row, e = i - r * per_row, h = e / units, j = e % units;
    const bool turns = (int)j < turning;
    // the unit's two pieces of 8 values
    const uint32_t d0 = INTER || !turns ? 16 * j : 8 * j, d1 = INTER || !turns ? 16 * j + 8 : p.rot / 2 + 8 * j;
    const size_t head = (size_t)h * p.head_dim;
    const __nv_bfloat16* x = p.x + (size_t)(row0 + r) * p.x_stride + head;
    __nv_bfloat16* y = p.out + (size_t)(row0 + r) * p.out_stride + head;
    uint4 a = __ldcs(reinterpret_cast<const uint4*>(x + d0)), b = __ldcs(reinterpret_cast<const uint4*>(x + d1));
    if (turns) {
      uint32_t u[4] = {a.x, a.y, a.z, a.w}, w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {   // pairs 8 j + 2 c and the next
        const float4 t = s_turn[r][c * turning + j];   // cos, sin, cos, sin
        if (INTER) {
          uint32_t& v = c < 2 ? u[2 * c] : w[2 * c - 4];
          uint32_t& z = c < 2 ? u[2 * c + 1] : w[2 * c - 3];
          v = pair_bf16(lo_f(v) * t.x - hi_f(v) * t.y, lo_f(v) * t.y + hi_f(v) * t.x);
          z = pair_bf16(lo_f(z) * t.z - hi_f(z) * t.w, lo_f(z) * t.w + hi_f(z) * t.z);
        } else {
          const float u0 = lo_f(u[c]), u1 = hi_f(u[c]), w0 = lo_f(w[c]), w1 = hi_f(w[c]);
          u[c] = pair_bf16(u0 * t.x - w0 * t.y, u1 * t.z - w1 * t.w);
          w[c] = pair_bf16(u0 * t.y + w0 * t.x, u1 * t.w + w1 * t.z);
        }
      }
      a = make_uint4(u[0], u[1], u[2], u[3]);
      b = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (turns || y != x) {
      __stcs(reinterpret_cast<uint4*>(y + d0), a);
      __stcs(reinterpret_cast<uint4*>(y + d1), b);
    }
  }
}

bool finite_all(const double* x, int n) {
  for (int i = 0; i < n; ++i)
    if (!std::isfinite(x[i])) return false;
  return true;
}

}  // namespace
}  // namespace tv

using namespace tv;

extern "C" {

int tv_rope_init(tv_rope* rope, int rot_dim, int interleaved, double theta, int scaling, double factor,
                 int32_t original_ctx, double low_turns, double high_turns, double gain) {
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  if (!rope || rot_dim < 16 || rot_dim > 2 * TV_ROPE_MAX_PAIRS || rot_dim % 16 != 0) return TV_E_ARG;
  if (interleaved != 0 && interleaved != 1) return TV_E_ARG;
  if (!std::isfinite(theta) || theta <= 0.0 || !std::isfinite((float)gain)) return TV_E_ARG;
  if (scaling < TV_ROPE_PLAIN || scaling > TV_ROPE_BLEND) return TV_E_ARG;
  if (scaling != TV_ROPE_PLAIN && (!std::isfinite(factor) || factor <= 0.0)) return TV_E_ARG;
  if (scaling == TV_ROPE_BLEND &&
      (original_ctx < 1 || !(low_turns >= 0.0) || !(high_turns > low_turns) || !std::isfinite(high_turns)))
    return TV_E_ARG;
  if (scaling == TV_ROPE_BASE) theta *= std::pow(factor, rot_dim / (rot_dim - 2.0));
  if (!std::isfinite(theta) || theta <= 0.0) return TV_E_ARG;   // beyond what a double holds
  tv_rope r = {};
  r.rot_dim = rot_dim;
  r.interleaved = interleaved;
  r.gain = gain;
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / rot_dim);
    if (scaling == TV_ROPE_LINEAR) f /= factor;
    if (scaling == TV_ROPE_BLEND) {
      double keep = (original_ctx * f / kTwoPi - low_turns) / (high_turns - low_turns);
      keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
      f = f * keep + f / factor * (1.0 - keep);
    }
    r.freq[i] = f;
  }
  if (!finite_all(r.freq, rot_dim / 2)) return TV_E_ARG;   // (nor may the frequencies be)
  *rope = r;
  return TV_OK;
}

int tv_rope_rows(const tv_rope* rope, const tv_bf16* x, size_t x_stride, tv_bf16* out, size_t out_stride, int n_heads,
                 int head_dim, const int32_t* positions, int rows, int32_t* dev_status, void* stream) {
  if (!rope || !x || !out || !positions || !dev_status || n_heads < 1 || rows < 1) return TV_E_ARG;
  if (rope->rot_dim < 16 || rope->rot_dim > 2 * kPairs || rope->rot_dim % 16 != 0) return TV_E_ARG;
  if ((rope->interleaved != 0 && rope->interleaved != 1) || !std::isfinite((float)rope->gain)) return TV_E_ARG;
  if (!finite_all(rope->freq, rope->rot_dim / 2)) return TV_E_ARG;
  if ((head_dim != 64 && head_dim != 128) || rope->rot_dim > head_dim || n_heads > 65536) return TV_E_UNSUPPORTED;
  if (!aligned16(x) || !aligned16(out) || x_stride % 8 != 0 || out_stride % 8 != 0) return TV_E_ARG;
  const size_t width = (size_t)n_heads * head_dim;
  if (x_stride < width || out_stride < width || (out == x && out_stride != x_stride)) return TV_E_ARG;
  const int sms = num_sms();
  if (sms <= 0) return TV_E_CUDA;
  RopeRows p;
  p.x = reinterpret_cast<const __nv_bfloat16*>(x);
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.pos = positions;
  p.status = dev_status;
  p.x_stride = x_stride;
  p.out_stride = out_stride;
  p.rows = rows;
  p.heads = n_heads;
  p.head_dim = head_dim;
  p.rot = rope->rot_dim;
  p.gain = (float)rope->gain;
  // a block a row until every SM has eight; then two
  p.per = 1;
  while (p.per < kMaxBlockRows && rows / (2 * p.per) >= 8 * sms) p.per *= 2;
  for (int i = 0; i < kPairs; ++i) {
    // a fraction of a turn, negative ones modulo one (the highest double below 1 is below 2^64 here, too)
    double t = i < p.rot / 2 ? rope->freq[i] / 6.283185307179586476925286766559 : 0.0;
    if (t >= 1.0 || t <= -1.0) t = std::fmod(t, 1.0);
    p.turn[i] = t < 0.0 ? 0ull - (uint64_t)(-t * 0x1p64) : (uint64_t)(t * 0x1p64);
  }
  const unsigned grid = (unsigned)((rows - 1) / p.per + 1);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return launch_pdl(rope->interleaved ? rope_kernel<true> : rope_kernel<false>, dim3(grid), dim3(kRopeThreads), 0, st, p);
}

}  // extern "C"
