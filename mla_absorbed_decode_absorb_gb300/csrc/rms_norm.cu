// Root-mean-square norm of [T, D] rows, with the residual's addition before it
// and a bf16 or an 8-bit output:
//
//   h = x + r            r_out = bf16(h)
//   y = h / sqrt(mean(h^2) + eps) * w
//   y_out = bf16(y)      or, for each 128 columns, s = max(max|y| / 448, 2^-100)
//                        and codes E4M3(y / s)
//
// One CTA owns one row and keeps it in registers between the two sweeps the
// formula needs (the sum of squares, then the scaling), so x and r are read
// once.  The sum, h and y stay in fp32: y comes from the unrounded h, and each
// output is rounded once.  A group of 128 columns is 16 neighbouring lanes of 8
// columns each, so its maximum is four shuffles.  Bound by HBM for many rows, by the launch and one
// round trip to memory for few (1 x 7168: 1.9 us).
#include "append_row.cuh"

namespace mla {
namespace {

constexpr float kScaleFloor = 7.888609052210118e-31f;  // 2^-100

struct NormParams {
  const uint16_t* x;
  const uint16_t* r;      // nullptr: no residual
  const uint16_t* w;
  uint16_t* r_out;
  uint16_t* y;            // bf16 output, or nullptr
  uint8_t* y8;            // 8-bit output, or nullptr
  float* s8;
  int64_t x_ld;
  int T, D, groups;
  float eps;
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// kChunks chunks of 8 columns per thread: chunk i of a thread is its index in
// the row + i * kSpan, kSpan threads to a row.  kSpan is a multiple of 32, so 16
// neighbouring lanes always hold one whole group of 128 columns.  kSpan = 32: a
// warp per row, kThreads / 32 rows per CTA; otherwise one row per CTA, which may
// have fewer threads than kThreads (kSpan = 0).
// (Threads of one or two chunks are held to 32 registers, which keeps an SM's 2048 threads in flight.)
template <int kChunks, int kThreads, int kSpan>
__global__ void __launch_bounds__(kThreads, kChunks <= 2 && kSpan == 0 ? 2048 / kThreads : 1)
rms_norm_kernel(const NormParams p) {
  __shared__ float warp_sum[kSpan == 32 ? 1 : 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tid = kSpan == 32 ? lane : static_cast<int>(threadIdx.x);
  const int span = kSpan == 32 ? 32 : static_cast<int>(blockDim.x);
  const int64_t row = kSpan == 32 ? static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + warp : blockIdx.x;
  const int chunks = p.D >> 3;
  grid_dep_wait();
  grid_dep_launch();
  if (kSpan == 32 && row >= p.T) return;

  const uint4* x = reinterpret_cast<const uint4*>(p.x + row * p.x_ld);
  const int64_t base = row * chunks;
  uint4 xv[kChunks], rv[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = tid + i * span;
    xv[i] = rv[i] = make_uint4(0, 0, 0, 0);
    if (c < chunks) {
      xv[i] = x[c];
      if (p.r != nullptr) rv[i] = reinterpret_cast<const uint4*>(p.r)[base + c];
    }
  }
  float h[kChunks][8];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = tid + i * span;
    unpack8(xv[i], h[i]);
    if (p.r != nullptr) {
      float r[8];
      unpack8(rv[i], r);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i][e] += r[e];
      if (c < chunks) reinterpret_cast<uint4*>(p.r_out)[base + c] = pack8(h[i]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(h[i][e], h[i][e], sum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (kSpan != 32) {
    if (lane == 0) warp_sum[warp] = sum;
    __syncthreads();
    // every warp adds the warps' sums in the same order
    sum = lane < static_cast<int>(blockDim.x >> 5) ? warp_sum[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  // The factor's power of two goes into h at once (exact), what is left is in [1, 2): h w alone could leave fp32's range
  // where v does not.  An infinity or a NaN stays whole.
  float inv = __fdiv_rn(1.f, __fsqrt_rn(__fdiv_rn(sum, static_cast<float>(p.D)) + p.eps));
  float power = __uint_as_float(__float_as_uint(inv) & 0x7f800000u);
  if (power == __uint_as_float(0x7f800000u)) {
    power = inv;
    inv = 1.f;
  } else {
    inv = __uint_as_float((__float_as_uint(inv) & 0x007fffffu) | 0x3f800000u);
  }
#pragma unroll
  for (int i = 0; i < kChunks; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) h[i][e] *= power;

#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = tid + i * span;
    float w[8];
    unpack8(c < chunks ? reinterpret_cast<const uint4*>(p.w)[c] : make_uint4(0, 0, 0, 0), w);
    if (p.y != nullptr && c < chunks) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = h[i][e] * inv * w[e];
      reinterpret_cast<uint4*>(p.y)[base + c] = pack8(v);
    }
    if (p.y8 != nullptr) {
      // v / s = h w * (448 / max|h w|): the row's factor cancels, and with it its rounding
      float a = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[i][e] *= w[e];
        a = fmaxf(a, fabsf(h[i][e]));
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
      const float s = fmaxf(__fdiv_rn(a * inv, 448.f), kScaleFloor);
      // at the floor (also where the row is not finite, or a is 0) the codes are v / 2^-100
      const bool at_floor = s == kScaleFloor;
      const float f = at_floor ? inv : __fdiv_rn(448.f, a), g = at_floor ? 0x1p100f : 1.f;
      uint16_t q[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) q[e] = e4m3x2(h[i][2 * e] * f * g, h[i][2 * e + 1] * f * g);
      if (c < chunks) {
        reinterpret_cast<uint2*>(p.y8)[base + c] =
            make_uint2(q[0] | (static_cast<uint32_t>(q[1]) << 16), q[2] | (static_cast<uint32_t>(q[3]) << 16));
        if ((c & 15) == 0) p.s8[row * p.groups + (c >> 4)] = s;
      }
    }
  }
}

template <int kChunks, int kThreads, int kSpan>
cudaError_t launch_shape(const NormParams& p, cudaStream_t stream) {
  const int chunks = p.D >> 3;
  const int rows = kSpan == 32 ? kThreads / 32 : 1;
  const int threads = kSpan == 32 ? kThreads : ((chunks + kChunks - 1) / kChunks + 31) / 32 * 32;
  const unsigned ctas = (static_cast<unsigned>(p.T) + rows - 1) / rows;  // T + rows - 1 may be no int
  return launch_kernel(rms_norm_kernel<kChunks, kThreads, kSpan>, dim3(ctas), dim3(threads), 0, stream, p);
}

}  // namespace

cudaError_t launch_rms_norm(const uint16_t* x, int64_t x_ld, const uint16_t* residual, uint16_t* residual_out,
                            const uint16_t* w, float eps, uint16_t* y, uint8_t* y8, float* y8_scale, int T, int D,
                            cudaStream_t stream) {
  const NormParams p{x, residual, w, residual_out, y, y8, y8_scale, x_ld, T, D, (D + 127) / 128, eps};
  const int chunks = D >> 3;
  // 512 columns or fewer in many rows: a warp per row (16384 x 512: 8.1 us, against 17.5 with a CTA of two warps
  // per row, which the rate of CTA launches bounds; 256 rows: 1.8 against 1.6 us)
  if (chunks <= 64 && T >= 1024) return launch_shape<2, 256, 32>(p, stream);
  // one chunk per thread while the rows fit the GPU at once (32 x 1536: 1.8 us, against 2.1 with two chunks;
  // 128 x 7168: 3.4 against 3.9), then two, which keep twice the bytes in flight per register (16384 x 7168 with
  // the residual, 8-bit output: 123 us against 155, 0.99 of the measured copy bandwidth; four chunks: 122)
  if (chunks <= 1024 && static_cast<int64_t>(T) * chunks <= 152 * 2048) return launch_shape<1, 1024, 0>(p, stream);
  if (chunks <= 1024) return launch_shape<2, 512, 0>(p, stream);
  return launch_shape<4, 512, 0>(p, stream);  // up to 16384 columns (8192 rows: 156 us, 1.01)
}

}  // namespace mla
