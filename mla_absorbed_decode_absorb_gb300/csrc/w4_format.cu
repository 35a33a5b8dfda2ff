// bf16 weights into the 4-bit format with group scales, and back.
//
//   s = bf16(max|w| / 7) over each 128 columns of a row (1 where that is zero)
//   u = clamp(round(w / s), -8, 7) + 8        w' = bf16((u - 8) s)
//
// The codes are those of exact arithmetic.  w and s have 8 significant bits, so
// a quotient w / s of at most 8 is either a tie k + 1/2 exactly or at least
// 2^-10 away from one.  w times an approximate 1 / s is off by at most 2^-19; added
// to 3 * 2^10, whose unit in the last place is 2^-12, it is rounded to a multiple of
// 2^-12: a tie becomes the tie again and nothing else becomes one.  Likewise
// max * (1 / 7) rounds to the bf16 that max / 7 rounds to, which is never within
// 2^-13 of a tie.  (With IEEE divisions and a rounding instruction per weight the
// kernel was bound by them: 7168 x 16384 took 71 us, against 50 now, 0.87 of the
// measured copy bandwidth; the way back takes 47 us, 0.93.)
//
// 16 lanes hold a group, 8 columns each; a thread has kUnits groups in flight,
// kThreads / 16 apart.  Both kernels stream.
#include "w4.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;                           // groups per thread
constexpr int kPerBlock = kThreads / 16 * kUnits;   // groups per CTA

// Where unit u (a group of 128 columns of one row) and lane `sub` of it lie:
// element offset of its 8 columns, and whether they exist.  K % 128 = 0 makes the
// weight one run of groups; else (kRagged) a row's last group has 64 columns.
template <bool kRagged>
__device__ __forceinline__ bool w4_place(uint32_t u, uint32_t units, uint32_t groups, int K, int sub, int64_t* at) {
  if (!kRagged) {
    *at = static_cast<int64_t>(u) * kW4Group + sub * 8;
    return u < units;
  }
  const uint32_t row = u / groups;
  const int col = static_cast<int>(u - row * groups) * kW4Group + sub * 8;
  *at = static_cast<int64_t>(row) * K + col;
  return u < units && col < K;
}

template <bool kRagged>
__global__ void __launch_bounds__(kThreads)
quantize_w4_kernel(const uint16_t* __restrict__ w, uint32_t* __restrict__ w4, uint16_t* __restrict__ scale,
                   uint32_t units, uint32_t groups, int K) {
  grid_dep_wait();
  grid_dep_launch();
  const int sub = threadIdx.x & 15;
  const uint32_t u0 = blockIdx.x * kPerBlock + (threadIdx.x >> 4);
  uint4 v[kUnits];
  int64_t at[kUnits];
  bool in[kUnits];
#pragma unroll
  for (int q = 0; q < kUnits; ++q) {
    in[q] = w4_place<kRagged>(u0 + q * (kThreads / 16), units, groups, K, sub, &at[q]);
    v[q] = in[q] ? *reinterpret_cast<const uint4*>(w + at[q]) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int q = 0; q < kUnits; ++q) {
    const uint32_t bits[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(bits[i] << 16);
      x[2 * i + 1] = __uint_as_float(bits[i] & 0xffff0000u);
    }
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(x[i]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    uint16_t sb = f32_to_bf16_bits(a * (1.f / 7.f));
    if (sb == 0) sb = 0x3f80;  // a group of zeros (or below bf16's smallest scale): s = 1
    const float s = bf16_bits_to_f32(sb);
    uint32_t word = 0;
    if (s >= 0x1p-100f) {
      // |w / s| < 7.5: no clamp.  c + 8 + 3 * 2^22 is an integer whose low four bits are the code; the eight are
      // summed at their places and the constant parts taken off together (mod 2^32).
      const float rs = __fdividef(1.f, s);
#pragma unroll
      for (int i = 7; i >= 0; --i)
        word = word * 16 + __float_as_uint(__fsub_rn(fmaf(x[i], rs, 0x1.8p11f), 0x1.8p11f) + 12582920.f);
      word -= 0x4b400000u * 0x11111111u;
    } else {
      // a scale so small that its reciprocal overflows, or itself rounded coarsely: 2^64 times both, and clamped
      const float rs = __fdividef(1.f, s * 0x1p64f);
#pragma unroll
      for (int i = 7; i >= 0; --i) {
        const float c = __fsub_rn(fmaf(x[i] * 0x1p64f, rs, 0x1.8p11f), 0x1.8p11f);
        word = word * 16 + (__float_as_uint(fminf(fmaxf(c, -8.f), 7.f) + 12582920.f) & 15u);
      }
    }
    const uint32_t u = u0 + q * (kThreads / 16);
    if (in[q]) w4[at[q] >> 3] = word;
    if (u < units && sub == 0) scale[u] = sb;
  }
}

template <bool kRagged>
__global__ void __launch_bounds__(kThreads)
dequantize_w4_kernel(const uint32_t* __restrict__ w4, const uint16_t* __restrict__ scale, uint16_t* __restrict__ w,
                     uint32_t units, uint32_t groups, int K) {
  grid_dep_wait();
  grid_dep_launch();
  const int sub = threadIdx.x & 15;
  const uint32_t u0 = blockIdx.x * kPerBlock + (threadIdx.x >> 4);
  uint32_t v[kUnits], s[kUnits];
  int64_t at[kUnits];
  bool in[kUnits];
#pragma unroll
  for (int q = 0; q < kUnits; ++q) {
    const uint32_t u = u0 + q * (kThreads / 16);
    in[q] = w4_place<kRagged>(u, units, groups, K, sub, &at[q]);
    v[q] = in[q] ? w4[at[q] >> 3] : 0;
    s[q] = in[q] ? scale[u] * 0x10001u : 0;  // the scale in both halves
  }
#pragma unroll
  for (int q = 0; q < kUnits; ++q) {
    uint32_t p[4];
    w4_pairs(v[q], p);
    // (u - 8) s has 12 significant bits: the bf16 product is the rounded exact one
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(p[i]) : "r"(p[i]), "r"(s[q]));
    if (in[q])
      *reinterpret_cast<uint4*>(w + at[q]) =
          make_uint4(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410),
                     __byte_perm(p[0], p[1], 0x7632), __byte_perm(p[2], p[3], 0x7632));
  }
}

unsigned blocks_for(uint32_t units) { return static_cast<unsigned>((static_cast<uint64_t>(units) + kPerBlock - 1) / kPerBlock); }

}  // namespace

cudaError_t launch_quantize_w4(const uint16_t* w, uint8_t* w4, uint16_t* scale, int N, int K, cudaStream_t stream) {
  const uint32_t groups = w4_groups(K), units = static_cast<uint32_t>(N) * groups;
  auto kernel = K % kW4Group != 0 ? quantize_w4_kernel<true> : quantize_w4_kernel<false>;
  return launch_kernel(kernel, dim3(blocks_for(units)), dim3(kThreads), 0, stream, w,
                       reinterpret_cast<uint32_t*>(w4), scale, units, groups, K);
}

cudaError_t launch_dequantize_w4(const uint8_t* w4, const uint16_t* scale, uint16_t* w, int N, int K,
                                 cudaStream_t stream) {
  const uint32_t groups = w4_groups(K), units = static_cast<uint32_t>(N) * groups;
  auto kernel = K % kW4Group != 0 ? dequantize_w4_kernel<true> : dequantize_w4_kernel<false>;
  return launch_kernel(kernel, dim3(blocks_for(units)), dim3(kThreads), 0, stream,
                       reinterpret_cast<const uint32_t*>(w4), scale, w, units, groups, K);
}

}  // namespace mla
