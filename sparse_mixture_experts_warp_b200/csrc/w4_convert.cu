// Conversion of expert weights to and from the 4-bit form (w4.cuh): moe_quantize_w4 and
// moe_dequantize_w4.
//
// Per row n of a matrix and group of g consecutive k, in fp32 with IEEE division and
// round-to-nearest-even throughout:
//   t = max |w| / 7                                      without zero points
//   t = (max(w, 0) - min(w, 0)) / 15                     with them
//   row_scale = max over the row's groups of t / 448     (448: the largest e4m3 number)
//   scale = e4m3(t / row_scale);  step = scale * row_scale;  r = 1 / step   (all 0 if t is 0)
//   code = clamp(rint(w r), -8, 7) + 8                   without zero points
//   zero = clamp(rint(-min(w, 0) r), 0, 15), code = clamp(rint(w r) + zero, 0, 15)   with them
// A row that holds a NaN or an infinity gets row_scale NaN or infinity and stands for NaN; a row
// whose largest t is below 2^-100 counts as zeros (row_scale 0), so 1 / step is always finite.
//
// Both directions stream memory: the wide weights once, the 4-bit form once.
#include "common.cuh"
#include "w4.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <bool BF16> struct Eight;              // eight consecutive weights as stored
template <> struct Eight<true> {
  uint4 a;
  __device__ __forceinline__ void load(const void* base, int64_t i) {
    a = __ldcs(static_cast<const uint4*>(base) + i);
  }
  __device__ __forceinline__ void widen(float (&w)[8]) const {
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[2 * i] = __uint_as_float(u[i] << 16);
      w[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
};
template <> struct Eight<false> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* base, int64_t i) {
    a = __ldcs(static_cast<const float4*>(base) + 2 * i);
    b = __ldcs(static_cast<const float4*>(base) + 2 * i + 1);
  }
  __device__ __forceinline__ void widen(float (&w)[8]) const {
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
};

// A block takes one row; a thread eight consecutive k (one word of codes) at a time, so the g / 8
// threads of a group are neighbouring lanes.  The row is read twice (the second time from
// cache): once for its largest step, once to quantise.
constexpr int kQThreads = 128;

template <bool BF16, bool ZEROS>
__global__ void __launch_bounds__(kQThreads)
quantize_w4_kernel(const void* __restrict__ W, int N, int K, int g, uint32_t* __restrict__ codes,
                   uint8_t* __restrict__ scales, uint8_t* __restrict__ zeros,
                   float* __restrict__ row_scale) {
  pdl_trigger();
  pdl_wait();
  __shared__ float s_max[kQThreads / 32];
  const int64_t row = blockIdx.x;               // matrix * N + n
  const int64_t m = row / N;
  const int n = (int)(row - m * N);
  const int words = K / 8, gw = g / 8, groups = (K + g - 1) / g;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rounds = (words + kQThreads - 1) / kQThreads;

  // the group's raw step t and smallest weight, in every lane of the group
  auto group_step = [&](const float (&w)[8], float& lo) {
    float hi = ZEROS ? 0.f : fabsf(w[0]);
    lo = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      hi = max_nan(hi, ZEROS ? w[i] : fabsf(w[i]));
      if (ZEROS) lo = min_nan(lo, w[i]);
    }
    for (int o = 1; o < gw; o <<= 1) {
      hi = max_nan(hi, __shfl_xor_sync(kFull, hi, o));
      if (ZEROS) lo = min_nan(lo, __shfl_xor_sync(kFull, lo, o));
    }
    return ZEROS ? __fdiv_rn(hi - lo, 15.f) : __fdiv_rn(hi, 7.f);
  };

  float most = 0.f;
  for (int r = 0; r < rounds; ++r) {
    const int i = r * kQThreads + threadIdx.x;
    float w[8] = {}, lo;
    if (i < words) {
      Eight<BF16> e;
      e.load(W, row * words + i);
      e.widen(w);
    }
    most = max_nan(most, group_step(w, lo));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = max_nan(most, __shfl_xor_sync(kFull, most, o));
  if (lane == 0) s_max[warp] = most;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kQThreads / 32; ++i) most = max_nan(most, s_max[i]);
  const float rs = most < 0x1p-100f ? 0.f : __fdiv_rn(most, 448.f);
  if (threadIdx.x == 0) row_scale[row] = rs;

  for (int r = 0; r < rounds; ++r) {
    const int i = r * kQThreads + threadIdx.x;
    float w[8] = {}, lo;
    if (i < words) {
      Eight<BF16> e;
      e.load(W, row * words + i);
      e.widen(w);
    }
    const float t = group_step(w, lo);
    if (i >= words) continue;
    const __nv_fp8_e4m3 sc(rs > 0.f ? __fdiv_rn(t, rs) : 0.f);
    const float step = static_cast<float>(sc) * rs;
    const float inv = step > 0.f ? __fdiv_rn(1.f, step) : 0.f;
    float z = 8.f;
    if (ZEROS) z = fminf(fmaxf(rintf(-lo * inv), 0.f), 15.f);
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float q = rintf(w[e] * inv);
      q = ZEROS ? fminf(fmaxf(q + z, 0.f), 15.f) : fminf(fmaxf(q, -8.f), 7.f) + 8.f;
      word |= (uint32_t)q << (4 * (e / 2 + 4 * (e & 1)));
    }
    // words of a block are 8 consecutive k each: k / 8 = 8 b + 4 j + c is word 8 b + 2 c + j
    const int b = i >> 3, j = (i >> 2) & 1, c = i & 3;
    codes[row * words + 8 * b + 2 * c + j] = word;
    if (i % gw == 0) {
      const int64_t at = (m * groups + i / gw) * N + n;
      scales[at] = sc.__x;
      if (ZEROS) zeros[at] = (uint8_t)z;
    }
  }
}

// One word of codes (eight consecutive weights) a thread.
template <bool BF16>
__global__ void __launch_bounds__(256)
dequantize_w4_kernel(const W4Ptrs w, int64_t total, int N, int K, int g, void* __restrict__ out) {
  pdl_trigger();
  pdl_wait();
  const int words = K / 8, groups = (K + g - 1) / g;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = i / words;              // i: 8 weights from k = 8 kw on
    const int kw = (int)(i - row * words);
    const int64_t m = row / N;
    const int n = (int)(row - m * N);
    const int b = kw >> 3, j = (kw >> 2) & 1, c = kw & 3;
    const uint32_t word = w.codes[row * words + 8 * b + 2 * c + j];
    const int64_t at = (m * groups + 8 * kw / g) * N + n;
    const float sc = w4_scale(w.scales[at]), rs = w.row_scale[row];
    const float z = w.zeros ? (float)w.zeros[at] : 8.f;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = rs * (sc * ((float)((word >> (4 * (e / 2 + 4 * (e & 1)))) & 15u) - z));
    if (BF16) {
      uint32_t p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
        p[e] = *reinterpret_cast<const uint32_t*>(&h);
      }
      __stcs(static_cast<uint4*>(out) + i, make_uint4(p[0], p[1], p[2], p[3]));
    } else {
      float4* o = static_cast<float4*>(out) + 2 * i;
      __stcs(o, make_float4(v[0], v[1], v[2], v[3]));
      __stcs(o + 1, make_float4(v[4], v[5], v[6], v[7]));
    }
  }
}

}  // namespace

cudaError_t launch_quantize_w4(int n_matrices, int N, int K, bool bf16, const void* W,
                               const moe_w4_t& o, cudaStream_t s) {
  const dim3 grid((unsigned)((int64_t)n_matrices * N)), block(kQThreads);
  auto k = bf16 ? (o.zeros ? quantize_w4_kernel<true, true> : quantize_w4_kernel<true, false>)
                : (o.zeros ? quantize_w4_kernel<false, true> : quantize_w4_kernel<false, false>);
  return launch_pdl(k, grid, block, 0, s, W, N, K, o.group, reinterpret_cast<uint32_t*>(o.codes),
                    o.scales, o.zeros, o.row_scale);
}

cudaError_t launch_dequantize_w4(int n_matrices, int N, int K, const moe_w4_t& w, bool bf16,
                                 void* out, cudaStream_t s) {
  const int64_t total = (int64_t)n_matrices * N * (K / 8);
  const int64_t blocks = (total + 255) / 256, most = (int64_t)num_sms() * 16;
  const dim3 grid((unsigned)(blocks < most ? blocks : most)), block(256);
  const W4Ptrs p{reinterpret_cast<const uint32_t*>(w.codes), w.scales, w.zeros, w.row_scale};
  auto k = bf16 ? dequantize_w4_kernel<true> : dequantize_w4_kernel<false>;
  return launch_pdl(k, grid, block, 0, s, p, total, N, K, w.group, out);
}

}  // namespace moe
