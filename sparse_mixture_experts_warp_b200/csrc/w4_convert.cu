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
// Both directions stream memory: the wide weights once, the 4-bit form once (8 x 14336 x 4096 with
// groups of 128, at the measured copy rate 183 us for bf16, 328 for fp32: quantise 235 and 337 us,
// dequantise 200 and 349, each alone; quantise, then dequantise, bf16, 460).  For bf16 the instructions cost more than that (schedulers 84% busy),
// which shapes both kernels: rounding by adding 1.5 * 2^23 and packing by multiply-add on the sums'
// bits instead of conversion instructions, a group's three divisions by one lane for the whole
// group, scales through shared memory (they are stored [group, row]: a row's own are N bytes
// apart).
#include <float.h>

#include <type_traits>

#include "common.cuh"
#include "w4.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kRound = 12582912.f;            // 1.5 * 2^23: x + kRound has rint(x) in its low bits
constexpr uint32_t kRoundBits = 0x4b400000u;

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
  __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void load(const void* base, int64_t i) {
    a = __ldcs(static_cast<const uint4*>(base) + i);
  }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
    return __uint_as_float(i & 1 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
  }
  // largest (magnitude, or weight and 0) and smallest (weight and 0), two at a time; NaN stay
  template <bool ZEROS>
  __device__ __forceinline__ void range(float& hi, float& lo) const {
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
    const __nv_bfloat162 none = __floats2bfloat162_rn(0.f, 0.f);
    __nv_bfloat162 most = none, least = none;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&u[i]);
      most = __hmax2_nan(most, ZEROS ? v : __habs2(v));
      if (ZEROS) least = __hmin2_nan(least, v);
    }
    hi = max_nan(__low2float(most), __high2float(most));
    lo = ZEROS ? min_nan(__low2float(least), __high2float(least)) : 0.f;
  }
};
template <> struct Eight<false> {
  float4 a, b;
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const void* base, int64_t i) {
    a = __ldcs(static_cast<const float4*>(base) + 2 * i);
    b = __ldcs(static_cast<const float4*>(base) + 2 * i + 1);
  }
  __device__ __forceinline__ float get(int i) const {
    const float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    return w[i];
  }
  template <bool ZEROS>
  __device__ __forceinline__ void range(float& hi, float& lo) const {
    hi = lo = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      hi = max_nan(hi, ZEROS ? get(i) : fabsf(get(i)));
      if (ZEROS) lo = min_nan(lo, get(i));
    }
  }
};

// A block takes `per_block` consecutive rows of a matrix, one after the other, a row with all its
// warps: a thread holds kWords runs of eight consecutive k (one word of codes each), so the g / 8
// threads of a group are neighbouring lanes.  Rows longer than the largest block holds are read
// again for their codes.
// Four words a lane: 8 took 295 us instead of 235 for 8 x 14336 x 4096 bf16, 2 took 348.
constexpr int kMaxWarps = 16, kWords = 4;
// the side tables of the longest rows (262144), groups of 32 with zero points, 4 rows a block
constexpr size_t kQuantMaxSmem = 262144 / 32 * 2 * 4;

template <bool BF16, bool ZEROS, int GROUP, bool TEAMS>
__global__ void __launch_bounds__(32 * kMaxWarps)
quantize_w4_kernel(const void* __restrict__ W, int N, int K, int per_block, int team_warps,
                   uint32_t* __restrict__ codes, uint8_t* __restrict__ scales,
                   uint8_t* __restrict__ zeros, float* __restrict__ row_scale) {
  extern __shared__ __align__(16) uint8_t s_side[];             // [groups][per_block] scales, zeros
  __shared__ float s_max[2][kMaxWarps];
  pdl_trigger();
  pdl_wait();
  constexpr int gw = GROUP / 8;                 // words of a group
  const int words = K / 8, groups = (K + GROUP - 1) / GROUP;
  const int lane = threadIdx.x & 31, warps = TEAMS ? team_warps : blockDim.x >> 5;
  const int team = TEAMS ? (threadIdx.x >> 5) / warps : 0;
  const int teams = TEAMS ? (blockDim.x >> 5) / warps : 1;
  const int warp = (threadIdx.x >> 5) - team * warps;
  const int64_t row0 = (int64_t)blockIdx.x * per_block;         // matrix * N + n
  const int64_t m = row0 / N;
  const int n0 = (int)(row0 - m * N);
  uint8_t* s_zero = s_side + groups * per_block;
  // The kWords words of a lane are of as many groups, the same for the gw >= kWords lanes of a
  // group: lane `sub` of them does the divisions for word `sub`.
  static_assert(gw >= kWords, "a lane per word");
  const int sub = lane & (gw - 1), mine = sub & (kWords - 1);
  Eight<BF16> e[kWords];
  float raw[kWords], lo[kWords];                // a word's group: range, smallest weight (or 0)
  auto fetch = [&](int64_t row, int base) {
    const int i = base + warp * 32 + lane, step = warps * 32;
    const int64_t at = row * words + i;
    if (base + kWords * step <= words) {
#pragma unroll
      for (int r = 0; r < kWords; ++r) e[r].load(W, at + r * step);
    } else {
#pragma unroll
      for (int r = 0; r < kWords; ++r) {
        e[r].zero();
        if (i + r * step < words) e[r].load(W, at + r * step);
      }
    }
  };
  auto ranges = [&]() {
#pragma unroll
    for (int r = 0; r < kWords; ++r) {
      float hi;
      e[r].template range<ZEROS>(hi, lo[r]);
#pragma unroll
      for (int o = 1; o < gw; o <<= 1) {
        hi = max_nan(hi, __shfl_xor_sync(kFull, hi, o));
        if (ZEROS) lo[r] = min_nan(lo[r], __shfl_xor_sync(kFull, lo[r], o));
      }
      raw[r] = ZEROS ? hi - lo[r] : hi;
    }
  };
  const int span = kWords * 32 * warps;         // words of a row that the block holds
  for (int j = team, flip = 0; j < per_block; j += teams, flip ^= 1) {
    const int64_t row = row0 + j;
    float most = 0.f;
    for (int base = 0; base < words; base += span) {
      fetch(row, base);
      ranges();
#pragma unroll
      for (int r = 0; r < kWords; ++r) most = max_nan(most, raw[r]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = max_nan(most, __shfl_xor_sync(kFull, most, o));
    if (warps > 1) {
      float* s = s_max[flip] + team * warps;
      if (lane == 0) s[warp] = most;
      __syncthreads();
      for (int i = 0; i < warps; ++i) most = max_nan(most, s[i]);
    }
    // (division is monotone: the largest range's quotient is the largest quotient)
    constexpr float kSpread = ZEROS ? 15.f : 7.f;
    most = __fdiv_rn(most, kSpread);
    const float rs = most < 0x1p-100f ? 0.f : __fdiv_rn(most, 448.f);
    if (warp == 0 && lane == 0) row_scale[row] = rs;

    for (int base = 0; base < words; base += span) {
      if (words > span) {
        fetch(row, base);
        ranges();
      }
      float my_raw = raw[0], my_lo = lo[0];
#pragma unroll
      for (int r = 1; r < kWords; ++r)
        if (mine == r) {
          my_raw = raw[r];
          my_lo = lo[r];
        }
      const float t = __fdiv_rn(my_raw, kSpread);
      const __nv_fp8_e4m3 sc(rs > 0.f ? __fdiv_rn(t, rs) : 0.f);
      const float step = static_cast<float>(sc) * rs;
      const float my_inv = step > 0.f ? __fdiv_rn(1.f, step) : 0.f;
      const int my_zero = ZEROS ? (int)fminf(fmaxf(rintf(-my_lo * my_inv), 0.f), 15.f) : 8;
      // a scale that is a normal e4m3 (from 2^-6 on, byte 8) is off by at most a 16th, so |w r|
      // is below 7.5 and its rounding needs no clamp; nor where the codes do not matter (r = 0),
      // but an infinity or a NaN has to stay in its nibble
      bool clamp = !(my_raw <= FLT_MAX) || (sc.__x < 8 && my_inv > 0.f);
      const int word0 = base + (mine * warps + warp) * 32 + lane;       // a word of that group
      if (sub < kWords && word0 < words) {
        s_side[word0 / gw * per_block + j] = sc.__x;
        if (ZEROS) s_zero[word0 / gw * per_block + j] = (uint8_t)my_zero;
      }
      clamp = __any_sync(kFull, clamp);
      // words of a block are 8 consecutive k each: k / 8 = 8 b + 4 j + c is word 8 b + 2 c + j
      // (in the row or not with the rest of its block)
      const int to = base + warp * 32 + (lane & ~7) + 2 * (lane & 3) + ((lane >> 2) & 1);
#pragma unroll
      for (int r = 0; r < kWords; ++r) {
        const int from = (lane & ~(gw - 1)) + r;
        const float inv = __shfl_sync(kFull, my_inv, from);
        const int zero = ZEROS ? __shfl_sync(kFull, my_zero, from) : 8;
        // clamped, then rounded: the bounds are whole numbers, so the order does not matter; the
        // sum of the eight rounded ones' bits, 16^p times each, is the word plus a constant
        const float least = ZEROS ? -(float)zero : -8.f, largest = ZEROS ? 15.f - zero : 7.f;
        uint32_t word = 0;
        if (ZEROS || clamp) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float q = fminf(fmaxf(e[r].get(k) * inv, least), largest) + kRound;
            word += __float_as_uint(q) << (4 * (k / 2 + 4 * (k & 1)));
          }
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            word += __float_as_uint(__fadd_rn(__fmul_rn(e[r].get(k), inv), kRound))   // (not fused)
                    << (4 * (k / 2 + 4 * (k & 1)));
        }
        // sum of kRoundBits 16^p (p = 0..7) is kRoundBits * 0x11111111, and each nibble gets zero
        word += (uint32_t)zero * 0x11111111u - kRoundBits * 0x11111111u;
        if (to + r * 32 * warps < words) codes[row * words + to + r * 32 * warps] = word;
      }
    }
  }
  __syncthreads();
  // the rows' scales (zero points), four rows a word
  const int quads = per_block / 4;
  for (int i = threadIdx.x; i < groups * quads; i += blockDim.x) {
    const int kg = i / quads, n = 4 * (i - kg * quads);
    const int64_t to = (m * groups + kg) * N + n0 + n;
    *reinterpret_cast<uint32_t*>(scales + to) =
        *reinterpret_cast<const uint32_t*>(s_side + kg * per_block + n);
    if (ZEROS)
      *reinterpret_cast<uint32_t*>(zeros + to) =
          *reinterpret_cast<const uint32_t*>(s_zero + kg * per_block + n);
  }
}

// A block takes 32 rows by kDqWords words of codes (eight consecutive weights each): their scales
// through shared memory, then a warp a row at a time.
constexpr int kDqRows = 32, kDqWords = 64, kDqThreads = 256;

__device__ __forceinline__ __nv_bfloat162 pair(uint32_t v) {
  return *reinterpret_cast<__nv_bfloat162*>(&v);
}
// (w & 0x000f000f) | 0x43004300 in one step (with two constants the compiler takes two)
__device__ __forceinline__ uint32_t nibble_pair(uint32_t w) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(w), "n"(0x000f000fu), "r"(0x43004300u));
  return r;
}

template <bool BF16>
__global__ void __launch_bounds__(kDqThreads)
dequantize_w4_kernel(const W4Ptrs w, int N, int K, int g, void* __restrict__ out) {
  pdl_trigger();
  pdl_wait();
  __shared__ uint32_t s_scale[16][kDqRows / 4], s_zero[16][kDqRows / 4];
  const int words = K / 8, groups = (K + g - 1) / g;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row0 = (int64_t)blockIdx.x * kDqRows;           // matrix * N + n
  const int64_t m = row0 / N;
  const int n0 = (int)(row0 - m * N), w0 = blockIdx.y * kDqWords;
  const int kg0 = 8 * w0 / g, here = min(kDqWords * 8 / g, groups - kg0);
  if (threadIdx.x < here * (kDqRows / 4)) {
    const int kg = threadIdx.x / (kDqRows / 4), i = threadIdx.x % (kDqRows / 4);
    const int64_t at = (m * groups + kg0 + kg) * N + n0 + 4 * i;
    s_scale[kg][i] = *reinterpret_cast<const uint32_t*>(w.scales + at);
    s_zero[kg][i] = w.zeros ? *reinterpret_cast<const uint32_t*>(w.zeros + at) : 0x08080808u;
  }
  __syncthreads();
  const int b = w0 / 8 + lane / 4, c = lane & 3;  // block, and the words 2 c, 2 c + 1 in it: k from
  // fp32: 32 bytes a lane in one store where the output allows; two of 16 reach every sector twice
  // (8 x 14336 x 4096: 349 against 496 us)
  const bool sectors = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
  const bool live = 8 * b < words;              // 8 c and from 32 + 8 c on
  const int k0 = 64 * b + 8 * c, kg = live ? k0 / g - kg0 : 0, kg1 = live ? (k0 + 32) / g - kg0 : 0;
#pragma unroll
  for (int i = 0; i < kDqRows / (kDqThreads / 32); ++i) {
    const int r = warp + i * (kDqThreads / 32);
    const int64_t row = row0 + r;
    if (!live) continue;
    const uint2 word = __ldcs(reinterpret_cast<const uint2*>(w.codes + row * words + 8 * b) + c);
    const float rs = __ldg(w.row_scale + row);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int shift = 8 * (r & 3);
      const float sf = w4_scale((s_scale[h ? kg1 : kg][r / 4] >> shift) & 0xffu);
      const __nv_bfloat162 sc = __float2bfloat162_rn(sf);
      const __nv_bfloat162 zf =
          pair((0x4300u + ((s_zero[h ? kg1 : kg][r / 4] >> shift) & 0xffu)) * 0x10001u);
      const uint32_t u = h ? word.y : word.x;
      float v[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // a pair as bf16: 128 + code by bits, minus 128 + zero, times the scale, all exact
        const __nv_bfloat162 x = __hmul2(__hsub2(pair(nibble_pair(u >> (4 * e))), zf), sc);
        v[2 * e] = rs * __low2float(x);
        v[2 * e + 1] = rs * __high2float(x);
      }
      const int64_t at = row * K + k0 + 32 * h;
      if (BF16) {
        uint32_t p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __nv_bfloat162 x = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
          p[e] = *reinterpret_cast<const uint32_t*>(&x);
        }
        __stcs(static_cast<uint4*>(out) + at / 8, make_uint4(p[0], p[1], p[2], p[3]));
      } else {
        float* o = static_cast<float*>(out) + at;
        if (sectors) {
          asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(o), "f"(v[0]),
                       "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                       : "memory");
        } else {
          reinterpret_cast<float4*>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
          reinterpret_cast<float4*>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_quantize_w4(int n_matrices, int N, int K, bool bf16, const void* W,
                               const moe_w4_t& o, cudaStream_t s) {
  const int64_t rows = (int64_t)n_matrices * N;
  const int words = K / 8, groups = (K + o.group - 1) / o.group;
  const int each = 32 * kWords;
  int warps = (words + each - 1) / each;
  if (warps > kMaxWarps) warps = kMaxWarps;
  // rows per block: 32 fill a sector of scales; fewer when the blocks would not fill the SMs a
  // few times over, or their scales 48 KB of shared memory (N is a multiple of 64)
  int per = 32;
  const size_t side = (size_t)groups * (o.zeros ? 2 : 1);
  while (per > 4 && (rows / per < (int64_t)num_sms() * 16 || side * per > 40960)) per /= 2;
  const size_t smem = side * per;
  // few rows: those of a block at once instead of one after the other, by as many teams of warps
  // (5632 rows of 1984 fp32 17.0 -> 13.5 us, 4096 of 4096 bf16 17.5 -> 14.3; a kernel of its own,
  // since rows that differ between the warps cost 239 -> 290 us at 114688 rows of 4096)
  int teams = 1;
  while (per == 4 && teams < 4 && 2 * teams * warps <= kMaxWarps) teams *= 2;
  auto go = [&](auto k) {
    if (smem > 40960) {
      cudaError_t e = allow_smem(k, kQuantMaxSmem);
      if (e != cudaSuccess) return e;
    }
    return launch_pdl(k, dim3((unsigned)(rows / per)), dim3(32 * warps * teams), smem, s, W, N, K,
                      per, warps, reinterpret_cast<uint32_t*>(o.codes), o.scales, o.zeros,
                      o.row_scale);
  };
  auto form = [&](auto group, auto many) {
    constexpr int G = decltype(group)::value;
    constexpr bool T = decltype(many)::value;
    if (bf16) return o.zeros ? go(quantize_w4_kernel<true, true, G, T>)
                             : go(quantize_w4_kernel<true, false, G, T>);
    return o.zeros ? go(quantize_w4_kernel<false, true, G, T>)
                   : go(quantize_w4_kernel<false, false, G, T>);
  };
  auto run = [&](auto group) {
    return teams > 1 ? form(group, std::true_type{}) : form(group, std::false_type{});
  };
  if (o.group == 32) return run(std::integral_constant<int, 32>{});
  if (o.group == 64) return run(std::integral_constant<int, 64>{});
  return run(std::integral_constant<int, 128>{});
}

cudaError_t launch_dequantize_w4(int n_matrices, int N, int K, const moe_w4_t& w, bool bf16,
                                 void* out, cudaStream_t s) {
  const int64_t rows = (int64_t)n_matrices * N;
  const dim3 grid((unsigned)(rows / kDqRows), (unsigned)((K / 8 + kDqWords - 1) / kDqWords));
  const W4Ptrs p{reinterpret_cast<const uint32_t*>(w.codes), w.scales, w.zeros, w.row_scale};
  auto k = bf16 ? dequantize_w4_kernel<true> : dequantize_w4_kernel<false>;
  return launch_pdl(k, grid, dim3(kDqThreads), 0, s, p, N, K, w.group, out);
}

}  // namespace moe
