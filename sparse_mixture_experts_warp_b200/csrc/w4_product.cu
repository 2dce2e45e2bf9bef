// Expert products on 4-bit weights (w4.cuh), the simple form: one warp per output column and up
// to 8 rows of a group, its lanes along K.
//
// "从 Dense FFN 到 MoE：用一个 Tiny Transformer 理解 Router、Top-K 与负载均衡" (f3dlife), section 3
// (SwiGLU expert: hidden = SiLU(x W_gate) * (x W_up), output = hidden W_down).
#include "common.cuh"
#include "w4.cuh"

namespace moe {
namespace {

constexpr int kRows = 8;
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float dot_w4(const W4Ptrs& w, int64_t grow, int64_t srow, int N, int K,
                                        int g, int n, const __nv_bfloat16* a, int nr, int lane,
                                        float (&acc)[kRows]) {
  const int words = K / 8;
  for (int r = 0; r < kRows; ++r) acc[r] = 0.f;
  for (int i = lane; i < words; i += 32) {
    const int k = (i >> 3) * W4_BLOCK + w4_word_k(i & 7);
    const uint32_t word = w.codes[(grow + n) * words + i];
    const int64_t at = (srow + k / g) * N + n;
    const float sc = w4_scale(w.scales[at]);
    const float z = w.zeros ? (float)w.zeros[at] : 8.f;
    for (int e = 0; e < 8; ++e) {
      const float v = sc * ((float)((word >> (4 * (e / 2 + 4 * (e & 1)))) & 15u) - z);
      for (int r = 0; r < nr; ++r)
        acc[r] = fmaf(v, __bfloat162float(a[(int64_t)r * K + k + e]), acc[r]);
    }
  }
  for (int r = 0; r < kRows; ++r)
    for (int o = 16; o > 0; o >>= 1) acc[r] += __shfl_xor_sync(kFull, acc[r], o);
  return w.row_scale[grow + n];
}

__global__ void __launch_bounds__(256)
w4_simple_kernel(const __nv_bfloat16* __restrict__ a, const int32_t* __restrict__ offsets,
                 const W4Ptrs wg, const W4Ptrs wu, int G, int N, int K, int g, int act,
                 int64_t a_rows, __nv_bfloat16* __restrict__ out) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int n = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (n >= N) return;
  // row tile blockIdx.y + i * gridDim.y of all groups' tiles
  int tile = 0;
  for (int e = 0; e < G; ++e) {
    const int lo = offsets[e], hi = offsets[e + 1];
    for (int r0 = lo; r0 < hi; r0 += kRows, ++tile) {
      if (tile % gridDim.y != blockIdx.y) continue;
      const int nr = hi - r0 < kRows ? hi - r0 : kRows;
      if (r0 < 0 || (int64_t)r0 + nr > a_rows) continue;
      const int64_t grow = (int64_t)e * N, srow = (int64_t)e * ((K + g - 1) / g);
      float u[kRows], gt[kRows];
      const float ru = dot_w4(wu, grow, srow, N, K, g, n, a + (int64_t)r0 * K, nr, lane, u);
      float rg = 0.f;
      if (wg.codes) rg = dot_w4(wg, grow, srow, N, K, g, n, a + (int64_t)r0 * K, nr, lane, gt);
      if (lane == 0)
        for (int r = 0; r < nr; ++r) {
          float v = ru * u[r];
          if (wg.codes) {
            const float x = rg * gt[r];
            v *= x / (1.f + expf(-x));
          } else if (act == MOE_ACT_RELU) {
            v = v < 0.f ? 0.f : v;               // a NaN stays one
          } else if (act == MOE_ACT_GELU) {
            v = 0.5f * v * (1.f + erff(v * 0.70710678118654752f));
          }
          out[(int64_t)(r0 + r) * N + n] = __float2bfloat16_rn(v);
        }
    }
  }
}

W4Ptrs ptrs(const moe_w4_t* w) {
  if (!w) return W4Ptrs{nullptr, nullptr, nullptr, nullptr};
  return W4Ptrs{reinterpret_cast<const uint32_t*>(w->codes), w->scales, w->zeros, w->row_scale};
}

}  // namespace

cudaError_t launch_w4_product(int act, const void* a, int64_t a_rows, int K, const moe_w4_t* gate,
                              const moe_w4_t* w, int G, int N, const int32_t* offsets, void* out,
                              cudaStream_t s) {
  if (a_rows <= 0) return cudaSuccess;
  int64_t tiles = a_rows / kRows + G;
  if (tiles > 256) tiles = 256;
  const dim3 grid((unsigned)((N + 7) / 8), (unsigned)tiles), block(256);
  return launch_pdl(w4_simple_kernel, grid, block, 0, s, static_cast<const __nv_bfloat16*>(a),
                    offsets, ptrs(gate), ptrs(w), G, N, K, w->group, act, a_rows,
                    static_cast<__nv_bfloat16*>(out));
}

}  // namespace moe
