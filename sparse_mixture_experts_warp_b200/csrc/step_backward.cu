// Gradients of the dispatch and of the weighted merge as steps of their own, for layers whose
// experts are the caller's (moe_permute_backward, moe_combine_backward).
//
// "从 Dense FFN 到 MoE：用一个 Tiny Transformer 理解 Router、Top-K 与负载均衡" (f3dlife), sections 5, 6
// and 9; "Top-k 路由（Top-k Routing）" (compassingai), Combine box and "門控網路的梯度流" (the gate
// scores of the selected experts carry the gradient, unselected experts none).
//   merge     out[t] = sum_j g[t,j] y[inv[t,j]]
//             dy[inv[t,j]] = g[t,j] dout[t],   dg[t,j] = <dout[t], y[inv[t,j]]>  (0 at inv = -1)
//   dispatch  x_perm[inv[t,j]] = x[t]
//             dx[t] = add[t] + sum over j with inv[t,j] >= 0 of dx_perm[inv[t,j]], in slot order
// Both walk a token's assignments through the inverse permutation, as the combine does: every
// row belongs to one (token, slot), so nothing is summed by atomics and results are
// deterministic.  All sums are fp32; each output is rounded once.
//
// Both only stream memory (a few operations a byte).  The merge's gradient keeps a token's dout
// in registers (4 vectors of 16 bytes a lane, as many warps a token as its row needs) and reads
// it once for all of the token's experts: the bytes are dout + y + dy.  4096 tokens top-2 of D =
// 4096, bf16: 29.7 us, 88% of the copy rate (33 with two rows of y under way at a time, 40 with 2
// vectors a lane, 29.7 with 8); 8190 tokens under expert choice, 64 x 256 rows of D = 2048: 35.2 us,
// 77% (41, 48 and 37).  The dispatch's gradient, 4096 tokens top-8 of D = 7168, a quarter of the rows
// dropped: 81 us, 90% (98 with 2 vectors a lane, 205 with 8).
#include "common.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kVec = 4;                       // 16-byte vectors of a row that a lane holds
constexpr int kSpan = 32 * kVec;              // vectors of a row that a warp holds
constexpr int kMaxSlots = 256;                // assignments of a token (k <= 32, E <= 256)
constexpr unsigned kFull = 0xffffffffu;

template <bool BF16> struct Vec;
template <> struct Vec<true> {
  static constexpr int N = 8;
  __device__ __forceinline__ static void widen(const uint4 u, float* a) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[2 * i] = __uint_as_float(w[i] << 16);
      a[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ static uint4 narrow(const float* a) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(a[2 * i], a[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Vec<false> {
  static constexpr int N = 4;
  __device__ __forceinline__ static void widen(const uint4 u, float* a) {
    a[0] = __uint_as_float(u.x); a[1] = __uint_as_float(u.y);
    a[2] = __uint_as_float(u.z); a[3] = __uint_as_float(u.w);
  }
  __device__ __forceinline__ static uint4 narrow(const float* a) {
    return make_uint4(__float_as_uint(a[0]), __float_as_uint(a[1]), __float_as_uint(a[2]),
                      __float_as_uint(a[3]));
  }
};

// y and dy may be the same rows (a lane reads its vectors before it writes them), so neither is
// __restrict__.  W warps take one token; a block of 8 warps 8 / W tokens.  Rows longer than
// W * kSpan vectors go in passes, whose dots add up in shared memory (each cell has one owner: no atomics).
template <bool BF16>
__global__ void __launch_bounds__(kWarps * 32)
combine_backward_kernel(const uint4* __restrict__ dout, const uint4* y,
                        const int32_t* __restrict__ inv, const float* __restrict__ gates, int T,
                        int K, int nvec, int W, uint4* dy, float* __restrict__ dgates) {
  pdl_trigger();
  pdl_wait();
  using V = Vec<BF16>;
  __shared__ float s_dot[kWarps][kMaxSlots];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = warp % W;
  const int64_t t = (int64_t)blockIdx.x * (kWarps / W) + warp / W;
  const bool live = t < T;
  if (live) {
    const int32_t* rows = inv + t * K;
    const float* g = gates + t * K;
    const int passes = (nvec + W * kSpan - 1) / (W * kSpan);
    for (int p = 0; p < passes; ++p) {
      const int v0 = (p * W + part) * kSpan + lane;
      uint4 d[kVec];
#pragma unroll
      for (int c = 0; c < kVec; ++c)
        d[c] = v0 + 32 * c < nvec ? __ldcs(dout + t * nvec + v0 + 32 * c)
                                  : make_uint4(0u, 0u, 0u, 0u);
      for (int j0 = 0; j0 < K; j0 += 32) {
        const int r_l = j0 + lane < K ? rows[j0 + lane] : -1;
        const float g_l = r_l >= 0 ? g[j0 + lane] : 0.f;
        unsigned left = __ballot_sync(kFull, r_l >= 0);
        while (left) {
          const int j = __ffs(left) - 1;
          left &= left - 1;
          const int64_t row = __shfl_sync(kFull, r_l, j);
          const float gj = __shfl_sync(kFull, g_l, j);
          uint4 u[kVec];
#pragma unroll
          for (int c = 0; c < kVec; ++c)
            u[c] = dgates && v0 + 32 * c < nvec ? __ldcs(y + row * nvec + v0 + 32 * c)
                                                : make_uint4(0u, 0u, 0u, 0u);
          float dot = 0.f;
#pragma unroll
          for (int c = 0; c < kVec; ++c) {
            float a[V::N], b[V::N];
            V::widen(d[c], a);
            V::widen(u[c], b);
#pragma unroll
            for (int i = 0; i < V::N; ++i) dot = fmaf(a[i], b[i], dot);
            if (dy && v0 + 32 * c < nvec) {
#pragma unroll
              for (int i = 0; i < V::N; ++i) a[i] *= gj;
              __stcs(dy + row * nvec + v0 + 32 * c, V::narrow(a));
            }
          }
          if (dgates) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
            if (lane == 0) s_dot[warp][j0 + j] = p ? s_dot[warp][j0 + j] + dot : dot;
          }
        }
      }
    }
  }
  if (!dgates) return;
  __syncthreads();
  if (live) {
    const int first = warp - part;
    for (int j = part * 32 + lane; j < K; j += W * 32) {
      float sum = 0.f;
      if (inv[t * K + j] >= 0)
        for (int w = 0; w < W; ++w) sum += s_dot[first + w][j];
      dgates[t * K + j] = sum;
    }
  }
}

// One warp per (token, kSpan vectors of its row).  add and dx may be the same rows.
template <bool BF16>
__global__ void __launch_bounds__(kWarps * 32)
permute_backward_kernel(const uint4* __restrict__ dxp, const int32_t* __restrict__ inv,
                        const uint4* add, int T, int K, int nvec, int spans, uint4* dx) {
  pdl_trigger();
  pdl_wait();
  using V = Vec<BF16>;
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t t = w / spans;
  if (t >= T) return;
  const int v0 = (int)(w - t * spans) * kSpan + lane;
  float a[kVec][V::N];
#pragma unroll
  for (int c = 0; c < kVec; ++c) {
    const uint4 u = add && v0 + 32 * c < nvec ? __ldcs(add + t * nvec + v0 + 32 * c)
                                              : make_uint4(0u, 0u, 0u, 0u);
    V::widen(u, a[c]);
  }
  for (int j0 = 0; j0 < K; j0 += 32) {
    const int r_l = j0 + lane < K ? inv[t * K + j0 + lane] : -1;
    unsigned left = __ballot_sync(kFull, r_l >= 0);
    while (left) {
      const int j = __ffs(left) - 1;
      left &= left - 1;
      const int64_t row = __shfl_sync(kFull, r_l, j);
      uint4 u[kVec];
#pragma unroll
      for (int c = 0; c < kVec; ++c)
        u[c] = v0 + 32 * c < nvec ? __ldcs(dxp + row * nvec + v0 + 32 * c)
                                  : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int c = 0; c < kVec; ++c) {
        float b[V::N];
        V::widen(u[c], b);
#pragma unroll
        for (int i = 0; i < V::N; ++i) a[c][i] += b[i];
      }
    }
  }
#pragma unroll
  for (int c = 0; c < kVec; ++c)
    if (v0 + 32 * c < nvec) dx[t * nvec + v0 + 32 * c] = V::narrow(a[c]);
}

int slots_of(const moe_desc_t& d) { return d.select == MOE_EXPERT_CHOICE ? d.E : d.k; }
int vectors_of(const moe_desc_t& d) { return d.D / (d.dtype == MOE_BF16 ? 8 : 4); }

}  // namespace

cudaError_t launch_combine_backward(const moe_desc_t& d, const void* dout, const void* y,
                                    const int32_t* inv, const float* gates, void* dy,
                                    float* dgates, cudaStream_t s) {
  const int nvec = vectors_of(d);
  int W = 1;
  while (W < kWarps && W * kSpan < nvec) W *= 2;
  const int per = kWarps / W;
  const dim3 grid((unsigned)((d.T + per - 1) / per)), block(kWarps * 32);
  auto k = d.dtype == MOE_BF16 ? combine_backward_kernel<true> : combine_backward_kernel<false>;
  return launch_pdl(k, grid, block, 0, s, static_cast<const uint4*>(dout),
                    static_cast<const uint4*>(y), inv, gates, d.T, slots_of(d), nvec, W,
                    static_cast<uint4*>(dy), dgates);
}

cudaError_t launch_permute_backward(const moe_desc_t& d, const void* dx_perm,
                                    const int32_t* inv, const void* add, void* dx,
                                    cudaStream_t s) {
  const int nvec = vectors_of(d);
  const int spans = (nvec + kSpan - 1) / kSpan;
  const int64_t warps = (int64_t)d.T * spans;
  const dim3 grid((unsigned)((warps + kWarps - 1) / kWarps)), block(kWarps * 32);
  auto k = d.dtype == MOE_BF16 ? permute_backward_kernel<true> : permute_backward_kernel<false>;
  return launch_pdl(k, grid, block, 0, s, static_cast<const uint4*>(dx_perm), inv,
                    static_cast<const uint4*>(add), d.T, slots_of(d), nvec, spans,
                    static_cast<uint4*>(dx));
}

}  // namespace moe
