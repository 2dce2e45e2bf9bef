// Grouped product on 4-bit weights (w4.cuh) for few rows per group: weight streaming on
// mma.sync.
//
// "别只比较 Top-k" (ailearn moe-comparison), the expert-work account: in a small decode batch each
// expert's products have a few rows and stream the weights; "从 Dense FFN 到 MoE：用一个 Tiny
// Transformer 理解 Router、Top-K 与负载均衡" (f3dlife), section 3.
//
// out[r, n] = epi(row_scale[n] * sum_groups scale * sum_k (code - zero) a[r, k]).  The time is the
// codes' bytes, and next to them the integer work of unpacking: 3 shifts and 4 mask-and-or steps
// per 8 codes (half rate on sm_100a).  So the weights go from shared memory straight into mma
// fragments as the whole numbers code - zero (exact in bf16), and the scale multiplies the fp32
// sum of its group of k (one step per 32..128 k instead of one per weight).
//
// A CTA of 16 warps takes a tile of RT * 16 weight rows (SwiGLU: RT * 8 features, 8 rows of
// W_gate above the same 8 of W_up in one m16n8k16 fragment) by up to P <= 8 tokens of a group:
// RT warps side by side, WK = 16 / RT along K.  Every warp streams its own 16 rows x 256 k stages
// through a private ring (TMA for the codes, 8-byte cp.async for scales and zero points), so
// nothing but the sum over the WK warps, once a tile through shared memory, waits for another
// warp, and the ring runs on into the next tile meanwhile.  CTAs own contiguous ranges of tiles
// (group by group, token tiles, then weight rows), so the P token rows are copied to shared
// memory about once per group.
#include <cuda.h>

#include "common.cuh"
#include "mbar.cuh"
#include "tc_ops.cuh"
#include "w4.cuh"
#include "w4_wait.cuh"

namespace moe {
namespace {

constexpr int ST_WARPS = 16;
constexpr int ST_THREADS = 32 * ST_WARPS;
constexpr int ST_K = 256;                       // k of a stage
constexpr int ST_STAGES = 3;
constexpr int ST_CODES = 16 * ST_K / 2;         // bytes of codes of a stage: 16 rows x 128
constexpr int ST_SIDE = 128;                    // scales (or zero points): up to 8 groups x 16 rows
constexpr int ST_TOK = 8;
constexpr int ST_PART = 16 * ST_TOK;            // fp32 partial sums of a warp
constexpr int ST_XPAD = 64;                     // bytes: rows of x start 64 bytes apart mod 128
constexpr size_t ST_FIXED = 1024 + (size_t)ST_WARPS * ST_STAGES * (ST_CODES + 2 * ST_SIDE + 8) +
                            2 * ST_WARPS * ST_PART * 4 + 16;
constexpr size_t ST_SMEM = 227 * 1024;

struct StreamParams {
  const __nv_bfloat16* a;                       // [rows, K]
  const int32_t* offsets;                       // [G + 1]
  W4Ptrs gate, w;                               // gate.codes null unless SwiGLU
  __nv_bfloat16* out;                           // [rows, N]
  int* err;
  int64_t rows;
  int G, N, K, act;
  int P;                                        // tokens per tile
  int RT, WK;
  int fault;                                    // test hook: the first stage of CTA 0 never comes
};

// A walk over tiles: group by group, token tile by token tile, feature tiles innermost.
struct StreamTile {
  int g, n0, row0, ntok;                        // n0: first feature
  __device__ __forceinline__ void start(int t, const int* grp_off, const int* tile_pre, int nt,
                                        int P, int feats) {
    g = 0;
    while (t >= tile_pre[g + 1]) ++g;
    const int local = t - tile_pre[g], j = local / nt;
    n0 = (local - j * nt) * feats;
    row0 = grp_off[g] + j * P;
    ntok = min(P, grp_off[g + 1] - row0);
  }
  // to the next tile; the caller has checked that there is one
  __device__ __forceinline__ void next(const int* grp_off, int N, int P, int feats) {
    n0 += feats;
    if (n0 < N) return;
    n0 = 0;
    row0 += P;
    while (row0 >= grp_off[g + 1]) row0 = grp_off[++g];
    ntok = min(P, grp_off[g + 1] - row0);
  }
};

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
// Arrives on bar once this thread's cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Four pairs code - zero of a word (z2 = 128 + zero twice).
__device__ __forceinline__ void unpack_word(uint32_t w, __nv_bfloat162 z2, uint32_t (&r)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t p = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&p), z2);
    r[i] = *reinterpret_cast<const uint32_t*>(&d);
  }
}
__device__ __forceinline__ __nv_bfloat162 zero2(uint32_t z) {
  uint32_t v = (0x4300u + z) * 0x10001u;
  return *reinterpret_cast<__nv_bfloat162*>(&v);
}

template <bool GLU, bool ZEROS, int GROUP>
__global__ void __launch_bounds__(ST_THREADS, 1)
w4_stream_kernel(const __grid_constant__ CUtensorMap tmC0,
                 const __grid_constant__ CUtensorMap tmC1, const StreamParams p) {
  constexpr int GS = ST_K / GROUP;              // scale groups of a stage
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* codes = smem + warp * (ST_STAGES * ST_CODES);
  uint8_t* side = smem + ST_WARPS * ST_STAGES * ST_CODES + warp * (ST_STAGES * 2 * ST_SIDE);
  float* part = reinterpret_cast<float*>(smem + ST_WARPS * ST_STAGES * (ST_CODES + 2 * ST_SIDE));
  uint64_t* bars = reinterpret_cast<uint64_t*>(part + 2 * ST_WARPS * ST_PART);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + ST_WARPS * ST_STAGES);
  uint8_t* xs = reinterpret_cast<uint8_t*>(bars + ST_WARPS * ST_STAGES) + 16;
  const int xpitch = 2 * p.K + ST_XPAD;
  int* grp_off = reinterpret_cast<int*>(xs + p.P * xpitch);       // [G + 1]
  int* tile_pre = grp_off + (p.G + 1);                            // [G + 1]
  const uint32_t full = smem_u32(bars + warp * ST_STAGES);
  const BarWait wait{abort_flag, p.err};

  const int feats = (GLU ? 8 : 16) * p.RT;
  const int nt = (p.N + feats - 1) / feats;
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST_WARPS * ST_STAGES; ++i) mbar_init(bars + i, 33);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  pdl_trigger();
  pdl_wait();
  if (warp == 1) {
    // group row starts and the tile prefix
    int carry = 0;
    if (lane == 0) {
      grp_off[0] = p.offsets[0];
      tile_pre[0] = 0;
    }
    for (int g0 = 0; g0 < p.G; g0 += 32) {
      const int g = g0 + lane;
      int tiles = 0;
      if (g < p.G) {
        const int lo = p.offsets[g], hi = p.offsets[g + 1];
        const int m = hi > lo ? hi - lo : 0;
        tiles = ((m + p.P - 1) / p.P) * nt;
        grp_off[g + 1] = hi;
      }
      int inc = tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kFullWarp, inc, o);
        if (lane >= o) inc += v;
      }
      if (g < p.G) tile_pre[g + 1] = carry + inc;
      carry += __shfl_sync(kFullWarp, inc, 31);
    }
  }
  __syncthreads();
  const int total = tile_pre[p.G];
  const int t_lo = (int)((int64_t)total * blockIdx.x / gridDim.x);
  const int t_hi = (int)((int64_t)total * (blockIdx.x + 1) / gridDim.x);
  const int nst = (p.K + ST_K - 1) / ST_K;
  const int groups = (p.K + GROUP - 1) / GROUP;
  const int wk = warp % p.WK, rt = warp / p.WK;
  const bool leader = elect_one();
  const int q = lane >> 2, c = lane & 3;        // fragment row / token, and column pair
  const int prow = ((q & 3) << 1) | (q >> 2);   // weight row of fragment row q: reads of the
                                                // swizzled rows are then free of bank conflicts
  // ---- this warp's stream: stages wk, wk + WK, .. of every tile ----
  StreamTile pl{};                              // tile and stage of the next request
  int pt = wk < nst ? t_lo : t_hi, ps = wk, slot = 0;
  if (pt < t_hi) pl.start(pt, grp_off, tile_pre, nt, p.P, feats);
  uint32_t issued = 0, par = 0;                 // per slot: under way; parity of its phase
  bool alive = true;
  // lane: 8 rows of a scale group, first or second half of the fragment's rows
  const int kg = lane >> 1, half = lane & 1;
  const uint8_t* scales = GLU && half == 0 ? p.gate.scales : p.w.scales;
  const uint8_t* zeros = GLU && half == 0 ? p.gate.zeros : p.w.zeros;
  const uint32_t side_dst = smem_u32(side) + 16 * kg + 8 * half;
  auto request = [&]() {                        // into `slot`, which the warp has read
    if (pt >= t_hi) return;
    const int n0 = pl.n0 + rt * (GLU ? 8 : 16);
    const uint32_t bar = full + 8 * slot;
    const bool load = !(p.fault == 1 && blockIdx.x == 0 && warp == 0 && pt == t_lo && ps == wk);
    if (leader) {
      bar_expect(bar, ST_CODES);
      if (load) {
        const uint32_t dst = smem_u32(codes + slot * ST_CODES);
        const int x = ps * (ST_K / 2), y = pl.g * p.N + n0;
        if (GLU) {
          bar_load(dst, &tmC1, bar, x, y);
          bar_load(dst + ST_CODES / 2, &tmC0, bar, x, y);
        } else {
          bar_load(dst, &tmC0, bar, x, y);
        }
      }
    }
    const int at = ps * GS + kg, n = GLU ? n0 : n0 + 8 * half;
    if (kg < GS && at < groups && n < p.N) {
      const int64_t src = (int64_t)(pl.g * groups + at) * p.N + n;
      cp_async8(side_dst + slot * 2 * ST_SIDE, scales + src);
      if (ZEROS) cp_async8(side_dst + slot * 2 * ST_SIDE + ST_SIDE, zeros + src);
    }
    cp_async_arrive(bar);
    if (load) issued |= 1u << slot;
    ps += p.WK;
    if (ps >= nst) {
      ps = wk;
      if (++pt < t_hi) pl.next(grp_off, p.N, p.P, feats);
    }
  };
  for (slot = 0; slot < ST_STAGES; ++slot) request();
  slot = 0;

  StreamTile tl{};
  if (t_lo < t_hi) tl.start(t_lo, grp_off, tile_pre, nt, p.P, feats);
  int x_row = -1, buf = 0;
  const int lane_at = ((c >> 1) ^ prow) << 4;   // 16-byte piece of block 0, swizzled
  for (int t = t_lo; t < t_hi; ++t, buf ^= 1) {
    const bool rows_ok = tl.row0 >= 0 && (int64_t)tl.row0 + tl.ntok <= p.rows;
    if (tl.row0 != x_row) {
      // token rows of the new group or token tile (every warp has read the old ones: it has
      // arrived at the last tile's barrier)
      if (!rows_ok && threadIdx.x == 0) atomicCAS(p.err, 0, DEVERR_BOUNDS);
      const int vec = p.K / 8;
      for (int r = 0; r < tl.ntok; ++r) {
        const uint4* src =
            reinterpret_cast<const uint4*>(p.a + ((int64_t)tl.row0 + r) * p.K);
        for (int v = threadIdx.x; v < vec; v += ST_THREADS)
          *reinterpret_cast<uint4*>(xs + r * xpitch + 16 * v) =
              rows_ok ? __ldg(src + v) : make_uint4(0u, 0u, 0u, 0u);
      }
      __syncthreads();
      x_row = tl.row0;
    }
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    // lanes without a token repeat the last one: their columns of the product are not used
    const uint8_t* xrow = xs + min(q, tl.ntok - 1) * xpitch + 16 * c;
    for (int s = wk; s < nst; s += p.WK) {
      if (alive) alive = wait(full + 8 * slot, (par >> slot) & 1u, DEVERR_TIMEOUT_TMA);
      if (alive) {
        const uint8_t* st = codes + slot * ST_CODES + prow * 128 + 8 * (c & 1);
        const uint8_t* sd = side + slot * 2 * ST_SIDE + prow;
        const uint8_t* xp = xrow + s * (2 * ST_K);
        const int here = (p.K - s * ST_K) / W4_BLOCK;       // 64-element blocks of the stage
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        __nv_bfloat162 z0 = zero2(8u), z1 = zero2(8u);
        auto block = [&](int b, bool last) {
          const int at = lane_at ^ (b << 5);
          const uint2 wa = *reinterpret_cast<const uint2*>(st + at);
          const uint2 wb = *reinterpret_cast<const uint2*>(st + ST_CODES / 2 + at);
#pragma unroll
          for (int j = 0; j < 2; ++j) {         // 32-element halves
            const int k = 64 * b + 32 * j;
            if (ZEROS && k % GROUP == 0) {
              z0 = zero2(sd[ST_SIDE + 16 * (k / GROUP)]);
              z1 = zero2(sd[ST_SIDE + 16 * (k / GROUP) + 8]);
            }
            const uint4 x = *reinterpret_cast<const uint4*>(xp + 2 * k);
            uint32_t ra[4], rb[4];
            unpack_word(j ? wa.y : wa.x, z0, ra);
            unpack_word(j ? wb.y : wb.x, z1, rb);
            const uint32_t a0[4] = {ra[0], rb[0], ra[1], rb[1]};
            const uint32_t a1[4] = {ra[2], rb[2], ra[3], rb[3]};
            mma_16816(sum, a0, x.x, x.y);
            mma_16816(sum, a1, x.z, x.w);
            if ((k + 32) % GROUP == 0 || (j == 1 && last)) {
              const float s0 = w4_scale(sd[16 * (k / GROUP)]);
              const float s1 = w4_scale(sd[16 * (k / GROUP) + 8]);
              acc[0] = fmaf(s0, sum[0], acc[0]);
              acc[1] = fmaf(s0, sum[1], acc[1]);
              acc[2] = fmaf(s1, sum[2], acc[2]);
              acc[3] = fmaf(s1, sum[3], acc[3]);
              sum[0] = sum[1] = sum[2] = sum[3] = 0.f;
            }
          }
        };
        if (here >= 4) {
#pragma unroll
          for (int b = 0; b < 4; ++b) block(b, false);
        } else {
#pragma unroll 1
          for (int b = 0; b < here; ++b) block(b, b == here - 1);
        }
        __syncwarp();
        par ^= 1u << slot;
        issued &= ~(1u << slot);
        request();
      }
      if (++slot == ST_STAGES) slot = 0;
    }
    // sum over the WK warps of a row tile
    float* mypart = part + (buf * ST_WARPS + warp) * ST_PART + prow * ST_TOK + 2 * c;
    *reinterpret_cast<float2*>(mypart) = make_float2(acc[0], acc[1]);
    *reinterpret_cast<float2*>(mypart + 8 * ST_TOK) = make_float2(acc[2], acc[3]);
    __syncthreads();
    if (rows_ok) {
      constexpr int per = GLU ? 8 : 16;
      for (int i = threadIdx.x; i < tl.ntok * feats; i += ST_THREADS) {
        const int tok = i / feats, f = i - tok * feats;
        const float* src =
            part + (buf * ST_WARPS + (f / per) * p.WK) * ST_PART + (f % per) * ST_TOK + tok;
        const int n = tl.n0 + f;
        if (n >= p.N) continue;
        float v = 0.f, u = 0.f;
        for (int w = 0; w < p.WK; ++w) {
          v += src[w * ST_PART];
          if (GLU) u += src[w * ST_PART + 8 * ST_TOK];
        }
        const int64_t nr = (int64_t)tl.g * p.N + n;
        if (GLU) {
          v *= __ldg(p.gate.row_scale + nr);
          u *= __ldg(p.w.row_scale + nr);
          v = __fdividef(v, 1.0f + __expf(-v)) * u;
        } else {
          v *= __ldg(p.w.row_scale + nr);
          if (p.act == MOE_ACT_RELU) v = v < 0.f ? 0.f : v;          // a NaN stays one
          if (p.act == MOE_ACT_GELU) v = 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
        }
        p.out[((int64_t)tl.row0 + tok) * p.N + n] = __float2bfloat16_rn(v);
      }
    }
    if (t + 1 < t_hi) tl.next(grp_off, p.N, p.P, feats);
  }
  // copies in flight land before the CTA exits (only after a wait that gave up)
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (!alive)
    for (int s = 0; s < ST_STAGES; ++s)
      if (issued & (1u << s))
        wait.drain(full + 8 * s, (par >> s) & 1u, DEVERR_TIMEOUT_TMA, kDrainNs);
}

}  // namespace

// Tokens per tile that the shared memory holds next to the rings; 0: K is too long.
int w4_stream_tokens(int K, int G) {
  const size_t table = (size_t)2 * (G + 1) * sizeof(int);
  if (ST_FIXED + table >= ST_SMEM) return 0;
  const size_t n = (ST_SMEM - ST_FIXED - table) / (2 * (size_t)K + ST_XPAD);
  return n < ST_TOK ? (int)n : ST_TOK;
}

cudaError_t launch_w4_stream(int act, const void* a, int64_t a_rows, int K, const moe_w4_t* gate,
                             const moe_w4_t* w, int G, int N, const int32_t* offsets, void* out,
                             cudaStream_t s) {
  if (a_rows <= 0 || G <= 0) return cudaSuccess;
  const bool glu = gate != nullptr;
  StreamParams p{};
  p.P = w4_stream_tokens(K, G);
  if (p.P < 1 || (int64_t)G * N > INT32_MAX) return cudaErrorInvalidValue;
  if (a_rows < p.P) p.P = (int)a_rows;
  alignas(64) CUtensorMap c0, c1;
  if (!make_map_u8(&c0, w->codes, (uint64_t)G * N, (uint64_t)K / 2, glu ? 8 : 16, 128, true) ||
      !make_map_u8(&c1, glu ? gate->codes : w->codes, (uint64_t)G * N, (uint64_t)K / 2,
                   glu ? 8 : 16, 128, true))
    return cudaErrorInvalidValue;
  auto ptrs = [](const moe_w4_t* q) {
    return W4Ptrs{reinterpret_cast<const uint32_t*>(q->codes), q->scales, q->zeros, q->row_scale};
  };
  p.a = static_cast<const __nv_bfloat16*>(a);
  p.offsets = offsets;
  p.w = ptrs(w);
  if (glu) p.gate = ptrs(gate);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.err = device_error_word();
  p.rows = a_rows;
  p.G = G;
  p.N = N;
  p.K = K;
  p.act = act;
  p.fault = gemm_fault();
  // as many warps along K as divide its stages well (idle warps in at most an eighth of the
  // rounds) and have two of them or more a tile, the rest side by side
  const int nst = (K + ST_K - 1) / ST_K;
  p.WK = ST_WARPS;
  while (p.WK > 1 && (2 * p.WK > nst || 8 * nst < 7 * p.WK * ((nst + p.WK - 1) / p.WK)))
    p.WK /= 2;
  p.RT = ST_WARPS / p.WK;
  const int feats = (glu ? 8 : 16) * p.RT;
  const int64_t tiles = ((a_rows + p.P - 1) / p.P + G) * (int64_t)((N + feats - 1) / feats);
  const int sms = num_sms();
  const int grid = (int)(tiles < sms ? tiles : sms);
  const size_t smem = ST_FIXED + (size_t)p.P * (2 * (size_t)K + ST_XPAD) +
                      (size_t)2 * (G + 1) * sizeof(int);
  auto run = [&](auto kern) {
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(grid), dim3(ST_THREADS), smem, s, c0, c1, p);
  };
#define MOE_W4_STREAM(GROUP)                                                               \
  if (w->group == GROUP)                                                                   \
    return glu ? (w->zeros ? run(w4_stream_kernel<true, true, GROUP>)                      \
                           : run(w4_stream_kernel<true, false, GROUP>))                    \
               : (w->zeros ? run(w4_stream_kernel<false, true, GROUP>)                     \
                           : run(w4_stream_kernel<false, false, GROUP>))
  MOE_W4_STREAM(32);
  MOE_W4_STREAM(64);
  MOE_W4_STREAM(128);
#undef MOE_W4_STREAM
  return cudaErrorInvalidValue;
}

}  // namespace moe
