// Grouped product on 4-bit weights (w4.cuh) with tcgen05: the weights are dequantised into
// tensor memory and feed the MMA from there.
//
// "从 Dense FFN 到 MoE：用一个 Tiny Transformer 理解 Router、Top-K 与负载均衡" (f3dlife), section 3
// (SwiGLU expert: hidden = SiLU(x W_gate) * (x W_up), output = hidden W_down); "别只比较 Top-k"
// (ailearn moe-comparison), the Execute step.
//
// out[r, n] = epi(row_scale[n] * sum_k scale[k / g, n] (code[n, k] - zero[k / g, n]) a[r, k]) for
// the rows r of group g.  The weights are the MMA's M side and the tokens its N side:
//   D[n, t] = sum_k w[n, k] a[row0 + t, k]       (TMEM lane = weight row, column = token)
// so one thread owns one weight row: its codes, its group scales, its row factor, and its lane of
// the A operand.  scale * (code - zero) is a bf16 exactly, so nothing is rounded on the way in.
// A tile is 128 weight rows by up to NT tokens of one group (a group's tiles alike); N of the MMA
// is the token count rounded up to 16.  SwiGLU: lanes 0..15 of every 32 hold 16 rows of W_gate,
// lanes 16..31 the same rows of W_up, so gate and up of a feature are one warp shuffle apart.
//
// Roles (one persistent CTA per SM; tiles group by group, weight tile by weight tile, token tiles
// innermost, so that the CTAs that run together share weight tiles through L2):
//   warp 0       TMA producer of the weights: 256 k of codes (128 rows x 128 bytes, 128-byte
//                swizzle: a thread's 16-byte reads of its row are free of bank conflicts), and
//                their scales and zero points, per stage;
//   warp 1       TMA producer of the token rows: 128 k (NT = 192) or 256 k per stage, in
//                boxes of 64 k (128-byte swizzle) by the whole tile's rows, or by 64 of them where
//                fewer do (up, Mixtral width, 2048 tokens: 989 us with boxes of 32 rows, 926 with
//                64, 897 with 192);
//   warp 2       MMA issuer (tcgen05.mma kind::f16, A from tensor memory) and TMEM owner;
//   warp 3       group table;
//   warps 4..    dequantisers: DQ sets of four warps, each takes every DQ-th
//                128-element k-block, thread by thread 16 words -> 64 columns of packed bf16
//                pairs (tcgen05.st), into its A stage of 64 columns;
//   then         epilogue: tcgen05.ld, row factor, activation, bf16 stores.
// TMEM: two accumulators, so that the epilogue of a tile overlaps the next one's main loop, and
// an A stage per dequantiser set: 2 x 192 and 2 x 64 columns, or 2 x 128 and 4 x 64.  (One
// accumulator of 256 columns left the tensor pipe idle for as long as an epilogue takes, a
// quarter of the time.)
// When few tokens share a weight the loop has to run at the rate of the weights' bytes (a stage
// of 16 KB of codes every 0.4 us), so stages are as long as memory allows: at 64-element A and
// token stages the barrier traffic of the one MMA thread alone took 1.2 us for 16 KB.
// What bounds it (8 groups of 14336 x 4096, gate and up): at 256 rows a group and more the pace
// of the dequantisers and the MMAs together, under the power cap (2048 tokens: 780 to 850 us, 1.13
// to 1.23 PFLOP/s; the tensor pipe is 81% busy in the 710 us that a single launch takes at full clock).
// At 8 to 64 rows a group 160 to 180 us (2.9 TB/s of codes): the MMA warp's own instructions,
// which share a scheduler with four dequantisers, so what they cost counts: one wait and branch
// for an A stage's eight MMAs and 32-bit descriptor arithmetic took 12 rows a group from 183 to
// 157 us, token stages of 256 instead of 128 k 64 rows from 192 to 175.  Twice the dequantisers
// (two warps a row, half an A stage each) made 2048 tokens 13% slower, a rolled loop over an A
// stage's halves 15%, predicated MMAs 7%; token boxes of exactly the tile's rows changed nothing
// at 12 rows a group and cost a third at 512.
// Every mbarrier wait is bounded (globaltimer); a wait that gives up records an error code in
// the device error word and the CTA drains what it has in flight and exits.
#include <cuda.h>

#include "common.cuh"
#include "mbar.cuh"
#include "tc_ops.cuh"
#include "w4.cuh"
#include "w4_wait.cuh"

namespace moe {
namespace {

constexpr int W4_ROWS = 128;                    // weight rows of a tile (TMEM lanes)
constexpr int W4_KS = 256;                      // k of a weight stage
constexpr int W4_KB = 64;                       // k of a token box
constexpr int W4_KA = 128;                      // k of an A stage
constexpr int W4_CODE_BYTES = W4_ROWS * W4_KS / 2;
constexpr int W4_SIDE_BYTES = 1024;             // scales (or zero points) of a stage: 8 x 128
constexpr int W4_W_STAGE = W4_CODE_BYTES + 2 * W4_SIDE_BYTES;
constexpr int W4_A_COLS = W4_KA / 2;
constexpr int W4_TMEM_COLS = 512;
constexpr int W4_FIRST_DQ = 4;

// Tokens of a tile; weight stages; token stages, their k and the rows of their boxes; accumulators;
// sets of four dequantisers and of four epilogue warps.  A weight stage of 256 k has two A blocks
// of 128: set i takes block i % 2 of every weight stage, or with four sets of every second one, and
// has an A stage of its own.  So a stage of either ring belongs to the same sets every round;
// others could be two rounds ahead and take a wait's parity for their own.
template <int NT> struct W4Shape;
template <> struct W4Shape<192> {
  static constexpr int WS = 3, XS = 3, XK = 128, XBOX = 64, ACCS = 2, DQ = 2, EPI = 2;
};
template <> struct W4Shape<128> {
  static constexpr int WS = 4, XS = 2, XK = 256, XBOX = 64, ACCS = 2, DQ = 4, EPI = 1;
};
template <> struct W4Shape<32> {
  static constexpr int WS = 8, XS = 4, XK = 256, XBOX = 32, ACCS = 2, DQ = 4, EPI = 1;
};
template <int NT> constexpr int w4_threads() {
  using S = W4Shape<NT>;
  static_assert(S::DQ == 2 || (S::DQ == 4 && S::WS % 2 == 0), "a weight stage has the same sets");
  static_assert(S::ACCS * (NT < 128 ? 128 : NT) + S::DQ * W4_A_COLS <= W4_TMEM_COLS,
                "TMEM columns");
  return 32 * (W4_FIRST_DQ + 4 * S::DQ + 4 * S::EPI);
}

struct W4Params {
  const int32_t* offsets;                       // [G + 1] device
  const float* rs0;                             // row factors [G, N]: up / down
  const float* rs1;                             // gate (SwiGLU)
  __nv_bfloat16* out;                           // [rows, N]
  int* err;
  int64_t rows;
  int G, N, K, group;
  int act;                                      // MOE_ACT_* or -1
  int zeros;
  int nt;                                       // weight tiles per group
  int fault;                                    // test hook: CTA 0 arms its first weight stage only
};

struct W4Tile {
  int g, n_idx, ntok, row0;
};

template <int NT>
__device__ __forceinline__ W4Tile w4_locate(int t, const int* grp_off, const int* tile_pre,
                                            int& g) {
  while (t >= tile_pre[g + 1]) ++g;
  const int m = grp_off[g + 1] - grp_off[g];
  const int mt = (m + NT - 1) / NT;
  const int per = ((m + mt - 1) / mt + 15) & ~15;     // rows of a token tile, alike for all
  const int local = t - tile_pre[g];
  W4Tile r;
  r.g = g;
  r.n_idx = local / mt;
  const int j = local - r.n_idx * mt;
  r.ntok = min(per, m - j * per);
  r.row0 = grp_off[g] + j * per;
  return r;
}

// (the halves of the token descriptor apart: only the low one changes)
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo,
                                             uint32_t b_hi, uint32_t acc, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ uint32_t bits(__nv_bfloat162 v) {
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ __nv_bfloat162 pair(uint32_t v) {
  return *reinterpret_cast<__nv_bfloat162*>(&v);
}

__device__ __forceinline__ __nv_bfloat162 scale_pair(uint8_t s) {
  return __float2bfloat162_rn(w4_scale(s));
}
__device__ __forceinline__ __nv_bfloat162 zero_pair(uint32_t z) {     // 128 + z
  return pair((0x4300u + z) * 0x10001u);
}

// (w & 0x000f000f) | 0x43004300 in one step (with two constants the compiler takes two)
__device__ __forceinline__ uint32_t nibbles(uint32_t w) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(w), "n"(0x000f000fu), "r"(0x43004300u));
  return r;
}
// Eight weights of a word as four bf16 pairs: (128 + code) by bits, minus (128 + zero), times
// scale; every step is exact.
__device__ __forceinline__ void dequant_word(uint32_t w, __nv_bfloat162 z, __nv_bfloat162 s,
                                             uint32_t* r) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = bits(__hmul2(__hsub2(pair(nibbles(w >> (4 * i))), z), s));
}

template <int NT, bool GLU>
__global__ void __launch_bounds__(w4_threads<NT>(), 1)
w4_gemm_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmXall,
               const __grid_constant__ CUtensorMap tmC0,
               const __grid_constant__ CUtensorMap tmC1, const __grid_constant__ CUtensorMap tmS0,
               const __grid_constant__ CUtensorMap tmS1, const __grid_constant__ CUtensorMap tmZ0,
               const __grid_constant__ CUtensorMap tmZ1, const W4Params p) {
  constexpr int WS = W4Shape<NT>::WS, XS = W4Shape<NT>::XS, XK = W4Shape<NT>::XK,
                ACCS = W4Shape<NT>::ACCS, DQ = W4Shape<NT>::DQ, AS = DQ,
                EPI = W4Shape<NT>::EPI, XBOX = W4Shape<NT>::XBOX;
  constexpr int ACC_PITCH = NT < 128 ? 128 : NT;      // columns between accumulators
  constexpr int A_COL = ACCS * ACC_PITCH;             // first column of the A ring
  constexpr int FIRST_EPI = W4_FIRST_DQ + 4 * DQ;
  constexpr int XBOX_BYTES = XBOX * W4_KB * 2;
  constexpr int XB = XK / W4_KB;                // 64-element boxes of a token stage
  constexpr int X_BOX = NT * W4_KB * 2;
  constexpr int X_STAGE = XB * X_BOX;
  constexpr int FEATS = GLU ? 64 : 128;         // outputs of a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* ws = smem + XS * X_STAGE;            // token stages, then weight stages
  uint64_t* bars = reinterpret_cast<uint64_t*>(ws + WS * W4_W_STAGE);
  constexpr int BARS = 2 * (WS + XS + AS + ACCS) + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* grp_off = reinterpret_cast<int*>(tmem_holder + 2);       // [G + 1]
  int* tile_pre = grp_off + (p.G + 1);                          // [G + 1]
  const uint32_t xs = smem_u32(smem);
  const uint32_t w_full = smem_u32(bars), w_empty = w_full + 8 * WS;
  const uint32_t x_full = w_empty + 8 * WS, x_empty = x_full + 8 * XS;
  const uint32_t a_full = x_empty + 8 * XS, a_empty = a_full + 8 * AS;
  const uint32_t t_full = a_empty + 8 * AS, t_empty = t_full + 8 * ACCS;
  const uint32_t drain = t_empty + 8 * ACCS;
  const BarWait wait{abort_flag, p.err};

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    uint64_t* b = bars;
    auto init = [&](int n, uint32_t count) {
      for (int i = 0; i < n; ++i) mbar_init(b++, count);
    };
    init(WS, 1);
    init(WS, 8);                                // two sets
    init(2 * XS, 1);
    init(AS, 4);
    init(AS, 1);
    init(ACCS, 1);
    init(ACCS, 4 * EPI);
    init(1, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_holder)),
                 "r"(W4_TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_trigger();
  pdl_wait();
  if (warp == 3) {
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
        tiles = ((m + NT - 1) / NT) * p.nt;
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
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // the CTA holds all 512 columns, so they start at 0: a constant keeps the MMA's addresses in
  // uniform registers
  constexpr uint32_t tmem_base = 0;
  const int total = tile_pre[p.G];
  const int nkb = p.K / W4_KB;                  // 64-element k-blocks
  const int nws = (nkb + 3) / 4;
  const int gs = W4_KS / p.group;               // scale rows of a weight stage
  const int groups = (p.K + p.group - 1) / p.group;

  const bool leader = elect_one();              // of the warp: the lane that issues

  if (warp == 0) {
    // ---------------- weights ----------------
    int stage = 0, g = 0;
    uint32_t phase = 0, issued = 0, issued_par = 0;
    bool ok = true;
    // a box moves its full size, parts outside the tensor as zeros
    const uint32_t tx = W4_CODE_BYTES + gs * W4_ROWS * (p.zeros ? 2 : 1);
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
      const W4Tile tl = w4_locate<NT>(t, grp_off, tile_pre, g);
      const int n0 = tl.n_idx * FEATS, row = tl.g * p.N + n0;
      for (int s = 0; s < nws; ++s) {
        if (!wait(w_empty + 8 * stage, phase ^ 1u, DEVERR_TIMEOUT_TMA)) {
          ok = false;
          break;
        }
        const uint32_t bar = w_full + 8 * stage;
        // test hook: the stage is armed but never loaded, so the dequantisers' wait runs out
        const bool load = !(p.fault == 1 && blockIdx.x == 0 && t == (int)blockIdx.x && s == 0);
        if (leader) bar_expect(bar, tx);
        if (leader && load) {
          const uint32_t c = xs + XS * X_STAGE + stage * W4_W_STAGE, sc = c + W4_CODE_BYTES,
                         z = sc + W4_SIDE_BYTES;
          const int kx = s * (W4_KS / 2), ky = tl.g * groups + s * gs;
          if (GLU) {
            bar_load(c, &tmC1, bar, kx, row);
            bar_load(c + W4_CODE_BYTES / 2, &tmC0, bar, kx, row);
            bar_load(sc, &tmS1, bar, n0, ky);
            bar_load(sc + W4_SIDE_BYTES / 2, &tmS0, bar, n0, ky);
            if (p.zeros) {
              bar_load(z, &tmZ1, bar, n0, ky);
              bar_load(z + W4_SIDE_BYTES / 2, &tmZ0, bar, n0, ky);
            }
          } else {
            bar_load(c, &tmC0, bar, kx, row);
            bar_load(sc, &tmS0, bar, n0, ky);
            if (p.zeros) bar_load(z, &tmZ0, bar, n0, ky);
          }
        }
        if (load) {
          issued |= 1u << stage;
          issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
        }
        if (++stage == WS) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // the last copies land before the CTA exits, whatever became of their consumers
    for (int s = 0; s < WS; ++s)
      if (issued & (1u << s))
        wait.drain(w_full + 8 * s, (issued_par >> s) & 1u, DEVERR_TIMEOUT_TMA, kDrainNs);
  } else if (warp == 1) {
    // ---------------- token rows ----------------
    int stage = 0, g = 0;
    uint32_t phase = 0, issued = 0, issued_par = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
      const W4Tile tl = w4_locate<NT>(t, grp_off, tile_pre, g);
      const int nbox = (tl.ntok + XBOX - 1) / XBOX;
      const bool all = nbox * XBOX == NT;       // as many rows as a box of the whole tile has
      for (int kb = 0; kb < nkb; kb += XB) {
        if (!wait(x_empty + 8 * stage, phase ^ 1u, DEVERR_TIMEOUT_TMA)) {
          ok = false;
          break;
        }
        const uint32_t bar = x_full + 8 * stage;
        const int here = min(XB, nkb - kb);
        if (leader) {
          bar_expect(bar, here * nbox * XBOX_BYTES);
          for (int h = 0; h < here; ++h) {
            const uint32_t to = xs + stage * X_STAGE + h * X_BOX;
            if (all)
              bar_load(to, &tmXall, bar, (kb + h) * W4_KB, tl.row0);
            else
              for (int b = 0; b < nbox; ++b)
                bar_load(to + b * XBOX_BYTES, &tmX, bar, (kb + h) * W4_KB, tl.row0 + b * XBOX);
          }
        }
        issued |= 1u << stage;
        issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
        if (++stage == XS) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    for (int s = 0; s < XS; ++s)
      if (issued & (1u << s))
        wait.drain(x_full + 8 * s, (issued_par >> s) & 1u, DEVERR_TIMEOUT_TMA, kDrainNs);
  } else if (warp == 2) {
    // ---------------- MMA issuer ----------------
    int xst = 0, ast = 0, it = 0, g = 0;
    uint32_t xph = 0, aph = 0;
    bool ok = true;
    const uint64_t bdesc = sdesc<W4_KB>(xs);
    const uint32_t b_lo = (uint32_t)bdesc, b_hi = (uint32_t)(bdesc >> 32);
    static_assert(XK % W4_KA == 0, "a token stage has whole A blocks");
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x, ++it) {
      const W4Tile tl = w4_locate<NT>(t, grp_off, tile_pre, g);
      const uint32_t idesc =
          idesc_bf16(W4_ROWS, __shfl_sync(kFullWarp, (tl.ntok + 15) & ~15, 0));
      const int acc = it % ACCS;
      const uint32_t d = tmem_base + acc * ACC_PITCH;
      if (!wait(t_empty + 8 * acc, (uint32_t)((it / ACCS) & 1) ^ 1u, DEVERR_TIMEOUT_MMA)) {
        ok = false;
        break;
      }
      tc_fence_after();
      for (int kb = 0; kb < 4 * nws && ok; kb += W4_KA / W4_KB) {     // (both A blocks of the last)
        if (!wait(a_full + 8 * ast, aph, DEVERR_TIMEOUT_MMA)) {
          ok = false;
          break;
        }
        const uint32_t a0 = tmem_base + A_COL + ast * W4_A_COLS;
        if (kb < nkb) {
          const int xb = kb % XB;               // first of its boxes within the token stage
          if (xb == 0 && !wait(x_full + 8 * xst, xph, DEVERR_TIMEOUT_MMA)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int end = min(W4_KA / W4_KB, nkb - kb);
          const bool last = (kb + end) % XB == 0 || kb + end == nkb;
          if (leader) {
            const uint32_t b = b_lo + (uint32_t)((xst * X_STAGE + xb * X_BOX) >> 4);
#pragma unroll
            for (int h = 0; h < W4_KA / W4_KB; ++h) {
              if (h >= end) break;
#pragma unroll
              for (int k = 0; k < W4_KB / 16; ++k)
                umma_bf16_ts(d, a0 + h * (W4_KB / 2) + 8 * k, b + h * (X_BOX >> 4) + 2 * k, b_hi,
                             (kb | h | k) ? 1u : 0u, idesc);
            }
            if (last) bar_commit(x_empty + 8 * xst);
          }
          if (last && ++xst == XS) {
            xst = 0;
            xph ^= 1u;
          }
        }
        if (leader) bar_commit(a_empty + 8 * ast);
        if (++ast == AS) {
          ast = 0;
          aph ^= 1u;
        }
      }
      if (ok && leader) bar_commit(t_full + 8 * acc);
    }
    // all MMAs issued by this thread complete before the CTA releases TMEM
    if (leader) bar_commit(drain);
    wait.drain(drain, 0u, DEVERR_TIMEOUT_MMA, ok ? kWaitNs : kDrainNs);
  } else if (warp >= W4_FIRST_DQ && warp < FIRST_EPI) {
    // ---------------- dequantisers ----------------
    const int q = warp & 3, set = (warp - W4_FIRST_DQ) >> 2;
    // row of the stage's codes, and where its scales start and step
    const int row = GLU ? (lane & 16) * 4 + 16 * q + (lane & 15) : 32 * q + lane;
    const int side = GLU ? (lane & 16) * (W4_SIDE_BYTES / 32) + 16 * q + (lane & 15) : row;
    const int pitch = GLU ? 64 : 128;
    const int shift = p.group == 32 ? 5 : p.group == 64 ? 6 : 7;
    const uint32_t trow = tmem_base + A_COL + ((uint32_t)(32 * q) << 16);
    const int b0 = (set & 1) * (W4_KA / W4_KB);         // first 64-element block of its A block
    const uint32_t a_col = trow + set * W4_A_COLS;
    int wst = 0;
    uint32_t wph = 0, aph = 1, mine = DQ == 4 ? set >> 1 : 0;   // own weight stage: mine is 0
    bool ok = true;
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
      for (int s = 0; s < nws; ++s) {
        if (mine == 0) {
          if (!wait(w_full + 8 * wst, wph, DEVERR_TIMEOUT_TMA)) {
            ok = false;
            break;
          }
          const uint8_t* st = ws + wst * W4_W_STAGE;
          const uint8_t* sc = st + W4_CODE_BYTES + side;
          const uint8_t* zp = sc + W4_SIDE_BYTES;
          // everything of the A stage's 128 k first: codes, scales, zero points (a block past K
          // is read as zeros or the next matrix's scales, and no MMA takes it)
          const uint8_t* src = st + row * 128;
          uint4 c[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            c[i] = *reinterpret_cast<const uint4*>(src + (((2 * b0 + i) ^ (row & 7)) << 4));
          __nv_bfloat162 s2[4], z2[4];        // per 32 k
          const int at = ((W4_KB * b0) >> shift) * pitch;
          s2[0] = scale_pair(sc[at]);
          z2[0] = zero_pair(p.zeros ? zp[at] : 8u);
          if (shift == 7) {
            s2[1] = s2[2] = s2[3] = s2[0];
            z2[1] = z2[2] = z2[3] = z2[0];
          } else if (shift == 6) {
            s2[1] = s2[0];
            z2[1] = z2[0];
            s2[2] = s2[3] = scale_pair(sc[at + pitch]);
            z2[2] = z2[3] = zero_pair(p.zeros ? zp[at + pitch] : 8u);
          } else {
#pragma unroll
            for (int i = 1; i < 4; ++i) {
              s2[i] = scale_pair(sc[at + i * pitch]);
              z2[i] = zero_pair(p.zeros ? zp[at + i * pitch] : 8u);
            }
          }
#pragma unroll
          for (int h = 0; h < W4_KA / W4_KB; ++h) {
            const uint4 lo = c[2 * h], hi = c[2 * h + 1];
            const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            uint32_t r[32];
#pragma unroll
            for (int j = 0; j < 2; ++j)       // 32-element halves of the block
#pragma unroll
              for (int i = 0; i < 4; ++i)
                dequant_word(w[2 * i + j], z2[2 * h + j], s2[2 * h + j], r + 16 * j + 4 * i);
            if (h == 0) {
              if (!wait(a_empty + 8 * set, aph, DEVERR_TIMEOUT_EPI)) {
                ok = false;
                break;
              }
              tc_fence_after();
            }
            tmem_st32(a_col + h * (W4_KB / 2), r);
          }
          if (!ok) break;
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            bar_arrive(a_full + 8 * set);
            bar_arrive(w_empty + 8 * wst);
          }
          aph ^= 1u;
        }
        if (DQ == 4) mine ^= 1u;
        if (++wst == WS) {
          wst = 0;
          wph ^= 1u;
        }
      }
    }
  } else if (warp >= FIRST_EPI) {
    // ---------------- epilogue ----------------
    const int q = warp & 3, set = (warp - FIRST_EPI) >> 2;
    int g = 0, it = 0;
    for (int t = blockIdx.x; t < total; t += gridDim.x, ++it) {
      const W4Tile tl = w4_locate<NT>(t, grp_off, tile_pre, g);
      const int acc = it % ACCS;
      const int feat = tl.n_idx * FEATS + (GLU ? 16 * q + (lane & 15) : 32 * q + lane);
      const float* rs = GLU && lane < 16 ? p.rs1 : p.rs0;
      const float f = feat < p.N ? __ldg(rs + (int64_t)tl.g * p.N + feat) : 0.f;
      if (!wait(t_full + 8 * acc, (uint32_t)((it / ACCS) & 1), DEVERR_TIMEOUT_EPI))
        break;
      tc_fence_after();
      const bool rows_ok = tl.row0 >= 0 && (int64_t)tl.row0 + tl.ntok <= p.rows;
      if (!rows_ok && lane == 0) atomicCAS(p.err, 0, DEVERR_BOUNDS);
      const bool st = rows_ok && feat < p.N;
      const uint32_t d = tmem_base + acc * ACC_PITCH + ((uint32_t)(32 * q) << 16);
      __nv_bfloat16* o = p.out + (int64_t)tl.row0 * p.N + feat;
#pragma unroll 1
      for (int c = 16 * set; c < tl.ntok; c += 16 * EPI) {
        uint32_t v[16];
        tmem_ld16(d + c, v);
        tmem_wait_ld();
        if (GLU) {
          // lane i and i + 16 hold gate and up of a feature: they take the even and the odd
          // tokens of a pair
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float even = __uint_as_float(v[i]) * f, odd = __uint_as_float(v[i + 1]) * f;
            const float got = __shfl_xor_sync(kFullWarp, lane < 16 ? odd : even, 16);
            const float gate = lane < 16 ? even : got, up = lane < 16 ? got : odd;
            const int tok = c + i + (lane >> 4);
            if (st && tok < tl.ntok)
              o[(int64_t)tok * p.N] =
                  __float2bfloat16_rn(__fdividef(gate, 1.0f + __expf(-gate)) * up);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float y = __uint_as_float(v[i]) * f;
            if (p.act == MOE_ACT_RELU) y = y < 0.f ? 0.f : y;        // a NaN stays one
            if (p.act == MOE_ACT_GELU) y = 0.5f * y * (1.0f + erff(y * 0.70710678118654752f));
            if (st && c + i < tl.ntok) o[(int64_t)(c + i) * p.N] = __float2bfloat16_rn(y);
          }
        }
      }
      // every TMEM read of this tile has completed: release the accumulator
      tc_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(t_empty + 8 * acc);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(W4_TMEM_COLS)
                 : "memory");
  }
}

template <int NT>
constexpr size_t w4_smem(int G) {
  using S = W4Shape<NT>;
  return 1024 + (size_t)S::XS * NT * S::XK * 2 + (size_t)S::WS * W4_W_STAGE +
         (2 * S::WS + 2 * S::XS + 2 * S::DQ + 2 * S::ACCS + 1) * 8 + 8 +
         (size_t)2 * (G + 1) * sizeof(int);
}

struct W4Maps {
  CUtensorMap x, xall, c0, c1, s0, s1, z0, z1;
};

template <int NT, bool GLU>
cudaError_t launch(const W4Maps& m, const W4Params& p, int64_t a_rows, cudaStream_t s) {
  const size_t smem = w4_smem<NT>(p.G);
  auto kern = w4_gemm_kernel<NT, GLU>;
  constexpr size_t most = w4_smem<NT>(1024);    // (groups of a call)
  static_assert(most <= kMaxSmem, "shared memory");
  cudaError_t e = allow_smem(kern, most);
  if (e != cudaSuccess) return e;
  const int64_t tiles = ((a_rows + NT - 1) / NT + p.G) * (int64_t)p.nt;
  const int sms = gemm_sm_count();
  const int grid = (int)(tiles < sms ? tiles : sms);
  return launch_pdl(kern, dim3(grid), dim3(w4_threads<NT>()), smem, s, m.x, m.xall, m.c0, m.c1,
                    m.s0, m.s1, m.z0, m.z1, p);
}

}  // namespace

cudaError_t launch_w4_gemm(int act, const void* a, int64_t a_rows, int K, const moe_w4_t* gate,
                           const moe_w4_t* w, int G, int N, const int32_t* offsets, void* out,
                           cudaStream_t s) {
  if (a_rows <= 0 || G <= 0) return cudaSuccess;
  const int groups = (K + w->group - 1) / w->group;
  // tensor-map coordinates are 32-bit
  if (a_rows > INT32_MAX || (int64_t)G * N > INT32_MAX || (int64_t)G * groups > INT32_MAX)
    return cudaErrorInvalidValue;
  const bool glu = gate != nullptr;
  const int feats = glu ? 64 : 128;
  // Tokens per tile by the groups' mean rows; groups differ, so a tile holds more than the mean.
  // Tiles of 32 / 128 / 192 tokens, us: 8 groups of 14336 x 4096, gate and up, 12 rows a group
  // 161 / 163 / 181, 32 rows 216 / 174 / 199, 96 rows 523 / 204 / 259, 128 rows 674 / 298 / 264;
  // 32 uneven groups of 2048 x 7168, 7 rows 152 / 161 / 175, 15 rows 174 / 164 / 177.
  const int64_t mean = (a_rows + G - 1) / G;
  const int nt_tok = mean > 112 ? 192 : mean > 12 ? 128 : 32;
  const int xbox = nt_tok == 32    ? W4Shape<32>::XBOX
                   : nt_tok == 128 ? W4Shape<128>::XBOX
                                   : W4Shape<192>::XBOX;
  alignas(64) W4Maps m;
  auto maps = [&](const moe_w4_t* q, CUtensorMap* c, CUtensorMap* sc, CUtensorMap* z) {
    const int gs = W4_KS / q->group;
    if (!make_map_u8(c, q->codes, (uint64_t)G * N, (uint64_t)K / 2, feats, 128, true)) return false;
    if (!make_map_u8(sc, q->scales, (uint64_t)G * groups, (uint64_t)N, gs, feats, false))
      return false;
    return make_map_u8(z, q->zeros ? q->zeros : q->scales, (uint64_t)G * groups, (uint64_t)N, gs,
                       feats, false);
  };
  if (!make_map(&m.x, a, (uint64_t)a_rows, (uint64_t)K, xbox, W4_KB) ||
      !make_map(&m.xall, a, (uint64_t)a_rows, (uint64_t)K, nt_tok, W4_KB) ||
      !maps(w, &m.c0, &m.s0, &m.z0) || !maps(glu ? gate : w, &m.c1, &m.s1, &m.z1))
    return cudaErrorInvalidValue;
  W4Params p{};
  p.offsets = offsets;
  p.rs0 = w->row_scale;
  p.rs1 = glu ? gate->row_scale : nullptr;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.err = device_error_word();
  p.rows = a_rows;
  p.G = G;
  p.N = N;
  p.K = K;
  p.group = w->group;
  p.act = act;
  p.zeros = w->zeros ? 1 : 0;
  p.nt = (N + feats - 1) / feats;
  p.fault = gemm_fault();
  if (nt_tok == 192)
    return glu ? launch<192, true>(m, p, a_rows, s) : launch<192, false>(m, p, a_rows, s);
  if (nt_tok == 128)
    return glu ? launch<128, true>(m, p, a_rows, s) : launch<128, false>(m, p, a_rows, s);
  return glu ? launch<32, true>(m, p, a_rows, s) : launch<32, false>(m, p, a_rows, s);
}

}  // namespace moe
