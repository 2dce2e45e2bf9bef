// Grouped product on 4-bit weights (w4.cuh) for few rows per group: weight streaming on
// mma.sync.
//
// "别只比较 Top-k" (ailearn moe-comparison), the expert-work account: in a small decode batch each
// expert's products have a few rows and stream the weights; "从 Dense FFN 到 MoE：用一个 Tiny
// Transformer 理解 Router、Top-K 与负载均衡" (f3dlife), section 3.
//
// out[r, n] = epi(row_scale[n] * sum_groups scale * sum_k (code - zero) a[r, k]).  The time is the
// codes' bytes, and next to them the integer work of unpacking (half rate on sm_100a).  So
//   - the weights go from shared memory straight into mma fragments as the whole numbers
//     code - zero, and the scale multiplies the fp32 sum of its group of k (one step per 32..128
//     k instead of one per weight);
//   - the product runs in fp16, whose 10 mantissa bits take a nibble at bits 0..3 or 4..7 of a
//     half word: one shift and four mask-and-or steps per 8 codes (bf16's 7 bits need three
//     shifts; putting a nibble into the mantissa of 1024 and taking 1024 off again is the method of
//     Kim et al., "Who Says Elephants Can't Run", 2022).  A token row is scaled by the power of two that brings its largest element to
//     [2^14, 2^15): its bf16 elements are then fp16 numbers exactly down to 2^-32 of the largest,
//     and what lies below is off by at most 2^-39 of it, far under the fp32 sums' own rounding.
//     The inverse power multiplies the finished sum.
//
// A CTA takes a tile of RT * 16 weight rows (SwiGLU: RT * 8 features, 8 rows of W_gate above the
// same 8 of W_up in one m16n8k16 fragment) by up to P <= 8 tokens of a group with 16 warps: RT
// side by side, WK = 16 / RT along K.  One more warp streams 256 k per warp and stage (TMA: codes,
// scales, zero points) into a ring that runs on from tile to tile; a warp that issued the copies
// of its own rows between its products spent half of its instructions on that.  The warps along K
// meet once a tile, where their partial sums go through shared memory.  CTAs own contiguous
// ranges of tiles (group by group, token tiles, then weight rows), so the P token rows are copied
// to shared memory about once per group.
#include <cuda.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "mbar.cuh"
#include "tc_ops.cuh"
#include "w4.cuh"
#include "w4_wait.cuh"

namespace moe {
namespace {

constexpr int ST_WARPS = 16;                    // that compute
constexpr int ST_THREADS = 32 * (ST_WARPS + 1);
constexpr int ST_K = 256;                       // k of a stage, per warp
constexpr int ST_STAGES = 3;
constexpr int ST_CODES = ST_WARPS * 16 * ST_K / 2;          // bytes of codes of a stage
constexpr int ST_SIDE = 2048;                   // its scales (or zero points)
constexpr int ST_STAGE = ST_CODES + 2 * ST_SIDE;
constexpr int ST_TOK = 8;
constexpr int ST_PART = 16 * ST_TOK;            // fp32 partial sums of a warp
constexpr int ST_XPAD = 64;                     // bytes: rows of x start 64 bytes apart mod 128
constexpr size_t ST_FIXED = 1024 + (size_t)ST_STAGES * ST_STAGE + 2 * ST_WARPS * ST_PART * 4 +
                            2 * ST_STAGES * 8 + 16 + 4 * ST_TOK * 4;

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
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// d = a b
__device__ __forceinline__ void mma_16816_first(float (&d)[4], const uint32_t (&a)[4],
                                                uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// The warps that compute, without the producer.
__device__ __forceinline__ void sync_compute() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * ST_WARPS) : "memory");
}

__device__ __forceinline__ uint32_t bits(__half2 v) { return *reinterpret_cast<uint32_t*>(&v); }
__device__ __forceinline__ __half2 halves(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }

// (w & mask) | 0x64006400: 1024 + nibble (mask 0x000f000f) or 1024 + 16 * nibble (0x00f000f0)
template <uint32_t MASK>
__device__ __forceinline__ uint32_t nibbles(uint32_t w) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(w), "n"(MASK), "r"(0x64006400u));
  return r;
}
// zero points of a row as the two forms' subtrahends
struct Zero {
  __half2 lo, hi;                               // 1024 + zero, -(64 + zero)
  __device__ __forceinline__ explicit Zero(uint32_t z)
      : lo(halves((0x6400u + z) * 0x10001u)), hi(halves(((0xd400u + 16u * z)) * 0x10001u)) {}
};
// Four pairs code - zero of a word, exact
__device__ __forceinline__ void unpack_word(uint32_t w, const Zero& z, uint32_t (&r)[4]) {
  const __half2 sixteenth = halves(0x2c002c00u);
  const uint32_t t = w >> 8;
  r[0] = bits(__hsub2(halves(nibbles<0x000f000fu>(w)), z.lo));
  r[1] = bits(__hfma2(halves(nibbles<0x00f000f0u>(w)), sixteenth, z.hi));
  r[2] = bits(__hsub2(halves(nibbles<0x000f000fu>(t)), z.lo));
  r[3] = bits(__hfma2(halves(nibbles<0x00f000f0u>(t)), sixteenth, z.hi));
}
// two e4m3 bytes as floats
__device__ __forceinline__ float2 scale_two(uint32_t a, uint32_t b) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(a + 256u * b), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// a bf16 in the low half of `v`, times p, as fp16 bits
__device__ __forceinline__ uint32_t to_half2(uint32_t v, float p) {
  const __half2 h = __floats2half2_rn(__uint_as_float(v << 16) * p,
                                      __uint_as_float(v & 0xffff0000u) * p);
  return bits(h);
}

// Per matrix: codes as [whole stages][rows][128 bytes], so that one copy brings what WK warps take
// (the issue of a copy per warp took longer than the bytes), and as [rows][bytes] for the rounds
// at K's end; scales and zero points.
struct StreamMaps {
  CUtensorMap codes, row_codes, scales, zeros;
};

template <bool GLU, bool ZEROS, int GROUP>
__global__ void __launch_bounds__(ST_THREADS, 1)
w4_stream_kernel(const __grid_constant__ StreamMaps m0, const __grid_constant__ StreamMaps m1,
                 const StreamParams p) {
  constexpr int GS = ST_K / GROUP;              // scale groups of a stage
  constexpr int MATS = GLU ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* part = reinterpret_cast<float*>(smem + ST_STAGES * ST_STAGE);
  uint64_t* bars = reinterpret_cast<uint64_t*>(part + 2 * ST_WARPS * ST_PART);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 2 * ST_STAGES);
  float* back = reinterpret_cast<float*>(bars + 2 * ST_STAGES) + 4;          // [2][ST_TOK]: the
                                                // tokens' inverse powers, by parity of x loads
  uint32_t* tops = reinterpret_cast<uint32_t*>(back + 2 * ST_TOK);           // [2][ST_TOK]: their
                                                // largest magnitudes
  uint8_t* xs = reinterpret_cast<uint8_t*>(tops + 2 * ST_TOK);
  const int xpitch = 2 * p.K + ST_XPAD;
  int* grp_off = reinterpret_cast<int*>(xs + p.P * xpitch);       // [G + 1]
  int* tile_pre = grp_off + (p.G + 1);                            // [G + 1]
  const uint32_t full = smem_u32(bars), empty = full + 8 * ST_STAGES;
  const BarWait wait{abort_flag, p.err};

  const int rows = (GLU ? 8 : 16) * p.RT;       // of a matrix in a tile: the tile's features
  const int feats = rows;
  const int feats_log = 31 - __clz(feats);      // RT is a power of two
  const int nt = (p.N + feats - 1) / feats;
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST_STAGES; ++i) {
      mbar_init(bars + i, 1);
      mbar_init(bars + ST_STAGES + i, ST_WARPS);
    }
    *abort_flag = 0;
    for (int i = 0; i < 2 * ST_TOK; ++i) tops[i] = 0;
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
  const bool leader = elect_one();
  if (t_lo >= t_hi) return;                     // the whole CTA
  StreamTile tl{};
  tl.start(t_lo, grp_off, tile_pre, nt, p.P, feats);

  if (warp == ST_WARPS) {
    // ---------------- producer ----------------
    const int groups = (p.K + GROUP - 1) / GROUP;
    int slot = 0;
    uint32_t phase = 0, issued = 0, issued_par = 0;
    bool ok = true;
    for (int t = t_lo; t < t_hi && ok; ++t) {
      const int row = tl.g * p.N + tl.n0;
      for (int s0 = 0; s0 < nst; s0 += p.WK) {
        // Warps that gave up on a stage go on to release it, with the flag raised before: no stage
        // is armed again whose copies never came.
        if (!wait(empty + 8 * slot, phase ^ 1u, DEVERR_TIMEOUT_TMA) ||
            __any_sync(kFullWarp, *abort_flag)) {
          ok = false;
          break;
        }
        const uint32_t bar = full + 8 * slot;
        // test hook: armed but never loaded, so the computing warps' wait runs out
        const bool load = !(p.fault == 1 && blockIdx.x == 0 && t == t_lo && s0 == 0);
        const bool whole = (s0 + p.WK) * ST_K <= p.K;
        const int n = min(p.WK, nst - s0);      // warps along K that have a stage
        if (leader) {
          bar_expect(bar, MATS * rows * (128 * n + GS * p.WK * (ZEROS ? 2 : 1)));
          if (load) {
            const int y = tl.g * groups + s0 * GS;
#pragma unroll
            for (int k = 0; k < MATS; ++k) {    // W_gate, then W_up; or the only matrix
              const StreamMaps& m = k == MATS - 1 ? m0 : m1;
              const uint32_t c = smem_u32(smem + slot * ST_STAGE) + k * rows * 128 * p.WK;
              const uint32_t d = smem_u32(smem + slot * ST_STAGE) + ST_CODES + k * rows * GS * p.WK;
              if (whole)
                bar_load_3d(c, &m.codes, bar, 0, row, s0);
              else
                for (int w = 0; w < n; ++w)
                  bar_load(c + w * rows * 128, &m.row_codes, bar, (s0 + w) * (ST_K / 2), row);
              bar_load(d, &m.scales, bar, tl.n0, y);
              if (ZEROS) bar_load(d + ST_SIDE, &m.zeros, bar, tl.n0, y);
            }
          }
        }
        if (load) {
          issued |= 1u << slot;
          issued_par = (issued_par & ~(1u << slot)) | (phase << slot);
        }
        if (++slot == ST_STAGES) {
          slot = 0;
          phase ^= 1u;
        }
      }
      if (t + 1 < t_hi) tl.next(grp_off, p.N, p.P, feats);
    }
    // the last copies land before the CTA exits, whatever became of their consumers
    for (int i = 0; i < ST_STAGES; ++i)
      if (issued & (1u << i))
        wait.drain(full + 8 * i, (issued_par >> i) & 1u, DEVERR_TIMEOUT_TMA, kDrainNs);
    return;
  }

  // ---------------- products ----------------
  const int wk = warp % p.WK, rt = warp / p.WK;
  const int q = lane >> 2, c = lane & 3;        // fragment row / token, and column pair
  const int prow = ((q & 3) << 1) | (q >> 2);   // weight row of fragment row q: reads of the
                                                // swizzled rows are then free of bank conflicts
  // this lane's bytes of a stage: 16-byte piece 0 of its two rows, and their scales
  const int code0 = wk * rows * 128 + rt * (GLU ? 1024 : 2048) + prow * 128 + 8 * (c & 1);
  const int code_up = GLU ? rows * 128 * p.WK : 1024;
  const int side0 = ST_CODES + wk * GS * rows + rt * (GLU ? 8 : 16) + prow;
  const int side_up = GLU ? rows * GS * p.WK : 8;
  const int lane_at = ((c >> 1) ^ prow) << 4;
  int slot = 0, x_row = -1, xbuf = 0, buf = 0;
  uint32_t phase = 0;
  bool alive = true;
  for (int t = t_lo; t < t_hi; ++t, buf ^= 1) {
    const bool rows_ok = tl.row0 >= 0 && (int64_t)tl.row0 + tl.ntok <= p.rows;
    if (tl.row0 != x_row) {
      // token rows of the new group or token tile (every warp has read the old ones: it has
      // arrived at the last tile's barrier): as they are, with the largest magnitude of each,
      // then scaled to fp16 in place, every vector by the thread that brought it
      if (!rows_ok && threadIdx.x == 0) atomicCAS(p.err, 0, DEVERR_BOUNDS);
      xbuf ^= 1;
      const int vec = p.K / 8;
      const uint4* src = reinterpret_cast<const uint4*>(p.a + (int64_t)tl.row0 * p.K);
#pragma unroll 1
      for (int r = 0; r < tl.ntok; ++r) {
        uint32_t top = 0;                       // as bits of a float
#pragma unroll 4
        for (int v = threadIdx.x; v < vec; v += 32 * ST_WARPS) {
          const uint4 u = rows_ok ? __ldg(src + (int64_t)r * vec + v) : make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4*>(xs + r * xpitch + 16 * v) = u;
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            top = max(top, max((w[i] << 16) & 0x7fffffffu, w[i] & 0x7fff0000u));
        }
        top = __reduce_max_sync(kFullWarp, top);
        if (lane == 0) atomicMax(&tops[xbuf * ST_TOK + r], top);
      }
      sync_compute();
#pragma unroll 1
      for (int r = 0; r < tl.ntok; ++r) {
        // 2^(141 - e) brings 2^(e - 127) to 2^14; infinities and NaN stay what they are
        const int e = min(max((int)(tops[xbuf * ST_TOK + r] >> 23), 15), 254);
        const float up = __uint_as_float((uint32_t)(268 - e) << 23);
        for (int v = threadIdx.x; v < vec; v += 32 * ST_WARPS) {
          uint4* at = reinterpret_cast<uint4*>(xs + r * xpitch + 16 * v);
          const uint4 u = *at;
          *at = make_uint4(to_half2(u.x, up), to_half2(u.y, up), to_half2(u.z, up),
                           to_half2(u.w, up));
        }
        if (threadIdx.x == 0) back[xbuf * ST_TOK + r] = 1.0f / up;
      }
      // the other buffer's, for the next load: its readers were before the barrier above
      if (threadIdx.x < ST_TOK) tops[(xbuf ^ 1) * ST_TOK + threadIdx.x] = 0;
      sync_compute();
      x_row = tl.row0;
    }
    // the factors of the feature that this thread finishes, under way during the products
    const int fin = tl.n0 + (threadIdx.x & (feats - 1));
    float rs_w = 0.f, rs_gate = 0.f;
    if (fin < p.N) {
      rs_w = __ldg(p.w.row_scale + (int64_t)tl.g * p.N + fin);
      if (GLU) rs_gate = __ldg(p.gate.row_scale + (int64_t)tl.g * p.N + fin);
    }
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    // lanes without a token repeat the last one: their columns of the product are not used
    const uint8_t* xrow = xs + min(q, tl.ntok - 1) * xpitch + 16 * c;
    for (int s = wk; s < nst + wk; s += p.WK) {
      if (alive) alive = wait(full + 8 * slot, phase, DEVERR_TIMEOUT_TMA);
      if (alive && s < nst) {
        const uint8_t* st = smem + slot * ST_STAGE + code0;
        const uint8_t* sd = smem + slot * ST_STAGE + side0;
        const uint8_t* xp = xrow + s * (2 * ST_K);
        const int here = (p.K - s * ST_K) / W4_BLOCK;       // 64-element blocks of the stage
        float sum[4];
        Zero z0(8u), z1(8u);
        auto block = [&](int b, bool last) {
          const int at = lane_at ^ (b << 5);
          const uint2 wa = *reinterpret_cast<const uint2*>(st + at);
          const uint2 wb = *reinterpret_cast<const uint2*>(st + code_up + at);
#pragma unroll
          for (int j = 0; j < 2; ++j) {         // 32-element halves
            const int k = 64 * b + 32 * j;
            const uint8_t* side = sd + k / GROUP * rows;
            if (ZEROS && k % GROUP == 0) {
              z0 = Zero(side[ST_SIDE]);
              z1 = Zero(side[ST_SIDE + side_up]);
            }
            const uint4 x = *reinterpret_cast<const uint4*>(xp + 2 * k);
            uint32_t ra[4], rb[4];
            unpack_word(j ? wa.y : wa.x, z0, ra);
            unpack_word(j ? wb.y : wb.x, z1, rb);
            const uint32_t a0[4] = {ra[0], rb[0], ra[1], rb[1]};
            const uint32_t a1[4] = {ra[2], rb[2], ra[3], rb[3]};
            if (k % GROUP == 0)
              mma_16816_first(sum, a0, x.x, x.y);
            else
              mma_16816(sum, a0, x.x, x.y);
            mma_16816(sum, a1, x.z, x.w);
            if ((k + 32) % GROUP == 0 || (j == 1 && last)) {
              const float2 sc = scale_two(side[0], side[side_up]);
              acc[0] = fmaf(sc.x, sum[0], acc[0]);
              acc[1] = fmaf(sc.x, sum[1], acc[1]);
              acc[2] = fmaf(sc.y, sum[2], acc[2]);
              acc[3] = fmaf(sc.y, sum[3], acc[3]);
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
      }
      __syncwarp();
      if (leader) bar_arrive(empty + 8 * slot);
      if (++slot == ST_STAGES) {
        slot = 0;
        phase ^= 1u;
      }
    }
    // sum over the WK warps of a row tile
    float* mypart = part + (buf * ST_WARPS + warp) * ST_PART + prow * ST_TOK + 2 * c;
    *reinterpret_cast<float2*>(mypart) = make_float2(acc[0], acc[1]);
    *reinterpret_cast<float2*>(mypart + 8 * ST_TOK) = make_float2(acc[2], acc[3]);
    sync_compute();
    if (rows_ok && fin < p.N) {
      constexpr int per = GLU ? 8 : 16;
      const int f = threadIdx.x & (feats - 1);  // (a multiple of feats threads: the same for each
                                                // of a thread's tokens)
      const float* src =
          part + (buf * ST_WARPS + (f / per) * p.WK) * ST_PART + (f % per) * ST_TOK;
      for (int tok = threadIdx.x >> feats_log; tok < tl.ntok; tok += 32 * ST_WARPS >> feats_log) {
        float v = 0.f, u = 0.f;
#pragma unroll 4
        for (int w = 0; w < p.WK; ++w) {
          v += src[w * ST_PART + tok];
          if (GLU) u += src[w * ST_PART + 8 * ST_TOK + tok];
        }
        // one after the other: a small row's power times a small row factor can be 0 or subnormal
        // where the result is not
        const float bk = back[xbuf * ST_TOK + tok];
        if (GLU) {
          v = v * bk * rs_gate;
          u = u * bk * rs_w;
          v = __fdividef(v, 1.0f + __expf(-v)) * u;
        } else {
          v = v * bk * rs_w;
          if (p.act == MOE_ACT_RELU) v = v < 0.f ? 0.f : v;          // a NaN stays one
          if (p.act == MOE_ACT_GELU) v = 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
        }
        p.out[((int64_t)tl.row0 + tok) * p.N + fin] = __float2bfloat16_rn(v);
      }
    }
    if (t + 1 < t_hi) tl.next(grp_off, p.N, p.P, feats);
  }
}

}  // namespace

// Tokens per tile that the shared memory holds next to the rings; 0: K is too long.
int w4_stream_tokens(int K, int G) {
  const size_t table = (size_t)2 * (G + 1) * sizeof(int);
  if (ST_FIXED + table >= kMaxSmem) return 0;
  const size_t n = (kMaxSmem - ST_FIXED - table) / (2 * (size_t)K + ST_XPAD);
  return n < ST_TOK ? (int)n : ST_TOK;
}

cudaError_t launch_w4_stream(int act, const void* a, int64_t a_rows, int K, const moe_w4_t* gate,
                             const moe_w4_t* w, int G, int N, const int32_t* offsets, void* out,
                             cudaStream_t s) {
  if (a_rows <= 0 || G <= 0) return cudaSuccess;
  const bool glu = gate != nullptr;
  const int gs = ST_K / w->group, groups = (K + w->group - 1) / w->group;
  StreamParams p{};
  p.P = w4_stream_tokens(K, G);
  // tensor-map coordinates are 32-bit
  if (p.P < 1 || (int64_t)G * N > INT32_MAX || (int64_t)G * groups > INT32_MAX)
    return cudaErrorInvalidValue;
  if (a_rows < p.P) p.P = (int)a_rows;
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
  p.WK = ST_WARPS / 2;                          // RT >= 2: a box of scales is 16 bytes or wider
  while (p.WK > 1 && (2 * p.WK > nst || 8 * nst < 7 * p.WK * ((nst + p.WK - 1) / p.WK)))
    p.WK /= 2;
  p.RT = ST_WARPS / p.WK;
  const int feats = (glu ? 8 : 16) * p.RT;
  alignas(64) StreamMaps m0, m1;
  auto maps = [&](const moe_w4_t* q, StreamMaps* m) {
    const uint64_t wrows = (uint64_t)G * N, srows = (uint64_t)G * groups, kb = (uint64_t)K / 2;
    return make_map_u8_3d(&m->codes, q->codes, wrows, K >= ST_K ? K / ST_K : 1, kb, feats, p.WK) &&
           make_map_u8(&m->row_codes, q->codes, wrows, kb, feats, 128, true) &&
           make_map_u8(&m->scales, q->scales, srows, (uint64_t)N, gs * p.WK, feats, false) &&
           make_map_u8(&m->zeros, q->zeros ? q->zeros : q->scales, srows, (uint64_t)N, gs * p.WK,
                       feats, false);
  };
  if (!maps(w, &m0) || !maps(glu ? gate : w, &m1)) return cudaErrorInvalidValue;
  const int64_t tiles = ((a_rows + p.P - 1) / p.P + G) * (int64_t)((N + feats - 1) / feats);
  const int sms = num_sms();
  const int grid = (int)(tiles < sms ? tiles : sms);
  const size_t smem = ST_FIXED + (size_t)p.P * (2 * (size_t)K + ST_XPAD) +
                      (size_t)2 * (G + 1) * sizeof(int);
  auto run = [&](auto kern) {
    cudaError_t e = allow_smem(kern, kMaxSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(grid), dim3(ST_THREADS), smem, s, m0, m1, p);
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
