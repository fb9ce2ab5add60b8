// A linear layer on microscaled 4-bit weights: out[t, n] = sum_k xq[t, k] wq[n, k], both
// factors e2m1 codes with a scale per block of K (e8m0 per 32, or e4m3 per 16 times one float),
// x quantised on the way in.
//
// Two forms, chosen by linear_fp4_by_rows.  With more than a few tokens or a large matrix, two launches:
//   1. fp4_prepare: x -> codes [T, K/2] and scales, and the weight's scales, both placed in the
//      128-row x 4-scale atoms that the tensor core reads (byte (row % 32) * 16 + (row / 32) * 4
//      + scale), one contiguous run a k-step of 256 elements and tile.  Bound by the read of x.
//   2. gemm_fp4_pair: CTA pairs, tcgen05.mma kind::mxf4nvf4 / mxf4 (cta_group::2): M = 256
//      tokens (128 a CTA), N = up to 224 weight rows (each CTA loads half, its partner's half
//      is read by the tensor core over the pair).  224 is the widest tile that leaves two
//      accumulators (448 columns) and the scales (48) in the 512 columns of TMEM, so the
//      epilogue of a tile runs under the next tile's products; a tile of 256 would read a
//      tenth fewer bytes a product and stall for its epilogue.  T = N = 8192, K = 4096: 106 us
//      (5.2 PFLOP/s; 99 us with e8m0 scales): the products 81, the copies of the scales into
//      tensor memory between them 16 (twelve a k-step, about 8 cycles each), loads 9, stores 7.
// With one token, or up to 16 of a matrix that is not large, one launch: every block quantises the
// rows of x (four at most) into shared memory, a warp takes a weight row at a time.  The products of
// two e2m1 numbers are multiples of 1/4 of at most 36, so eight of them add up exactly in a half;
// each block of 16 is then scaled and added in fp32.  Bound by instructions (6.7 a weight and
// thread) and a row's latency: 4096 x 4096, one token, 6.1 us at 11 % of DRAM.
#include <atomic>

#include "../../include/moe.h"
#include "moe_block.h"
#include "moe_fp4.cuh"
#include "moe_internal.h"
#include "moe_pair.cuh"

namespace moe {
namespace {

// ---------------------------------------------------------------- quantisation

__device__ __forceinline__ float element(const RowView& x, int64_t row, int64_t c) {
  const int64_t off = row * x.s0 + c * x.s1;
  return x.dtype == MOE_F32
             ? static_cast<const float*>(x.data)[off]
             : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(x.data)[off]) << 16);
}

// 32 neighbours of a row; wide: bf16 or f32 with unit inner stride and 16-byte aligned rows
__device__ __forceinline__ void read32(const RowView& x, bool wide, int64_t row, int64_t c, float (&v)[32]) {
  if (wide && x.dtype == MOE_BF16) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x.data) + row * x.s0 + c);
    uint4 r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = p[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
        v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    }
  } else if (wide) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x.data) + row * x.s0 + c);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 r = p[i];
      v[4 * i] = r.x; v[4 * i + 1] = r.y; v[4 * i + 2] = r.z; v[4 * i + 3] = r.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = element(x, row, c + i);
  }
}

// 16 neighbours of a row, as read32
__device__ __forceinline__ void read16(const RowView& x, bool wide, int64_t row, int64_t c, float (&v)[16]) {
  if (wide && x.dtype == MOE_BF16) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x.data) + row * x.s0 + c);
    const uint4 a = p[0], b = p[1];
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  } else if (wide) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x.data) + row * x.s0 + c);
    float4 r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = p[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[4 * i] = r[i].x; v[4 * i + 1] = r[i].y; v[4 * i + 2] = r[i].z; v[4 * i + 3] = r[i].w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = element(x, row, c + i);
  }
}

// Codes (16 bytes) and scales (kNv: two e4m3 bytes; else one e8m0 byte) of 32 elements.
template <bool kNv>
__device__ __forceinline__ uint32_t quant32(const float (&v)[32], float G, uint32_t (&w)[4]) {
  if constexpr (kNv) {
    uint32_t a[2], b[2];
    const float inv6 = 1.0f / (6.0f * G);
    const uint32_t s0 = nv_quant16(v, amax16(v), G, inv6, a), s1 = nv_quant16(v + 16, amax16(v + 16), G, inv6, b);
    w[0] = a[0]; w[1] = a[1]; w[2] = b[0]; w[3] = b[1];
    return s0 | (s1 << 8);
  } else {
    return mx_quant32(v, w);
  }
}

constexpr int kAtomBytes = 512;
constexpr int kStepElems = 256;  // elements of K a pipeline stage holds (128 bytes a row)
template <bool kNv>
constexpr int atoms_per_step() { return kNv ? 4 : 2; }

struct FpPrepare {
  RowView x;
  int wide;
  int64_t T, K, N;
  int num_k, ntile, nh;   // k-steps, weight rows a tile, 128-row blocks a tile
  int64_t row_tiles, x_blocks, n_nt;  // 16-row tiles and blocks of x, tiles of the weight
  const float* x_global;
  uint8_t* codes;         // [T, num_k * 128]
  uint8_t* x_atoms;       // [128-row block][k-step][atom]
  const uint8_t* w_sf;
  int64_t ws0, ws1;
  uint8_t* w_atoms;       // [tile][k-step][atom][block]
};

// Blocks of 16 x 16 threads.  The first x_blocks walk over tiles of 16 rows x 256 elements of x,
// a thread 16 neighbours of a row, the next tile's on their way while the last ones are quantised;
// the others place the weight's scales.  kFast: bf16, 16-byte loads.  T = 8192, K = 4096: 23 us, 21 of
// them without the arithmetic (reading x and writing the codes would take 13); more rows on their
// way at once, or whole rows a block, were slower (32 and 24.5 us).
template <bool kNv, bool kFast>
__global__ void __launch_bounds__(256, 4) fp4_prepare_kernel(const FpPrepare g) {
  constexpr int kAtoms = atoms_per_step<kNv>();
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x < g.x_blocks) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float G = 1.0f, inv6 = 0.0f;
    if (kNv) {
      G = *g.x_global;
      inv6 = 1.0f / (6.0f * G);
    }
    // a block keeps its k-step and goes down the rows
    const int step = static_cast<int>(blockIdx.x % g.num_k), c = step * 256 + tx * 16;
    const int64_t first = blockIdx.x / g.num_k, stride = g.x_blocks / g.num_k;
    const bool cols = c < g.K;
    uint4 next[2];
    auto fetch = [&](int64_t rb) {
      const int64_t row = rb * 16 + ty;
      if (row < g.T && cols) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(g.x.data) + row * g.x.s0 + c);
        next[0] = p[0];
        next[1] = p[1];
      }
    };
    if (kFast) fetch(first);
    for (int64_t rb = first; rb < g.row_tiles; rb += stride) {
      const uint4 cur[2] = {next[0], next[1]};
      if (kFast) fetch(rb + stride);
      const int64_t row = rb * 16 + ty;
      uint32_t sc = 0;
      if (row < g.T && cols) {
        float v[16], amax;
        if constexpr (kFast) {
          const uint32_t w[8] = {cur[0].x, cur[0].y, cur[0].z, cur[0].w,
                                 cur[1].x, cur[1].y, cur[1].z, cur[1].w};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
          }
          // magnitudes order as integers: two a step
          uint32_t m = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
          amax = max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
        } else {
          read16(g.x, g.wide, row, c, v);
          amax = amax16(v);
        }
        uint32_t w[2];
        if constexpr (kNv) {
          sc = nv_quant16(v, amax, G, inv6, w);
        } else {
          // (K is a multiple of 32: both threads of a block are here)
          amax = max_nan(amax, __shfl_xor_sync(0x3u << (threadIdx.x & 30), amax, 1));
          const int e = mx_scale_exp(amax);
          const float f = exp2i_neg(e);
          w[0] = cvt_e2m1x8(v, f);
          w[1] = cvt_e2m1x8(v + 8, f);
          sc = amax != amax ? kNanE8m0 : static_cast<uint32_t>(e + 127);
        }
        *reinterpret_cast<uint2*>(g.codes + row * (static_cast<int64_t>(g.num_k) * 128) + (c >> 1)) = make_uint2(w[0], w[1]);
      }
      // the threads of an atom's word (four blocks of 16, or of 32) hand their scales to the first
      constexpr int kStep = kNv ? 1 : 2;  // threads a scale
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) sc |= __shfl_down_sync(0xffffffffu, sc, o * kStep) << (8 * o);
      if (tx % (4 * kStep) == 0) {
        const int r = static_cast<int>(row & 127);
        *reinterpret_cast<uint32_t*>(g.x_atoms + (((row >> 7) * g.num_k + step) * kAtoms + tx / (4 * kStep)) * kAtomBytes +
                                     (r & 31) * 16 + (r >> 5) * 4) = sc;
      }
    }
    return;
  }
  const int64_t wb = static_cast<int64_t>(blockIdx.x) - g.x_blocks;
  const int step = static_cast<int>(wb % g.num_k);
  // [tile][atom][128-row block][lane] of this step
  const int64_t i = wb / g.num_k * 256 + threadIdx.x;
  const int lane = static_cast<int>(i & 31), log_nh = g.nh - 1;
  const int h = static_cast<int>(i >> 5) & (g.nh - 1), a = static_cast<int>(i >> (5 + log_nh)) & (kAtoms - 1);
  const int64_t tile = i >> (5 + log_nh + (kNv ? 2 : 1));
  if (tile >= g.n_nt) return;
  const int64_t q = (static_cast<int64_t>(step) * kAtoms + a) * 4, nq = g.K / (kNv ? 16 : 32);
  const bool whole = g.ws1 == 1 && q + 4 <= nq && (reinterpret_cast<uintptr_t>(g.w_sf) | g.ws0) % 4 == 0;
  uint32_t word[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = h * 128 + lane + 32 * j;
    const int64_t n = tile * g.ntile + r;
    word[j] = 0;
    if (r >= g.ntile || n >= g.N) continue;
    const uint8_t* p = g.w_sf + n * g.ws0 + q * g.ws1;
    if (whole) {
      word[j] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      for (int b = 0; b < 4; ++b)
        if (q + b < nq) word[j] |= static_cast<uint32_t>(p[b * g.ws1]) << (8 * b);
    }
  }
  const int64_t atom = ((tile * g.num_k + step) * kAtoms + a) * g.nh + h;
  *reinterpret_cast<uint4*>(g.w_atoms + atom * kAtomBytes + lane * 16) = make_uint4(word[0], word[1], word[2], word[3]);
}

// One thread a block of 32: codes and scales in plain row-major form.
__global__ void __launch_bounds__(256) quantize_nv_kernel(RowView x, int wide, int64_t rows, int64_t K,
                                                          const float* global, uint8_t* codes, int64_t ld,
                                                          uint8_t* sf, int64_t sf_ld, int code16, int sf2) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t per_row = K / 32, total = rows * per_row;
  const float G = *global;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t row = i / per_row, c = i - row * per_row;
    float v[32];
    read32(x, wide, row, c * 32, v);
    uint32_t w[4];
    const uint32_t sc = quant32<true>(v, G, w);
    uint8_t* d = codes + row * ld + c * 16;
    if (code16) {
      *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      for (int b = 0; b < 16; ++b) d[b] = static_cast<uint8_t>(w[b >> 2] >> (8 * (b & 3)));
    }
    uint8_t* s = sf + row * sf_ld + c * 2;
    if (sf2) {
      *reinterpret_cast<uint16_t*>(s) = static_cast<uint16_t>(sc);
    } else {
      s[0] = static_cast<uint8_t>(sc);
      s[1] = static_cast<uint8_t>(sc >> 8);
    }
  }
}

// ---------------------------------------------------------------- the product on CTA pairs

constexpr int kTokRows = 128;                  // token rows of a CTA
constexpr int kRowBytes = 128;                 // 256 codes
constexpr int kMaxTile = 224;                  // weight rows of a pair's tile
constexpr int kEpiWarps = 8;                   // two per TMEM lane quadrant
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr int kTmemCols = 512;
constexpr int kStagingBytes = 32 * 64;         // a warp's 32 x 32 bf16 outputs
constexpr int kSfCol = 2 * kMaxTile;

template <bool kNv>
struct Cfg {
  static constexpr int kAtoms = atoms_per_step<kNv>();
  static constexpr int kABytes = kTokRows * kRowBytes;
  static constexpr int kBBytes = (kMaxTile / 2) * kRowBytes;
  static constexpr int kSfaBytes = kAtoms * kAtomBytes;
  static constexpr int kSfbBytes = 2 * kAtoms * kAtomBytes;
  static constexpr int kStageBytes = kABytes + kBBytes + kSfaBytes + kSfbBytes;
  static constexpr int kStages = 5;
  static_assert(kStageBytes % 1024 == 0 && kBBytes % 1024 == 0, "swizzle atoms");
  static_assert(kSfCol + 3 * 4 * kAtoms <= kTmemCols, "TMEM budget");
  static constexpr size_t kSmem = 1024 + size_t(kStages) * kStageBytes + kEpiWarps * kStagingBytes +
                                  (2 * kStages + 5) * 8 + 16;
  static_assert(kSmem <= 232448, "shared memory per block");
};

struct FpGemm {
  int64_t T, N, total;     // total: tiles
  int num_k, ntile, nh, n_mt;
  const float* x_global;   // null: 1
  const float* w_global;
  __nv_bfloat16* out;
  int64_t os0, os1;
  int vec_out;
  DeviceErrors* err;
};

// D (+)= (A SFA) (B SFB)^T on the pair: 64 codes of K an instruction
template <bool kNv>
__device__ __forceinline__ void mma_fp4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                             uint32_t sfb, uint32_t accumulate) {
  if constexpr (kNv)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.block16 [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
        : "memory");
}
__device__ __forceinline__ void tmem_cp_pair(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

template <bool kNv>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_fp4_pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                         const __grid_constant__ CUtensorMap tmSfx, const __grid_constant__ CUtensorMap tmSfw,
                         const FpGemm g) {
  using C = Cfg<kNv>;
  constexpr int kStages = C::kStages, kAtoms = C::kAtoms;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* stages = base;
  uint8_t* staging = base + kStages * C::kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + kEpiWarps * kStagingBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;

  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmSfx);
    tma_prefetch_desc(&tmSfw);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers exist before any cross-CTA arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  pdl_wait();
  const int64_t pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    if (elect_one()) {
      uint32_t stage = 0, phase = 0;
      int8_t last_phase[kStages];
      for (int s = 0; s < kStages; ++s) last_phase[s] = -1;
      const uint64_t pol = l2_policy_evict_last();
      const int half = g.ntile / 2;
      const uint32_t bytes_pair =
          2u * static_cast<uint32_t>(C::kABytes + half * kRowBytes + C::kSfaBytes + g.nh * C::kSfaBytes);
      bool ok = true;
      for (int64_t item = pair; item < g.total && ok; item += n_pairs) {
        const int32_t nt = static_cast<int32_t>(item / g.n_mt), mt = static_cast<int32_t>(item - int64_t(nt) * g.n_mt);
        const int32_t row = mt * 2 * kTokRows + static_cast<int32_t>(rank) * kTokRows;
        const int32_t col = nt * g.ntile + static_cast<int32_t>(rank) * half;
        for (int kb = 0; kb < g.num_k; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, g.err)) { ok = false; break; }
          uint8_t* sa = stages + stage * C::kStageBytes;
          uint8_t* sb = sa + C::kABytes;
          uint8_t* sfa = sb + C::kBBytes;
          uint8_t* sfb = sfa + C::kSfaBytes;
          if (leader) mbar_arrive_expect_tx(&full[stage], bytes_pair);
          const uint32_t fb = mapa_shared(smem_u32(&full[stage]), 0);
          tma_load_2d_pair(sa, &tmX, fb, kb * kRowBytes, row, pol);
          tma_load_2d_pair(sb, &tmW, fb, kb * kRowBytes, col, pol);
          tma_load_2d_pair(sfa, &tmSfx, fb, 0, ((row / kTokRows) * g.num_k + kb) * kAtoms, pol);
          tma_load_2d_pair(sfb, &tmSfw, fb, 0, (nt * g.num_k + kb) * kAtoms * g.nh, pol);
          last_phase[stage] = static_cast<int8_t>(phase);
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok && leader) {
        for (int s = 0; s < kStages; ++s)
          if (last_phase[s] >= 0) mbar_wait(&full[s], static_cast<uint32_t>(last_phase[s]), g.err);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader only)
    if (leader && elect_one()) {
      uint32_t stage = 0, phase = 0, buf = 0, acc_phase = 0;
      bool ok = true, issued = false;
      const uint32_t sf_a = tmem_base + kSfCol, sf_b = sf_a + 4 * kAtoms;
      for (int64_t item = pair; item < g.total && ok; item += n_pairs) {
        if (!mbar_wait(&tempty[buf], acc_phase ^ 1u, g.err)) { ok = false; break; }
        tc_fence_after();
        const uint32_t acc = tmem_base + buf * kMaxTile;
        for (int kb = 0; kb < g.num_k; ++kb) {
          if (!mbar_wait(&full[stage], phase, g.err)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(stages + stage * C::kStageBytes);
          const uint32_t b_addr = a_addr + C::kABytes;
          const uint32_t sfa = b_addr + C::kBBytes, sfb = sfa + C::kSfaBytes;
          // copies and products of one thread run in the order they are issued, so the
          // scales of a step follow the products of the step before into the same columns
#pragma unroll
          for (int a = 0; a < kAtoms; ++a) tmem_cp_pair(sf_a + 4 * a, plain_rows16_desc(sfa + kAtomBytes * a));
          for (int a = 0; a < kAtoms * g.nh; ++a) tmem_cp_pair(sf_b + 4 * a, plain_rows16_desc(sfb + kAtomBytes * a));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint32_t atom = kNv ? kk : kk >> 1, id = kNv ? 0u : 2u * (kk & 1);
            uint32_t idesc = idesc_mxf4(2 * kTokRows, g.ntile, id, id);
            if (kNv) idesc &= ~(1u << 23);  // scale format e4m3
            mma_fp4_pair<kNv>(acc, sw128_kmajor_desc(a_addr + kk * 32), sw128_kmajor_desc(b_addr + kk * 32), idesc,
                              (sf_a + 4 * atom) | (id << 30), (sf_b + 4 * atom * g.nh) | (id << 30),
                              (kb > 0 || kk > 0) ? 1u : 0u);
          }
          issued = true;
          commit_pair(&empty[stage], 0x3);
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        commit_pair(&tfull[buf], 0x3);
        if (++buf == 2) { buf = 0; acc_phase ^= 1u; }
      }
      if (issued) {
        // let every tcgen05 operation of the pair (and its arrivals) finish
        commit_pair(drain, 0x1);
        mbar_wait(drain, 0, g.err);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int quad = warp & 3, part2 = (warp - 2) >> 2;
    const uint32_t stg = smem_u32(staging + (warp - 2) * kStagingBytes);
    const float scale = (g.x_global ? *g.x_global : 1.0f) * (g.w_global ? *g.w_global : 1.0f);
    uint32_t buf = 0, acc_phase = 0;
    for (int64_t item = pair; item < g.total; item += n_pairs) {
      const int64_t nt = item / g.n_mt, mt = item - nt * g.n_mt;
      const int64_t row0 = mt * 2 * kTokRows + rank * kTokRows + quad * 32;
      if (!mbar_wait(&tfull[buf], acc_phase, g.err)) break;
      tc_fence_after();
      const uint32_t acc = tmem_base + buf * kMaxTile + (static_cast<uint32_t>(quad * 32) << 16);
      for (int c = part2; c * 32 < g.ntile; c += 2) {
        const int64_t col0 = nt * g.ntile + c * 32;
        if (col0 >= g.N || row0 >= g.T) break;
        uint32_t v[32];
        tmem_ld32(acc + c * 32, v);
        tmem_wait_ld();
        // the row's 64 bytes in four parts, at a position turned by the row: neither the
        // stores (a lane a row) nor the loads (four lanes a row) meet in a bank
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = pack_bf16x2(scale * __uint_as_float(v[8 * p + 2 * i]), scale * __uint_as_float(v[8 * p + 2 * i + 1]));
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stg + lane * 64 + ((p ^ (lane >> 1)) & 3) * 16),
                       "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                       : "memory");
        }
        __syncwarp();
        if (g.vec_out) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int j = q * 8 + (lane >> 2), p = lane & 3;
            uint4 w;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                         : "r"(stg + j * 64 + ((p ^ (j >> 1)) & 3) * 16));
            if (row0 + j >= g.T) continue;
            const int64_t col = col0 + p * 8;
            __nv_bfloat16* dst = g.out + (row0 + j) * g.os0 + col;
            if (col + 8 <= g.N) {
              *reinterpret_cast<uint4*>(dst) = w;
            } else {
              const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
              for (int i = 0; i < 8 && col + i < g.N; ++i)
                reinterpret_cast<uint16_t*>(dst)[i] = static_cast<uint16_t>(ws[i >> 1] >> (16 * (i & 1)));
            }
          }
        } else {
          for (int j = 0; j < 32 && row0 + j < g.T; ++j) {
            uint16_t one;
            asm volatile("ld.shared.b16 %0, [%1];"
                         : "=h"(one)
                         : "r"(stg + j * 64 + (((lane >> 3) ^ (j >> 1)) & 3) * 16 + (lane & 7) * 2));
            if (col0 + lane < g.N)
              reinterpret_cast<uint16_t*>(g.out)[(row0 + j) * g.os0 + (col0 + lane) * g.os1] = one;
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cluster(mapa_shared(smem_u32(&tempty[buf]), 0));
      if (++buf == 2) { buf = 0; acc_phase ^= 1u; }
    }
  }

  pdl_launch_dependents();
  __syncthreads();
  cluster_sync_all();  // neither CTA leaves while the other may still signal it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

// ---------------------------------------------------------------- a few rows

constexpr int kRowsThreads = 256;

struct FpRows {
  RowView x;
  int wide;
  int T, K, groups;        // groups: blocks of 32
  int64_t N;
  const float* x_global;
  const float* w_global;
  const uint8_t* w;
  int64_t w_ld;
  const uint8_t* w_sf;
  int64_t ws0, ws1;
  __nv_bfloat16* out;
  int64_t os0, os1;
};

// Four tokens a blockIdx.y.  x in shared memory: halves [T][group of 32][4 parts of 16 bytes, turned by the group] and the
// scales of each group of 16 (kNv) or 32 as floats.
template <bool kNv, int kT>
__global__ void __launch_bounds__(kRowsThreads, kT <= 2 ? 4 : 2) linear_fp4_rows_kernel(const FpRows g) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kScales = kNv ? 2 : 1;
  const int G = g.groups;
  uint8_t* xh = smem;
  float* xs = reinterpret_cast<float*>(smem + static_cast<size_t>(kT) * G * 64);
  const int lane = threadIdx.x & 31;
  uint4 wv[4];
  uint32_t sv[4];
  // 128 blocks of 32 of a weight row: codes and scales, a lane four of them
  auto fetch = [&](int64_t n, int c0) {
    const uint8_t* wr = g.w + n * g.w_ld;
    const uint8_t* sr = g.w_sf + n * g.ws0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = c0 + 32 * u;
      wv[u] = make_uint4(0, 0, 0, 0);
      sv[u] = 0;
      if (c < G) {
        wv[u] = *reinterpret_cast<const uint4*>(wr + c * 16);
        sv[u] = sr[c * kScales * g.ws1];
        if (kNv) sv[u] |= static_cast<uint32_t>(sr[(2 * c + 1) * g.ws1]) << 8;
      }
    }
  };
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (kRowsThreads / 32);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kRowsThreads / 32) + (threadIdx.x >> 5);
  const int t0 = blockIdx.y * kT, nt = g.T - t0;  // (of the last four some may be missing)
  pdl_wait();
  pdl_launch_dependents();
  if (first < g.N) fetch(first, lane);  // on their way while x is quantised
  const float xg = kNv ? *g.x_global : 1.0f;
  for (int i = threadIdx.x; i < kT * G * 2; i += kRowsThreads) {  // blocks of 16 (G is whole: pairs stay together)
    const int t = i / (2 * G), c16 = i - t * 2 * G, c = c16 >> 1;
    float v[16];
    if (t < nt) {
      read16(g.x, g.wide, t0 + t, c16 * 16, v);
    } else {
#pragma unroll
      for (int q = 0; q < 16; ++q) v[q] = 0.0f;
    }
    uint32_t w[2];
    const float amax = amax16(v);
    if constexpr (kNv) {
      xs[i] = e4m3x2_floats(nv_quant16(v, amax, xg, 1.0f / (6.0f * xg), w)).x;
    } else {
      const float both = max_nan(amax, __shfl_xor_sync(0x3u << (threadIdx.x & 30), amax, 1));
      const int e = mx_scale_exp(both);
      const float f = exp2i_neg(e);
      w[0] = cvt_e2m1x8(v, f);
      w[1] = cvt_e2m1x8(v + 8, f);
      if ((c16 & 1) == 0) xs[t * G + c] = both != both ? both : exp2i_neg(-e);
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      uint4 h;
      h.x = e2m1x2_halves(w[q] & 0xffu);
      h.y = e2m1x2_halves((w[q] >> 8) & 0xffu);
      h.z = e2m1x2_halves((w[q] >> 16) & 0xffu);
      h.w = e2m1x2_halves(w[q] >> 24);
      const int p = 2 * (c16 & 1) + q;
      *reinterpret_cast<uint4*>(xh + (static_cast<size_t>(t * G + c) * 4 + ((p ^ (c >> 1)) & 3)) * 16) = h;
    }
  }
  __syncthreads();
  const float scale = xg * (g.w_global ? *g.w_global : 1.0f);
  for (int64_t n = first; n < g.N; n += stride) {
    float acc[kT];
#pragma unroll
    for (int t = 0; t < kT; ++t) acc[t] = 0.0f;
    for (int c0 = lane; c0 < G; c0 += 128) {
      if (n != first || c0 != lane) fetch(n, c0);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int c = c0 + 32 * u;
        if (c >= G) break;
        const uint32_t words[4] = {wv[u].x, wv[u].y, wv[u].z, wv[u].w};
        float ws[2];
        if (kNv) {
          const float2 s = e4m3x2_floats(sv[u]);
          ws[0] = s.x;
          ws[1] = s.y;
        } else {
          ws[0] = ws[1] = sv[u] == kNanE8m0 ? __uint_as_float(0x7fffffffu) : exp2i_neg(127 - static_cast<int>(sv[u]));
        }
        __half2 wh[16];
#pragma unroll
        for (int p = 0; p < 4; ++p)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const uint32_t h = e2m1x2_halves((words[p] >> (8 * b)) & 0xffu);
            wh[4 * p + b] = *reinterpret_cast<const __half2*>(&h);
          }
#pragma unroll
        for (int t = 0; t < kT; ++t) {
          const int i = t * G + c;
          float part[2];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            __half2 s = __float2half2_rn(0.0f);
#pragma unroll
            for (int p = 2 * q; p < 2 * q + 2; ++p) {
              const uint4 h = *reinterpret_cast<const uint4*>(xh + (static_cast<size_t>(i) * 4 + ((p ^ (c >> 1)) & 3)) * 16);
              s = __hfma2(*reinterpret_cast<const __half2*>(&h.x), wh[4 * p], s);
              s = __hfma2(*reinterpret_cast<const __half2*>(&h.y), wh[4 * p + 1], s);
              s = __hfma2(*reinterpret_cast<const __half2*>(&h.z), wh[4 * p + 2], s);
              s = __hfma2(*reinterpret_cast<const __half2*>(&h.w), wh[4 * p + 3], s);
            }
            const float2 f = __half22float2(s);
            part[q] = f.x + f.y;
          }
          if (kNv)
            acc[t] += part[0] * (xs[2 * i] * ws[0]) + part[1] * (xs[2 * i + 1] * ws[1]);
          else  // (the smaller scale first: the scales' product can leave fp32's range where the term does not,
                // and a sum times the smaller one is exact, being a multiple of 2^-129)
            acc[t] = fmaf((part[0] + part[1]) * min_nan(xs[i], ws[0]), max_nan(xs[i], ws[0]), acc[t]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < kT; ++t) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
      if (lane == 0 && t < nt) g.out[(t0 + t) * g.os0 + n * g.os1] = __float2bfloat16_rn(acc[t] * scale);
    }
  }
}

size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

template <typename K>
cudaError_t raise_smem(K kernel, size_t bytes, std::atomic<unsigned long long>& configured) {
  int dev = 0;
  cudaError_t rc = cudaGetDevice(&dev);
  if (rc != cudaSuccess) return rc;
  if (dev < 64 && (configured.load() & (1ull << dev))) return cudaSuccess;
  rc = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (rc == cudaSuccess && dev < 64) configured.fetch_or(1ull << dev);
  return rc;
}

constexpr size_t kRowsSmemMax = 160 << 10;

template <bool kNv, int kT>
cudaError_t launch_rows(const FpRows& r, int num_sms, cudaStream_t st) {
  static std::atomic<unsigned long long> configured{0};
  const size_t smem = static_cast<size_t>(kT) * r.groups * (64 + (kNv ? 8 : 4));
  cudaError_t rc = raise_smem(linear_fp4_rows_kernel<kNv, kT>, kRowsSmemMax, configured);
  if (rc != cudaSuccess) return rc;
  int64_t blocks = (r.N + kRowsThreads / 32 - 1) / (kRowsThreads / 32);
  if (blocks > 4 * num_sms) blocks = 4 * num_sms;
  return launch_pdl(linear_fp4_rows_kernel<kNv, kT>, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>((r.T + kT - 1) / kT)),
                    dim3(kRowsThreads), smem, st, r);
}

// Weight rows of a pair's tile: the width whose waves of tiles take the fewest steps.  A step
// costs the products (2 cycles a weight row on 256 tokens) or the loads of its 32 KB and more.
constexpr int kPairs = 74;
int tile_of(int64_t T, int64_t N) {
  const int64_t n_mt = (T + 2 * kTokRows - 1) / (2 * kTokRows);
  int best = kMaxTile;
  int64_t best_cost = INT64_MAX;
  for (int tile = kMaxTile; tile >= 32; tile -= 32) {
    const int64_t waves = (n_mt * ((N + tile - 1) / tile) + kPairs - 1) / kPairs;
    const int64_t step = 2 * tile > 256 + tile / 2 ? 2 * tile : 256 + tile / 2;
    if (waves * step < best_cost) {
      best_cost = waves * step;
      best = tile;
    }
  }
  return best;
}

}  // namespace

// By rows a call takes about 3 us and one for every 4.5 M weights times tokens; the pairs' two launches
// 5, one for every 900 of K and one for every 5 M weights, up to a few hundred tokens.  Measured by
// rows / on pairs: 4096 x 4096, 2 tokens 8.5 / 11.7 us; 512 x 4096, 16 tokens 9.4 / 9.4; 1024 x 2048, 16
// tokens 10.6 / 7.3; 256 x 512, 16 tokens 2.9 / 5.5.
bool linear_fp4_by_rows(int64_t T, int64_t N, int64_t K) {
  return T <= 16 && (T - 1) * N * K <= (8 << 20) + 5120 * K &&
         (T < 4 ? T : 4) * (K / 32) * 72 <= static_cast<int64_t>(kRowsSmemMax);
}

LinearFp4Plan linear_fp4_plan(int64_t T, int64_t N, int64_t K, bool nv) {
  LinearFp4Plan p = {};
  if (linear_fp4_by_rows(T, N, K)) return p;
  const int64_t atoms = nv ? 4 : 2;
  p.num_k = (K + kStepElems - 1) / kStepElems;
  p.ntile = tile_of(T, N);
  p.nh = p.ntile > 128 ? 2 : 1;
  p.n_mt = (T + 2 * kTokRows - 1) / (2 * kTokRows);
  p.n_nt = (N + p.ntile - 1) / p.ntile;
  p.x_atoms = p.n_mt * 2 * p.num_k * atoms;
  p.w_atoms = p.n_nt * p.num_k * atoms * p.nh;
  p.codes_off = 0;
  p.x_off = round256(static_cast<size_t>(T) * p.num_k * kRowBytes);
  p.w_off = p.x_off + static_cast<size_t>(p.x_atoms) * kAtomBytes;
  p.total = p.w_off + static_cast<size_t>(p.w_atoms) * kAtomBytes;
  return p;
}

cudaError_t launch_linear_fp4_rows(const LinearFp4& a, int num_sms, cudaStream_t st) {
  FpRows r = {};
  r.x = a.x;
  r.wide = a.wide;
  r.T = static_cast<int>(a.T);
  r.K = static_cast<int>(a.K);
  r.groups = static_cast<int>(a.K / 32);
  r.N = a.N;
  r.x_global = a.x_global;
  r.w_global = a.w_global;
  r.w = a.w;
  r.w_ld = a.w_ld;
  r.w_sf = a.w_sf;
  r.ws0 = a.ws0;
  r.ws1 = a.ws1;
  r.out = a.out;
  r.os0 = a.os0;
  r.os1 = a.os1;
  switch ((a.T < 4 ? a.T : 4) * 2 + (a.nv ? 1 : 0)) {
    case 2: return launch_rows<false, 1>(r, num_sms, st);
    case 3: return launch_rows<true, 1>(r, num_sms, st);
    case 4: return launch_rows<false, 2>(r, num_sms, st);
    case 5: return launch_rows<true, 2>(r, num_sms, st);
    case 6: return launch_rows<false, 3>(r, num_sms, st);
    case 7: return launch_rows<true, 3>(r, num_sms, st);
    case 8: return launch_rows<false, 4>(r, num_sms, st);
    case 9: return launch_rows<true, 4>(r, num_sms, st);
  }
  return cudaErrorInvalidValue;
}

namespace {
template <bool kNv>
cudaError_t launch_pair_path(const LinearFp4& a, const LinearFp4Plan& p, const CUtensorMap (&maps)[4], uint8_t* ws,
                             int num_sms, cudaStream_t st) {
  FpPrepare f = {};
  f.x = a.x;
  f.wide = a.wide;
  f.T = a.T;
  f.K = a.K;
  f.N = a.N;
  f.num_k = static_cast<int>(p.num_k);
  f.ntile = p.ntile;
  f.nh = p.nh;
  f.n_nt = p.n_nt;
  f.row_tiles = p.n_mt * 2 * kTokRows / 16;
  int64_t per_step = 4 * num_sms / p.num_k;  // resident blocks
  per_step = per_step < 1 ? 1 : per_step > f.row_tiles ? f.row_tiles : per_step;
  f.x_blocks = per_step * p.num_k;
  f.x_global = a.x_global;
  f.codes = ws + p.codes_off;
  f.x_atoms = ws + p.x_off;
  f.w_sf = a.w_sf;
  f.ws0 = a.ws0;
  f.ws1 = a.ws1;
  f.w_atoms = ws + p.w_off;
  const int64_t w_blocks = (p.n_nt * atoms_per_step<kNv>() * p.nh * 32 + 255) / 256 * p.num_k;
  const dim3 blocks(static_cast<unsigned>(f.x_blocks + w_blocks));
  cudaError_t rc = a.wide && a.x.dtype == MOE_BF16 ? launch_pdl(fp4_prepare_kernel<kNv, true>, blocks, dim3(256), 0, st, f)
                                                   : launch_pdl(fp4_prepare_kernel<kNv, false>, blocks, dim3(256), 0, st, f);
  if (rc != cudaSuccess) return rc;
  FpGemm g = {};
  g.T = a.T;
  g.N = a.N;
  g.total = p.n_mt * p.n_nt;
  g.num_k = static_cast<int>(p.num_k);
  g.ntile = p.ntile;
  g.nh = p.nh;
  g.n_mt = static_cast<int>(p.n_mt);
  g.x_global = a.x_global;
  g.w_global = a.w_global;
  g.out = a.out;
  g.os0 = a.os0;
  g.os1 = a.os1;
  g.vec_out = a.os1 == 1 && reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && a.os0 % 8 == 0;
  g.err = a.err;
  static std::atomic<unsigned long long> configured{0};
  rc = raise_smem(gemm_fp4_pair_kernel<kNv>, Cfg<kNv>::kSmem, configured);
  if (rc != cudaSuccess) return rc;
  int64_t pairs = g.total < num_sms / 2 ? g.total : num_sms / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<kNv>::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, gemm_fp4_pair_kernel<kNv>, maps[0], maps[1], maps[2], maps[3], g);
}
}  // namespace

cudaError_t launch_linear_fp4_pairs(const LinearFp4& a, const LinearFp4Plan& p, const CUtensorMap (&maps)[4],
                                    uint8_t* ws, int num_sms, cudaStream_t st) {
  return a.nv ? launch_pair_path<true>(a, p, maps, ws, num_sms, st)
              : launch_pair_path<false>(a, p, maps, ws, num_sms, st);
}

cudaError_t launch_quantize_nv(const RowView& x, bool wide, int64_t rows, int64_t K, const float* global,
                               uint8_t* codes, int64_t ld, uint8_t* sf, int64_t sf_ld, cudaStream_t st) {
  int64_t blocks = (rows * (K / 32) + 255) / 256;
  if (blocks > (1 << 20)) blocks = 1 << 20;
  const int code16 = reinterpret_cast<uintptr_t>(codes) % 16 == 0 && ld % 16 == 0;
  const int sf2 = reinterpret_cast<uintptr_t>(sf) % 2 == 0 && sf_ld % 2 == 0;
  return launch_pdl(quantize_nv_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, x, wide ? 1 : 0, rows, K,
                    global, codes, ld, sf, sf_ld, code16, sf2);
}

}  // namespace moe
