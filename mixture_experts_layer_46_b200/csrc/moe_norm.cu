// The RMS norms around a block and their gradients.
//
//   before:  xn  = x r w,                r = 1 / sqrt(mean(x^2) + eps)
//   after:   out = alpha x + a(g) y r w  (r of y; without normalize r = 1), and, on request,
//            the next block's norm of that sum in the same pass: nxt = out r' w'
// and, given dout, with yh = y r, d = dout a(g), p = d w:
//   after backward:   dy = r (p - yh mean(p yh)),  dw = sum_t d yh,
//                     dg = sum over the gate's broadcast axes of dout yh w a'(g)
//   before backward:  dx = alpha dres + r (p - xh mean(p xh)),  p = dxn w,  dw = sum_t dxn xh
//
// All four are bound by memory traffic: every row is read once into registers (8 * kVec
// elements a thread), reduced over the block in fp32, and written once.  Blocks walk over
// rows (grid = resident blocks), so the weight vectors come from L1 after the first row and
// the column sums of a gradient stay in registers until the block's last row; then each
// block writes one fp32 partial row, and a second launch adds the partial rows in a fixed
// order (no atomics: the same inputs give the same bits).
//
// Three ways to read share the code.  With inner stride 1, 16-byte aligned rows and H a
// multiple of 8 a thread takes 8 neighbours at a time: straight from memory where a block has
// one row, from a ring of rows in shared memory where it walks over several.  Otherwise it takes
// every blockDim-th element through the strides, which keeps a warp's accesses together.
// Arithmetic is fp32 throughout; each output is rounded once, to its own type.
//
// Measured, H=4096 bf16: before 49 us and after + next 92 us at T=16384, each alone from a cold cache
// (5.5 and 5.8 TB/s of the 6.5 that a copy gets; 139 us one after the other); the gradients 24 us each at
// T=4096 without their column sums.
#include <atomic>
#include <initializer_list>

#include "../../include/moe.h"
#include "moe_block.h"
#include "moe_gate.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

struct Vec8 {
  float v[8];
};

// Arithmetic on eight floats, two an instruction.
__device__ __forceinline__ uint64_t pair(const Vec8& a, int i) {
  return static_cast<uint64_t>(__float_as_uint(a.v[2 * i])) | (static_cast<uint64_t>(__float_as_uint(a.v[2 * i + 1])) << 32);
}
__device__ __forceinline__ uint64_t both(float f) {
  return static_cast<uint64_t>(__float_as_uint(f)) | (static_cast<uint64_t>(__float_as_uint(f)) << 32);
}
__device__ __forceinline__ void set_pair(Vec8& a, int i, uint64_t p) {
  a.v[2 * i] = __uint_as_float(static_cast<uint32_t>(p));
  a.v[2 * i + 1] = __uint_as_float(static_cast<uint32_t>(p >> 32));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// a *= f
__device__ __forceinline__ void scale8(Vec8& a, float f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) set_pair(a, i, mul2(pair(a, i), both(f)));
}
// a *= b
__device__ __forceinline__ void mul8(Vec8& a, const Vec8& b) {
#pragma unroll
  for (int i = 0; i < 4; ++i) set_pair(a, i, mul2(pair(a, i), pair(b, i)));
}
// a += f b
__device__ __forceinline__ void axpy8(Vec8& a, float f, const Vec8& b) {
#pragma unroll
  for (int i = 0; i < 4; ++i) set_pair(a, i, fma2(pair(b, i), both(f), pair(a, i)));
}
// acc (two floats) += a b
__device__ __forceinline__ void dot8(uint64_t& acc, const Vec8& a, const Vec8& b) {
#pragma unroll
  for (int i = 0; i < 4; ++i) acc = fma2(pair(a, i), pair(b, i), acc);
}
__device__ __forceinline__ float sum_of(uint64_t acc) {
  return __uint_as_float(static_cast<uint32_t>(acc)) + __uint_as_float(static_cast<uint32_t>(acc >> 32));
}

// How a kernel reads its row tensors: through the strides, 16 bytes a load, or from the ring.  The
// ring comes in three forms: any types, all bf16, and a float stream around a bf16 block; known
// types halve the instructions, which bound the ring otherwise (T=16384 H=4096 bf16, after + next:
// 37 a element with types as arguments).
enum { kStrided = 0, kWide = 1, kRing = 2, kRingBf16 = 3, kRingF32 = 4 };
constexpr bool is_ring(int mode) { return mode >= kRing; }
// the type of a tensor of the residual stream (x, out, their gradients), and of the block's (y, the
// normed rows, the gate)
template <int kMode>
__device__ __forceinline__ int32_t stream_type(const RowView& t) {
  return kMode == kRingBf16 ? MOE_BF16 : kMode == kRingF32 ? MOE_F32 : t.dtype;
}
template <int kMode>
__device__ __forceinline__ int32_t block_type(const RowView& t) {
  return kMode >= kRingBf16 ? MOE_BF16 : t.dtype;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Eight elements of one row: element i of slot v is column (tid + v * threads) * 8 + i (wide)
// or tid + (v * 8 + i) * threads.  Columns past H read as zero.
template <bool kWideCols>
__device__ __forceinline__ int col_of(int slot, int i) {
  return kWideCols ? (static_cast<int>(threadIdx.x) + slot * static_cast<int>(blockDim.x)) * 8 + i
                   : static_cast<int>(threadIdx.x) + (slot * 8 + i) * static_cast<int>(blockDim.x);
}

// Eight elements as they were read.  Loads and conversions are apart: a conversion next to its
// load, under the branch on the type, would make every load wait for the one before.
struct Raw8 {
  uint32_t w[8];
};

// eight neighbours at element c of a row that starts at `row` (16-byte aligned)
__device__ __forceinline__ void read8(const void* row, int c, int32_t dtype, Raw8& o) {
  if (dtype == MOE_F32) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(row) + c);
    const uint4 a = p[0], b = p[1];
    o.w[0] = a.x; o.w[1] = a.y; o.w[2] = a.z; o.w[3] = a.w;
    o.w[4] = b.x; o.w[5] = b.y; o.w[6] = b.z; o.w[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + c);
    o.w[0] = a.x; o.w[1] = a.y; o.w[2] = a.z; o.w[3] = a.w;
  }
}

__device__ __forceinline__ const char* row_ptr(const RowView& t, int64_t row, int32_t dtype) {
  return static_cast<const char*>(t.data) + row * t.s0 * (dtype == MOE_F32 ? 4 : 2);
}

__device__ __forceinline__ void zero8(Raw8& o) {
#pragma unroll
  for (int i = 0; i < 8; ++i) o.w[i] = 0u;
}

template <int kMode>
__device__ __forceinline__ void load8(const RowView& t, int64_t row, int slot, int H, Raw8& o) {
  const char* base = row_ptr(t, row, t.dtype);
  zero8(o);
  if (kMode != kStrided) {
    const int c = col_of<true>(slot, 0);
    if (c < H) read8(base, c, t.dtype, o);
  } else if (t.dtype == MOE_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = col_of<false>(slot, i);
      if (c < H) o.w[i] = reinterpret_cast<const uint32_t*>(base)[c * t.s1];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = col_of<false>(slot, i);
      if (c < H) o.w[i] = reinterpret_cast<const uint16_t*>(base)[c * t.s1];
    }
  }
}

template <int kMode>
__device__ __forceinline__ Vec8 unpack8(const Raw8& r, int32_t dtype) {
  Vec8 o;
  if (dtype == MOE_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] = __uint_as_float(r.w[i]);
  } else if (kMode != kStrided) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o.v[2 * i] = bf16_lo(r.w[i]);
      o.v[2 * i + 1] = bf16_hi(r.w[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] = bf16_lo(r.w[i]);
  }
  return o;
}

template <int kMode>
__device__ __forceinline__ void store8(const RowView& t, int32_t dtype, int64_t row, int slot, int H, const Vec8& o) {
  char* base = const_cast<char*>(row_ptr(t, row, dtype));
  if (kMode != kStrided) {
    const int c = col_of<true>(slot, 0);
    if (c >= H) return;
    if (dtype == MOE_F32) {
      float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + c);
      p[0] = make_float4(o.v[0], o.v[1], o.v[2], o.v[3]);
      p[1] = make_float4(o.v[4], o.v[5], o.v[6], o.v[7]);
    } else {
      *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(base) + c) =
          make_uint4(pack_bf16x2(o.v[0], o.v[1]), pack_bf16x2(o.v[2], o.v[3]),
                     pack_bf16x2(o.v[4], o.v[5]), pack_bf16x2(o.v[6], o.v[7]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = col_of<false>(slot, i);
      if (c >= H) continue;
      if (dtype == MOE_F32)
        reinterpret_cast<float*>(base)[c * t.s1] = o.v[i];
      else
        reinterpret_cast<__nv_bfloat16*>(base)[c * t.s1] = __float2bfloat16_rn(o.v[i]);
    }
  }
}

// The ring: a block's next rows on their way into shared memory by bulk copies (one copy a
// tensor and row, all of a stage on one mbarrier) while the current row is reduced, so that
// memory never waits for the two barriers of a reduction.
struct Ring {
  const RowRing& a;
  char* smem;
  uint64_t* full;
  uint32_t stage, phase;
  bool ok;

  __device__ __forceinline__ Ring(const RowRing& args, char* raw) : a(args) {
    full = reinterpret_cast<uint64_t*>(raw);
    smem = raw + 128;
    stage = 0;
    phase = 0;
    ok = true;
  }
  // thread 0: the copies of row t into stage s
  __device__ __forceinline__ void fill(int s, int64_t t) {
    mbar_arrive_expect_tx(&full[s], a.stage_bytes);
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (a.in[i].data)
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                smem_u32(smem + s * a.stage_bytes + a.off[i])),
            "l"(row_ptr(a.in[i], t, a.in[i].dtype)), "r"(a.bytes[i]), "r"(smem_u32(&full[s]))
            : "memory");
  }
  __device__ __forceinline__ void start(int64_t T) {
    if (threadIdx.x == 0) {
      for (int s = 0; s < a.stages; ++s) mbar_init(&full[s], 1);
      fence_barrier_init();
      fence_proxy_async_smem();
      for (int s = 0; s < a.stages; ++s) {
        const int64_t t = blockIdx.x + static_cast<int64_t>(s) * gridDim.x;
        if (t < T) fill(s, t);
      }
    }
    __syncthreads();
  }
  // waits (bounded) for the current stage
  __device__ __forceinline__ void wait() {
    if (ok && !mbar_wait(&full[stage], phase, threadIdx.x == 0 ? a.err : nullptr)) ok = false;
  }
  // Where a wait gave up, copies may still be on their way into the block's memory, so thread 0 lets them
  // land, again with a limit, before the block may leave: after the last row by finish() (of a
  // barrier's two parities one is its last completed phase's, which does not wait, the other the
  // phase's that a copy would complete), or at once by wait_landing(), which knows the stages filled
  // by the row.  The gradient of the norm after takes the second form, the other kernels the first:
  // the other way round the compiler orders their rows' loads worse (T=4096 H=4096 bf16, gradient after 30.5
  // instead of 26.2 us; T=16384 H=1024, gradient before 26.5 instead of 22.5).
  __device__ __forceinline__ void finish() {
    if (ok || threadIdx.x != 0) return;
    for (int i = 0; i < 2 * a.stages; ++i) mbar_wait(&full[i >> 1], i & 1, nullptr, kWaitLimitNs / 8);
  }
  __device__ __forceinline__ void wait_landing(int64_t t, int64_t T) {
    if (!ok || mbar_wait(&full[stage], phase, threadIdx.x == 0 ? a.err : nullptr)) return;
    ok = false;
    for (int s = 0; threadIdx.x == 0 && s < a.stages && t < T; ++s, t += gridDim.x)
      mbar_wait(&full[(stage + s) % a.stages], phase ^ (stage + s >= static_cast<uint32_t>(a.stages) ? 1u : 0u), nullptr);
  }
  __device__ __forceinline__ void read(int i, int32_t dtype, int slot, int H, Raw8& o) const {
    const int c = col_of<true>(slot, 0);
    zero8(o);
    if (c < H) read8(smem + stage * a.stage_bytes + a.off[i], c, dtype, o);
  }
  // every thread has read its part of row t: the stage takes the row `stages` rounds on
  __device__ __forceinline__ void next(int64_t t, int64_t T) {
    __syncthreads();
    const int64_t n = t + static_cast<int64_t>(a.stages) * gridDim.x;
    if (threadIdx.x == 0 && n < T && ok) fill(stage, n);
    if (++stage == static_cast<uint32_t>(a.stages)) { stage = 0; phase ^= 1u; }
  }
};

// row tensor i of the kernel: from the ring, or from memory
template <int kMode>
__device__ __forceinline__ void input8(const Ring& ring, int i, int32_t dtype, int64_t row, int slot, int H, Raw8& o) {
  if (is_ring(kMode))
    ring.read(i, dtype, slot, H, o);
  else
    load8<kMode>(ring.a.in[i], row, slot, H, o);
}

// a weight vector (or ones): element c at data[c * s1]
template <int kMode>
__device__ __forceinline__ Vec8 load_weight(const RowView& t, int slot, int H) {
  Vec8 o;
  if (t.data) {
    constexpr int kHow = kMode == kStrided ? kStrided : kWide;
    Raw8 r;
    load8<kHow>(t, 0, slot, H, r);
    o = unpack8<kHow>(r, t.dtype);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] = 1.0f;
  }
  return o;
}

__device__ __forceinline__ float scalar_at(const RowView& t, int64_t off) {
  return t.dtype == MOE_F32 ? static_cast<const float*>(t.data)[off]
                            : bf16_lo(static_cast<const uint16_t*>(t.data)[off]);
}

// the derivative of the gate's activation, from the gate's value
// (the slopes from e = exp(-|.|), which keeps their relative accuracy where the function is flat:
// sigmoid' = e / (1 + e)^2 with e = exp(-|g|), tanh' = 4 e / (1 + e)^2 with e = exp(-2 |g|))
__device__ __forceinline__ float gate_slope(float g, int act) {
  if (act == MOE_GATE_SIGMOID) {
    const float e = expf(-fabsf(g)), q = 1.0f / (1.0f + e);
    return e * q * q;
  }
  if (act == MOE_GATE_TANH) {
    const float e = expf(-2.0f * fabsf(g)), q = 1.0f / (1.0f + e);
    return 4.0f * e * q * q;
  }
  return 1.0f;
}

// the same on eight values, the choice of function outside the loop
__device__ __forceinline__ void gate_values(Vec8& g, int act) {
  if (act == MOE_GATE_NONE) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) g.v[i] = gate_value(g.v[i], act);
}
__device__ __forceinline__ void gate_slopes(Vec8& g, int act) {
#pragma unroll
  for (int i = 0; i < 8; ++i) g.v[i] = gate_slope(g.v[i], act);
}

// Sum of v over the block; every thread gets it.  One barrier a call: two scratch rows are
// used in turn, and a row is written again only after the other one's barrier.  (Up to eight
// warps every thread adds their sums itself: two broadcast loads and no second tree.)
template <int kMaxThreads>
__device__ __forceinline__ float block_sum(float v, float (*scratch)[32], int& turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  float* s = scratch[turn];
  turn ^= 1;
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  if (kMaxThreads <= 256) {
    const float4 a = *reinterpret_cast<const float4*>(s), b = *reinterpret_cast<const float4*>(s + 4);
    const float e[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    float r = e[0] + e[1];
#pragma unroll
    for (int i = 2; i < 8; ++i) r += i < warps ? e[i] : 0.0f;
    return r;
  }
  float r = static_cast<int>(threadIdx.x & 31) < warps ? s[threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
  return r;
}

// 1 / sqrt(sum / H + eps): the fast root (2 ulp) and one step of Newton's (a correctly rounded
// root and two divisions were a fifth of a row's instructions).  A zero, infinite or tiny argument
// keeps the fast root's value, which the step would turn into NaN.
__device__ __forceinline__ float inv_root(float sum, float inv_h, float eps) {
  const float a = fmaf(sum, inv_h, eps), y = rsqrtf(a);
  const float e = fmaf(-a * y, y, 1.0f);
  const float r = fmaf(0.5f * y, e, y);
  return a > 1e-30f && a < 1e30f ? r : y;
}

// Threads of resident blocks on an SM, and rows on their way in a block's ring.  More of either
// asks DRAM for too many streams at once: before + after + next at T=16384 H=4096, compared on one
// box, took 156 us with 768 threads and four rows, 134 with 512 and four, 132 with 512 and three, 146
// with two, 210 with 256.
constexpr int kResident = 512;
constexpr int64_t kRingBytes = 96 << 10;  // of an SM's blocks together
constexpr int min_blocks(int threads_per_sm, int max_threads) {
  return threads_per_sm / max_threads < 1 ? 1 : threads_per_sm / max_threads;
}

// ---------------------------------------------------------------- forward

template <int kVec, int kMode, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads, min_blocks(kResident, kMaxThreads))
    norm_before_kernel(const NormBefore g) {
  extern __shared__ __align__(128) char smem[];
  __shared__ __align__(16) float scratch[2][32];
  pdl_wait();
  pdl_launch_dependents();
  int turn = 0;
  const float inv_h = 1.0f / static_cast<float>(g.H);
  const int32_t xt = stream_type<kMode>(g.ring.in[0]);
  Ring ring(g.ring, smem);
  if (is_ring(kMode)) ring.start(g.T);
  Vec8 w[kVec];
#pragma unroll
  for (int v = 0; v < kVec; ++v) w[v] = load_weight<kMode>(g.w, v, g.H);
  for (int64_t t = blockIdx.x; t < g.T; t += gridDim.x) {
    if (is_ring(kMode)) ring.wait();
    Raw8 raw[kVec];
#pragma unroll
    for (int v = 0; v < kVec; ++v) input8<kMode>(ring, 0, xt, t, v, g.H, raw[v]);
    if (is_ring(kMode)) ring.next(t, g.T);
    Vec8 x[kVec];
    uint64_t ss = 0;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      x[v] = unpack8<kMode>(raw[v], xt);
      dot8(ss, x[v], x[v]);
    }
    const float r = inv_root(block_sum<kMaxThreads>(sum_of(ss), scratch, turn), inv_h, g.eps);
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      scale8(x[v], r);
      mul8(x[v], w[v]);
      store8<kMode>(g.out, block_type<kMode>(g.out), t, v, g.H, x[v]);
    }
    if (g.rstd && threadIdx.x == 0) g.rstd[t * g.rstd_s] = r;
  }
  if (is_ring(kMode)) ring.finish();
}

// One pass over (y, x, gate): out and, with a next norm, its output too.  The row of out is
// kept in registers unrounded between the two reductions, the weights (a per-channel gate
// multiplied in) for all of the block's rows.
template <int kVec, int kMode, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads, min_blocks(kResident, kMaxThreads))
    norm_after_kernel(const NormAfter g) {
  extern __shared__ __align__(128) char smem[];
  __shared__ __align__(16) float scratch[2][32];
  pdl_wait();
  pdl_launch_dependents();
  int turn = 0;
  const float inv_h = 1.0f / static_cast<float>(g.H);
  const int32_t yt = block_type<kMode>(g.ring.in[0]), xt = stream_type<kMode>(g.ring.in[1]), gtt = block_type<kMode>(g.ring.in[2]);
  Ring ring(g.ring, smem);
  if (is_ring(kMode)) ring.start(g.T);
  const bool have_x = g.ring.in[1].data != nullptr;
  const bool gate_full = g.ring.in[2].data != nullptr;
  const bool want_next = g.nxt.data || g.next_rstd;
  Vec8 w[kVec], wn[kVec];
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    w[v] = load_weight<kMode>(g.w, v, g.H);
    if (g.nxt.data) wn[v] = load_weight<kMode>(g.wn, v, g.H);
    if (g.gate_mode == kGateChannel) {
      Vec8 c = load_weight<kMode>(g.gate, v, g.H);
      gate_values(c, g.act);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[v].v[i] *= c.v[i];
    }
  }
  const bool gate_row = g.gate_mode == kGateToken || g.gate_mode == kGateOne;
  float gate_next = gate_row && blockIdx.x < g.T ? scalar_at(g.gate, blockIdx.x * g.gate.s0) : 0.0f;
  for (int64_t t = blockIdx.x; t < g.T; t += gridDim.x) {
    const float gate_now = gate_next;  // read a row ahead
    if (gate_row && t + gridDim.x < g.T) gate_next = scalar_at(g.gate, (t + gridDim.x) * g.gate.s0);
    if (is_ring(kMode)) ring.wait();
    Raw8 y[kVec], x[kVec], gt[kVec];
#pragma unroll
    for (int v = 0; v < kVec; ++v) input8<kMode>(ring, 0, yt, t, v, g.H, y[v]);
    if (!is_ring(kMode)) {  // (the ring's rows wait in shared memory until they are needed)
#pragma unroll
      for (int v = 0; v < kVec; ++v) {
        if (have_x) input8<kMode>(ring, 1, xt, t, v, g.H, x[v]);
        if (gate_full) input8<kMode>(ring, 2, gtt, t, v, g.H, gt[v]);
      }
    }
    // a gate of one number a row (or one in all) is part of the row's factor
    float f = 1.0f;
    if (gate_row) f = gate_value(gate_now, g.act);
    Vec8 o[kVec];
#pragma unroll
    for (int v = 0; v < kVec; ++v) o[v] = unpack8<kMode>(y[v], yt);
    float r = 1.0f;
    if (g.normalize) {
      uint64_t ss = 0;
#pragma unroll
      for (int v = 0; v < kVec; ++v) dot8(ss, o[v], o[v]);
      r = inv_root(block_sum<kMaxThreads>(sum_of(ss), scratch, turn), inv_h, g.eps);
    }
    if (g.rstd && threadIdx.x == 0) g.rstd[t * g.rstd_s] = r;
    f *= r;
    uint64_t ss = 0;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      scale8(o[v], f);
      mul8(o[v], w[v]);
      if (gate_full) {
        if (is_ring(kMode)) input8<kMode>(ring, 2, gtt, t, v, g.H, gt[v]);
        Vec8 c = unpack8<kMode>(gt[v], gtt);
        gate_values(c, g.act);
        mul8(o[v], c);
      }
      if (have_x) {
        if (is_ring(kMode)) input8<kMode>(ring, 1, xt, t, v, g.H, x[v]);
        const Vec8 c = unpack8<kMode>(x[v], xt);
        axpy8(o[v], g.alpha, c);
      }
      store8<kMode>(g.out, stream_type<kMode>(g.out), t, v, g.H, o[v]);
      dot8(ss, o[v], o[v]);
    }
    if (is_ring(kMode)) ring.next(t, g.T);
    if (want_next) {
      const float rn = inv_root(block_sum<kMaxThreads>(sum_of(ss), scratch, turn), inv_h, g.eps);
      if (g.next_rstd && threadIdx.x == 0) g.next_rstd[t * g.next_rstd_s] = rn;
      if (g.nxt.data) {
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
          scale8(o[v], rn);
          mul8(o[v], wn[v]);
          store8<kMode>(g.nxt, block_type<kMode>(g.nxt), t, v, g.H, o[v]);
        }
      }
    }
  }
  if (is_ring(kMode)) ring.finish();
}

// ---------------------------------------------------------------- backward

// Partial column sums of this block into row blockIdx.x of part [gridDim.x, H].
template <int kVec, int kMode>
__device__ __forceinline__ void store_partial(float* part, int H, const Vec8 (&acc)[kVec]) {
  RowView p;
  p.data = part;
  p.s0 = H;
  p.s1 = 1;
  p.dtype = MOE_F32;
#pragma unroll
  for (int v = 0; v < kVec; ++v) store8<kMode == kStrided ? kStrided : kWide>(p, MOE_F32, blockIdx.x, v, H, acc[v]);
}

template <int kVec, int kMode, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads, min_blocks(kResident, kMaxThreads))
    norm_before_backward_kernel(const NormBeforeBackward g) {
  extern __shared__ __align__(128) char smem[];
  __shared__ __align__(16) float scratch[2][32];
  pdl_wait();
  pdl_launch_dependents();
  int turn = 0;
  const float inv_h = 1.0f / static_cast<float>(g.H);
  const int32_t dt = block_type<kMode>(g.ring.in[0]), xt = stream_type<kMode>(g.ring.in[1]), rt = stream_type<kMode>(g.ring.in[2]);
  Ring ring(g.ring, smem);
  if (is_ring(kMode)) ring.start(g.T);
  const bool have_res = g.ring.in[2].data != nullptr;
  Vec8 dw[kVec], w[kVec];
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    w[v] = load_weight<kMode>(g.w, v, g.H);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[v].v[i] = 0.0f;
  }
  float r_next = blockIdx.x < g.T ? g.rstd[blockIdx.x * g.rstd_s] : 0.0f;
  for (int64_t t = blockIdx.x; t < g.T; t += gridDim.x) {
    const float r = r_next;
    if (t + gridDim.x < g.T) r_next = g.rstd[(t + gridDim.x) * g.rstd_s];
    if (is_ring(kMode)) ring.wait();
    Raw8 rd[kVec], rx[kVec], res[kVec];
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      input8<kMode>(ring, 0, dt, t, v, g.H, rd[v]);
      input8<kMode>(ring, 1, xt, t, v, g.H, rx[v]);
      if (!is_ring(kMode) && have_res) input8<kMode>(ring, 2, rt, t, v, g.H, res[v]);
    }
    Vec8 p[kVec], x[kVec];
    uint64_t dot = 0;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      p[v] = unpack8<kMode>(rd[v], dt);
      x[v] = unpack8<kMode>(rx[v], xt);
      scale8(x[v], r);
#pragma unroll
      for (int i = 0; i < 4; ++i) set_pair(dw[v], i, fma2(pair(p[v], i), pair(x[v], i), pair(dw[v], i)));
      mul8(p[v], w[v]);
      dot8(dot, p[v], x[v]);
    }
    const float c = block_sum<kMaxThreads>(sum_of(dot), scratch, turn) * inv_h;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      axpy8(p[v], -c, x[v]);
      scale8(p[v], r);
      if (have_res) {
        if (is_ring(kMode)) input8<kMode>(ring, 2, rt, t, v, g.H, res[v]);
        const Vec8 d = unpack8<kMode>(res[v], rt);
        axpy8(p[v], g.alpha, d);
      }
      store8<kMode>(g.dx, stream_type<kMode>(g.dx), t, v, g.H, p[v]);
    }
    if (is_ring(kMode)) ring.next(t, g.T);
  }
  if (g.part) store_partial<kVec, kMode>(g.part, g.H, dw);
  if (is_ring(kMode)) ring.finish();
}

template <int kVec, int kMode, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads, min_blocks(kResident, kMaxThreads))
    norm_after_backward_kernel(const NormAfterBackward g) {
  extern __shared__ __align__(128) char smem[];
  __shared__ __align__(16) float scratch[2][32];
  pdl_wait();
  pdl_launch_dependents();
  int turn = 0;
  const float inv_h = 1.0f / static_cast<float>(g.H);
  const int32_t dt = stream_type<kMode>(g.ring.in[0]), yt = block_type<kMode>(g.ring.in[1]), gtt = block_type<kMode>(g.ring.in[2]);
  Ring ring(g.ring, smem);
  if (is_ring(kMode)) ring.start(g.T);
  const bool gate_full = g.gate_mode == kGateFull;
  const bool gate_col = g.gate_mode == kGateChannel;
  const bool gate_row = g.gate_mode == kGateToken || g.gate_mode == kGateOne;
  Vec8 dw[kVec], w[kVec];  // w: the weight, a per-channel gate's value multiplied in
  float dall = 0.0f;       // one gate in all: this block's rows
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    w[v] = load_weight<kMode>(g.w, v, g.H);
    if (gate_col) {
      Vec8 c = load_weight<kMode>(g.gate, v, g.H);
      gate_values(c, g.act);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[v].v[i] *= c.v[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[v].v[i] = 0.0f;
  }
  // a row's numbers are read a row ahead
  float r_next = 1.0f, gate_next = 0.0f;
  auto fetch_row = [&](int64_t t) {
    if (t >= g.T) return;
    if (g.normalize) r_next = g.rstd[t * g.rstd_s];
    if (gate_row) gate_next = scalar_at(g.gate, t * g.gate.s0);
  };
  fetch_row(blockIdx.x);
  for (int64_t t = blockIdx.x; t < g.T; t += gridDim.x) {
    const float r = r_next, raw = gate_next;
    fetch_row(t + gridDim.x);
    float rowv = 1.0f, rowslope = 1.0f;
    if (gate_row) {
      rowv = gate_value(raw, g.act);
      rowslope = gate_slope(raw, g.act);
    }
    if (is_ring(kMode)) ring.wait_landing(t, g.T);
    Raw8 rd[kVec], ry[kVec], rg[kVec];
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      input8<kMode>(ring, 0, dt, t, v, g.H, rd[v]);
      input8<kMode>(ring, 1, yt, t, v, g.H, ry[v]);
      if (!is_ring(kMode) && gate_full) input8<kMode>(ring, 2, gtt, t, v, g.H, rg[v]);
    }
    Vec8 d[kVec], y[kVec];
    uint64_t dot = 0, gsum = 0;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      d[v] = unpack8<kMode>(rd[v], dt);
      y[v] = unpack8<kMode>(ry[v], yt);
      scale8(y[v], r);
      if (gate_full) {
        if (is_ring(kMode)) input8<kMode>(ring, 2, gtt, t, v, g.H, rg[v]);
        Vec8 c = unpack8<kMode>(rg[v], gtt);
        if (g.dgate.data) {
          Vec8 e = c;
          gate_slopes(e, g.act);
          mul8(e, d[v]);
          mul8(e, y[v]);
          mul8(e, w[v]);
          store8<kMode>(g.dgate, g.dgate.dtype, t, v, g.H, e);
        }
        gate_values(c, g.act);
        mul8(d[v], c);
      }
      // the column sum of dout yh: times a(g) it is dw, and for a gate that is the same in every
      // row of the column times w a'(g) it is dg, so one sum serves both there
      if (gate_row) {
        Vec8 e = d[v];
        mul8(e, y[v]);
        dot8(gsum, e, w[v]);
        scale8(d[v], rowv);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) set_pair(dw[v], i, fma2(pair(d[v], i), pair(y[v], i), pair(dw[v], i)));
      mul8(d[v], w[v]);
      dot8(dot, d[v], y[v]);
    }
    if (is_ring(kMode)) ring.next(t, g.T);
    float c = 0.0f;
    if (g.normalize) c = block_sum<kMaxThreads>(sum_of(dot), scratch, turn) * inv_h;
    if (gate_row && g.dgate.data) {
      const float s = block_sum<kMaxThreads>(sum_of(gsum), scratch, turn);
      if (g.gate_mode == kGateOne) {
        dall += s;
      } else if (threadIdx.x == 0) {
        const float o = s * rowslope;
        const int64_t off = t * g.dgate.s0;
        if (g.dgate.dtype == MOE_F32)
          static_cast<float*>(const_cast<void*>(g.dgate.data))[off] = o;
        else
          static_cast<__nv_bfloat16*>(const_cast<void*>(g.dgate.data))[off] = __float2bfloat16_rn(o);
      }
    }
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      if (!g.normalize) y[v] = Vec8();  // (dy does not depend on y, its infinities and NaNs included)
      axpy8(d[v], -c, y[v]);
      scale8(d[v], r);
      store8<kMode>(g.dy, block_type<kMode>(g.dy), t, v, g.H, d[v]);
    }
  }
  if (g.part) store_partial<kVec, kMode>(g.part, g.H, dw);
  if (g.part_gate && threadIdx.x == 0) g.part_gate[blockIdx.x] = dall;
}

// Adds up the partial rows, in row order within each of the strips (1024 / kCols) and then over the
// strips: dw[c] = a(g) sum (the gate is folded into the terms unless it is per channel), and for a
// per-channel gate dgate[c] = w a'(g) sum.  blockIdx.y = 1 sums the one-number gate's partials.
// Narrow matrices have few columns and many rows: 8 columns a block there (gradient of the norm
// before, T=16384 H=256: 22 -> 18 us).
__device__ __forceinline__ void store1(const RowView& t, int64_t off, float v) {
  if (t.dtype == MOE_F32)
    static_cast<float*>(const_cast<void*>(t.data))[off] = v;
  else
    static_cast<__nv_bfloat16*>(const_cast<void*>(t.data))[off] = __float2bfloat16_rn(v);
}
template <int kCols>
__global__ void __launch_bounds__(1024) column_sum_kernel(const ColumnSum g) {
  constexpr int kStrips = 1024 / kCols;
  __shared__ float acc[kStrips][kCols + 1];
  pdl_wait();
  pdl_launch_dependents();
  const bool one = blockIdx.y == 1;
  const float* part = one ? g.part_gate : g.part;
  const int n = one ? 1 : g.H;
  const int c = blockIdx.x * kCols + threadIdx.x;
  if (one && blockIdx.x != 0) return;
  float s = 0.0f;
  if (c < n && part)
    for (int base = threadIdx.y; base < g.rows; base += 10 * kStrips) {
      float v[10];  // (ten loads a trip to memory)
#pragma unroll
      for (int i = 0; i < 10; ++i) {
        const int row = base + i * kStrips;
        v[i] = row < g.rows ? part[static_cast<int64_t>(row) * n + c] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 10; ++i) s += v[i];
    }
  acc[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (kStrips > 32) {  // (two steps: 128 sums one after another take longer than the loads)
    if (threadIdx.y < 32) {
      s = acc[threadIdx.y][threadIdx.x];
#pragma unroll
      for (int i = 1; i < kStrips / 32; ++i) s += acc[threadIdx.y + 32 * i][threadIdx.x];
      acc[threadIdx.y][threadIdx.x] = s;
    }
    __syncthreads();
  }
  if (threadIdx.y != 0 || c >= n) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) s += acc[i][threadIdx.x];
  if (one) {
    store1(g.dgate, 0, s * gate_slope(scalar_at(g.gate, 0), g.act));
    return;
  }
  float a = 1.0f;
  if (g.gate_mode == kGateChannel) {
    const float raw = scalar_at(g.gate, c * g.gate.s1);
    a = gate_value(raw, g.act);
    if (g.dgate.data)
      store1(g.dgate, c * g.dgate.s1, s * gate_slope(raw, g.act) * (g.w.data ? scalar_at(g.w, c * g.w.s1) : 1.0f));
  }
  if (g.dw.data) store1(g.dw, c * g.dw.s1, s * a);
}

// ---------------------------------------------------------------- launch

// Threads and 8-element slots of a block that holds one row of H elements.
struct Shape {
  int vec, threads;
};
Shape shape_of(int64_t H, bool wide) {
  const int n = static_cast<int>((H + 7) / 8);
  // (two slots halve what a row costs besides its elements: T=16384 H=1024 after + next 41 -> 33 us;
  // through the strides, where an element is a load, one is faster: 1023 x 1407 f32 16 against 20)
  // Rows of more than 8192 take four on 512 threads.  That spills too (per thread, from the ring: none before
  // and after, 60 bytes in the gradient before, 260 to 380 in the one after; up to 700 where two rows fit no
  // ring), but less than two on 1024, with 64 registers: T=4096 H=16384 after + next 129 against 100 us.
  // At H=4096 four are slower (92 against 104).
  const int vec = n <= (wide ? 64 : 256) ? 1 : wide && n > 1024 ? 4 : 2;
  Shape s;
  s.vec = vec;
  s.threads = ((n + vec - 1) / vec + 31) / 32 * 32;
  return s;
}

int64_t blocks_of(int64_t T, int threads, int num_sms, int threads_per_sm) {
  int per = threads_per_sm / threads;
  if (per < 1) per = 1;
  if (per > 16) per = 16;
  const int64_t g = static_cast<int64_t>(num_sms) * per;
  return T < g ? T : g;
}

// The ring of a wide call in which blocks walk over several rows: as many stages (two to eight) as
// fit kRingBytes on an SM of `per_sm` blocks; none where two rows do not fit its 220 KB.
int ring_of(RowRing* r, int H, int64_t T, int64_t grid, int per_sm) {
  r->stage_bytes = 0;
  for (int i = 0; i < 3; ++i) {
    if (!r->in[i].data) continue;
    r->off[i] = r->stage_bytes;
    r->bytes[i] = static_cast<uint32_t>(H) * (r->in[i].dtype == MOE_F32 ? 4u : 2u);
    r->stage_bytes += r->bytes[i];
  }
  const int64_t room = (220 << 10) / per_sm - 1024 - 128;
  int64_t n = room / r->stage_bytes;
  const int64_t want = kRingBytes / (per_sm * r->stage_bytes);
  if (n > want && n > 2) n = want < 2 ? 2 : want;
  if (n > 8) n = 8;
  const int64_t rows = (T + grid - 1) / grid;
  if (n > rows) n = rows;
  r->stages = static_cast<int>(n);
  return rows > 1 && n >= 2 ? 128 + r->stages * static_cast<int>(r->stage_bytes) : 0;
}

template <auto kKernel, typename Args>
cudaError_t launch_rows(const Args& g, int threads, int64_t grid, int smem, cudaStream_t st) {
  if (smem > 0) {  // (the 48 KB that need no raised limit hold the kernel's own shared memory too)
    static std::atomic<unsigned long long> configured{0};  // devices whose limit is raised already
    int dev = 0;
    cudaError_t rc = cudaGetDevice(&dev);
    if (rc != cudaSuccess) return rc;
    if (dev >= 64 || !(configured.load() & (1ull << dev))) {
      rc = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 << 10);
      if (rc != cudaSuccess) return rc;
      if (dev < 64) configured.fetch_or(1ull << dev);
    }
  }
  return launch_pdl(kKernel, dim3(static_cast<unsigned>(grid)), dim3(static_cast<unsigned>(threads)), smem, st, g);
}

// Launches K<slots, mode, threads bound> for a row of H elements.
#define MOE_NORM_WIDE(K, M, g, s, grid, smem, st)                                                     \
  ((s).vec == 1         ? launch_rows<K<1, M, 256>>(g, (s).threads, grid, smem, st)                   \
   : (s).vec == 4       ? launch_rows<K<4, M, 512>>(g, (s).threads, grid, smem, st)                   \
   : (s).threads <= 256 ? launch_rows<K<2, M, 256>>(g, (s).threads, grid, smem, st)                   \
                        : launch_rows<K<2, M, 512>>(g, (s).threads, grid, smem, st))
#define MOE_NORM_STRIDED(K, g, s, grid, st)                                                           \
  ((s).vec == 1         ? launch_rows<K<1, kStrided, 256>>(g, (s).threads, grid, 0, st)               \
   : (s).threads <= 256 ? launch_rows<K<2, kStrided, 256>>(g, (s).threads, grid, 0, st)               \
   : (s).threads <= 512 ? launch_rows<K<2, kStrided, 512>>(g, (s).threads, grid, 0, st)               \
                        : launch_rows<K<2, kStrided, 1024>>(g, (s).threads, grid, 0, st))
#define MOE_NORM_LAUNCH(K, g, mode, s, grid, smem, st)                                                \
  ((mode) == kStrided    ? MOE_NORM_STRIDED(K, g, s, grid, st)                                        \
   : (mode) == kWide     ? MOE_NORM_WIDE(K, kWide, g, s, grid, 0, st)                                 \
   : (mode) == kRingBf16 ? MOE_NORM_WIDE(K, kRingBf16, g, s, grid, smem, st)                          \
   : (mode) == kRingF32  ? MOE_NORM_WIDE(K, kRingF32, g, s, grid, smem, st)                           \
                         : MOE_NORM_WIDE(K, kRing, g, s, grid, smem, st))

// the ring's form from the types of the stream's and the block's tensors (absent ones do not count)
int mode_of(bool wide, int smem, std::initializer_list<const RowView*> stream, std::initializer_list<const RowView*> block) {
  if (!wide) return kStrided;
  if (smem == 0) return kWide;
  bool b16 = true, f32 = true;
  for (const RowView* v : stream)
    if (v->data) (v->dtype == MOE_F32 ? b16 : f32) = false;
  for (const RowView* v : block)
    if (v->data && v->dtype != MOE_BF16) b16 = f32 = false;
  return b16 ? kRingBf16 : f32 ? kRingF32 : kRing;
}

template <typename Args>
int prepare(Args* g, const Shape& s, bool wide, int threads_per_sm, int64_t grid) {
  const int per = threads_per_sm / s.threads < 1 ? 1 : threads_per_sm / s.threads > 16 ? 16 : threads_per_sm / s.threads;
  return wide ? ring_of(&g->ring, g->H, g->T, grid, per) : 0;
}

}  // namespace

int64_t norm_backward_rows(int64_t T, int64_t H, bool wide, int num_sms) {
  return blocks_of(T, shape_of(H, wide).threads, num_sms < kNormMaxSms ? num_sms : kNormMaxSms, kResident);
}

cudaError_t launch_norm_before(NormBefore g, bool wide, int num_sms, cudaStream_t st) {
  const Shape s = shape_of(g.H, wide);
  const int64_t grid = blocks_of(g.T, s.threads, num_sms, kResident);
  const int smem = prepare(&g, s, wide, kResident, grid);
  const int mode = mode_of(wide, smem, {&g.ring.in[0]}, {&g.out});
  return MOE_NORM_LAUNCH(norm_before_kernel, g, mode, s, grid, smem, st);
}

cudaError_t launch_norm_after(NormAfter g, bool wide, int num_sms, cudaStream_t st) {
  const Shape s = shape_of(g.H, wide);
  const int64_t grid = blocks_of(g.T, s.threads, num_sms, kResident);
  const int smem = prepare(&g, s, wide, kResident, grid);
  const int mode = mode_of(wide, smem, {&g.ring.in[1], &g.out}, {&g.ring.in[0], &g.ring.in[2], &g.nxt});
  return MOE_NORM_LAUNCH(norm_after_kernel, g, mode, s, grid, smem, st);
}

cudaError_t launch_norm_before_backward(NormBeforeBackward g, bool wide, int num_sms, cudaStream_t st) {
  const Shape s = shape_of(g.H, wide);
  const int64_t grid = norm_backward_rows(g.T, g.H, wide, num_sms);
  const int smem = prepare(&g, s, wide, kResident, grid);
  const int mode = mode_of(wide, smem, {&g.ring.in[1], &g.ring.in[2], &g.dx}, {&g.ring.in[0]});
  return MOE_NORM_LAUNCH(norm_before_backward_kernel, g, mode, s, grid, smem, st);
}

cudaError_t launch_norm_after_backward(NormAfterBackward g, bool wide, int num_sms, cudaStream_t st) {
  const Shape s = shape_of(g.H, wide);
  const int64_t grid = norm_backward_rows(g.T, g.H, wide, num_sms);
  const int smem = prepare(&g, s, wide, kResident, grid);
  const int mode = mode_of(wide, smem, {&g.ring.in[0]}, {&g.ring.in[1], &g.ring.in[2], &g.dy});
  return MOE_NORM_LAUNCH(norm_after_backward_kernel, g, mode, s, grid, smem, st);
}

cudaError_t launch_column_sum(const ColumnSum& g, cudaStream_t st) {
  const unsigned y = g.part_gate ? 2 : 1;
  if (g.H <= 1024)
    return launch_pdl(column_sum_kernel<8>, dim3(static_cast<unsigned>((g.H + 7) / 8), y), dim3(8, 128), 0, st, g);
  return launch_pdl(column_sum_kernel<32>, dim3(static_cast<unsigned>((g.H + 31) / 32), y), dim3(32, 32), 0, st, g);
}

}  // namespace moe
