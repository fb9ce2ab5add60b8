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
// Two element layouts share the code: kWide reads 8 neighbours a thread with 16-byte loads
// (inner stride 1, 16-byte aligned rows, H a multiple of 8); otherwise a thread takes every
// blockDim-th element through the strides, which keeps a warp's accesses together.
// Arithmetic is fp32 throughout; each output is rounded once, to its own type.
#include "../../include/moe.h"
#include "moe_block.h"
#include "moe_internal.h"

namespace moe {
namespace {

struct Vec8 {
  float v[8];
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Eight elements of one row: element i of slot v is column (tid + v * threads) * 8 + i (wide)
// or tid + (v * 8 + i) * threads.  Columns past H read as zero.
template <bool kWide>
__device__ __forceinline__ int col_of(int slot, int i) {
  return kWide ? (static_cast<int>(threadIdx.x) + slot * static_cast<int>(blockDim.x)) * 8 + i
               : static_cast<int>(threadIdx.x) + (slot * 8 + i) * static_cast<int>(blockDim.x);
}

template <bool kWide>
__device__ __forceinline__ void load8(const RowView& t, int64_t row, int slot, int H, Vec8& o) {
  const int64_t base = row * t.s0;
  if (kWide) {
    const int c = col_of<true>(slot, 0);
    if (c >= H) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o.v[i] = 0.0f;
      return;
    }
    if (t.dtype == MOE_F32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(t.data) + base + c);
      const float4 a = p[0], b = p[1];
      o.v[0] = a.x; o.v[1] = a.y; o.v[2] = a.z; o.v[3] = a.w;
      o.v[4] = b.x; o.v[5] = b.y; o.v[6] = b.z; o.v[7] = b.w;
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(t.data) + base + c);
      o.v[0] = bf16_lo(a.x); o.v[1] = bf16_hi(a.x); o.v[2] = bf16_lo(a.y); o.v[3] = bf16_hi(a.y);
      o.v[4] = bf16_lo(a.z); o.v[5] = bf16_hi(a.z); o.v[6] = bf16_lo(a.w); o.v[7] = bf16_hi(a.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = col_of<false>(slot, i);
      float f = 0.0f;
      if (c < H) {
        const int64_t off = base + c * t.s1;
        f = t.dtype == MOE_F32 ? static_cast<const float*>(t.data)[off]
                               : bf16_lo(static_cast<const uint16_t*>(t.data)[off]);
      }
      o.v[i] = f;
    }
  }
}

template <bool kWide>
__device__ __forceinline__ void store8(const RowView& t, int64_t row, int slot, int H, const Vec8& o) {
  const int64_t base = row * t.s0;
  void* data = const_cast<void*>(t.data);
  if (kWide) {
    const int c = col_of<true>(slot, 0);
    if (c >= H) return;
    if (t.dtype == MOE_F32) {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(data) + base + c);
      p[0] = make_float4(o.v[0], o.v[1], o.v[2], o.v[3]);
      p[1] = make_float4(o.v[4], o.v[5], o.v[6], o.v[7]);
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(data) + base + c) =
          make_uint4(pack_bf16x2(o.v[0], o.v[1]), pack_bf16x2(o.v[2], o.v[3]),
                     pack_bf16x2(o.v[4], o.v[5]), pack_bf16x2(o.v[6], o.v[7]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = col_of<false>(slot, i);
      if (c >= H) continue;
      const int64_t off = base + c * t.s1;
      if (t.dtype == MOE_F32)
        static_cast<float*>(data)[off] = o.v[i];
      else
        static_cast<__nv_bfloat16*>(data)[off] = __float2bfloat16_rn(o.v[i]);
    }
  }
}

// a weight vector (or ones): element c at data[c * s1]
template <bool kWide>
__device__ __forceinline__ void load_weight(const RowView& t, int slot, int H, Vec8& o) {
  if (t.data) {
    load8<kWide>(t, 0, slot, H, o);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] = 1.0f;
  }
}

__device__ __forceinline__ float scalar_at(const RowView& t, int64_t off) {
  return t.dtype == MOE_F32 ? static_cast<const float*>(t.data)[off]
                            : bf16_lo(static_cast<const uint16_t*>(t.data)[off]);
}

// the gate's activation and its derivative, from the gate's value
__device__ __forceinline__ float gate_value(float g, int act) {
  if (act == MOE_GATE_SIGMOID) return 1.0f / (1.0f + expf(-g));
  if (act == MOE_GATE_TANH) return tanhf(g);
  return g;
}
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

// Sum of v over the block; every thread gets it.  One barrier a call: two scratch rows are
// used in turn, and a row is written again only after the other one's barrier.
__device__ __forceinline__ float block_sum(float v, float (*scratch)[32], int& turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  float* s = scratch[turn];
  turn ^= 1;
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = static_cast<int>(threadIdx.x & 31) < warps ? s[threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
  return r;
}

__device__ __forceinline__ float inv_root(float sum, int H, float eps) {
  return 1.0f / sqrtf(sum / static_cast<float>(H) + eps);
}

// ---------------------------------------------------------------- forward

template <int kVec, bool kWide, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads) norm_before_kernel(const NormBefore g) {
  __shared__ float scratch[2][32];
  pdl_wait();
  pdl_launch_dependents();
  int turn = 0;
  for (int64_t t = blockIdx.x; t < g.T; t += gridDim.x) {
    Vec8 x[kVec];
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < kVec; ++v) load8<kWide>(g.x, t, v, g.H, x[v]);
#pragma unroll
    for (int v = 0; v < kVec; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += x[v].v[i] * x[v].v[i];
    const float r = inv_root(block_sum(ss, scratch, turn), g.H, g.eps);
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      Vec8 w;
      load_weight<kWide>(g.w, v, g.H, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) w.v[i] *= x[v].v[i] * r;
      store8<kWide>(g.out, t, v, g.H, w);
    }
    if (g.rstd && threadIdx.x == 0) g.rstd[t * g.rstd_s] = r;
  }
}

// One pass over (y, x, gate): out and, with a next norm, its output too.  The row of out is
// kept in registers unrounded between the two reductions.
template <int kVec, bool kWide, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads) norm_after_kernel(const NormAfter g) {
  __shared__ float scratch[2][32];
  pdl_wait();
  pdl_launch_dependents();
  int turn = 0;
  for (int64_t t = blockIdx.x; t < g.T; t += gridDim.x) {
    Vec8 o[kVec], x[kVec];
#pragma unroll
    for (int v = 0; v < kVec; ++v) load8<kWide>(g.y, t, v, g.H, o[v]);
    if (g.x.data) {
#pragma unroll
      for (int v = 0; v < kVec; ++v) load8<kWide>(g.x, t, v, g.H, x[v]);
    }
    float r = 1.0f;
    if (g.normalize) {
      float ss = 0.0f;
#pragma unroll
      for (int v = 0; v < kVec; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += o[v].v[i] * o[v].v[i];
      r = inv_root(block_sum(ss, scratch, turn), g.H, g.eps);
    }
    if (g.rstd && threadIdx.x == 0) g.rstd[t * g.rstd_s] = r;
    // a gate of one number a row (or one in all) is part of the row's factor
    float rowg = 1.0f;
    if (g.gate.data && g.gate_one_col) rowg = gate_value(scalar_at(g.gate, t * g.gate.s0), g.act);
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      Vec8 w;
      load_weight<kWide>(g.w, v, g.H, w);
      if (g.gate.data && !g.gate_one_col) {
        Vec8 gt;
        load8<kWide>(g.gate, t, v, g.H, gt);
#pragma unroll
        for (int i = 0; i < 8; ++i) w.v[i] *= gate_value(gt.v[i], g.act);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w.v[i] *= rowg;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float z = o[v].v[i] * r * w.v[i];
        if (g.x.data) z += g.alpha * x[v].v[i];
        o[v].v[i] = z;
        ss += z * z;
      }
      store8<kWide>(g.out, t, v, g.H, o[v]);
    }
    if (g.nxt.data || g.next_rstd) {
      const float rn = inv_root(block_sum(ss, scratch, turn), g.H, g.eps);
      if (g.next_rstd && threadIdx.x == 0) g.next_rstd[t * g.next_rstd_s] = rn;
      if (g.nxt.data) {
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
          Vec8 w;
          load_weight<kWide>(g.wn, v, g.H, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) w.v[i] *= o[v].v[i] * rn;
          store8<kWide>(g.nxt, t, v, g.H, w);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- backward

// Partial column sums of this block into row blockIdx.x of part [gridDim.x, H].
template <int kVec, bool kWide>
__device__ __forceinline__ void store_partial(float* part, int H, const Vec8 (&acc)[kVec]) {
  RowView p;
  p.data = part;
  p.s0 = H;
  p.s1 = 1;
  p.dtype = MOE_F32;
#pragma unroll
  for (int v = 0; v < kVec; ++v) store8<kWide>(p, blockIdx.x, v, H, acc[v]);
}

template <int kVec, bool kWide, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads) norm_before_backward_kernel(const NormBeforeBackward g) {
  __shared__ float scratch[2][32];
  pdl_wait();
  pdl_launch_dependents();
  int turn = 0;
  Vec8 dw[kVec];
#pragma unroll
  for (int v = 0; v < kVec; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[v].v[i] = 0.0f;
  for (int64_t t = blockIdx.x; t < g.T; t += gridDim.x) {
    Vec8 p[kVec], x[kVec], d[kVec];
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      load8<kWide>(g.dout, t, v, g.H, p[v]);
      load8<kWide>(g.x, t, v, g.H, x[v]);
      if (g.dres.data) load8<kWide>(g.dres, t, v, g.H, d[v]);
    }
    const float r = g.rstd[t * g.rstd_s];
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      Vec8 w;
      load_weight<kWide>(g.w, v, g.H, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[v].v[i] *= r;
        dw[v].v[i] += p[v].v[i] * x[v].v[i];
        p[v].v[i] *= w.v[i];
        dot += p[v].v[i] * x[v].v[i];
      }
    }
    const float c = block_sum(dot, scratch, turn) / static_cast<float>(g.H);
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float z = r * (p[v].v[i] - x[v].v[i] * c);
        if (g.dres.data) z += g.alpha * d[v].v[i];
        p[v].v[i] = z;
      }
      store8<kWide>(g.dx, t, v, g.H, p[v]);
    }
  }
  if (g.part) store_partial<kVec, kWide>(g.part, g.H, dw);
}

template <int kVec, bool kWide, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads) norm_after_backward_kernel(const NormAfterBackward g) {
  __shared__ float scratch[2][32];
  pdl_wait();
  pdl_launch_dependents();
  int turn = 0;
  const bool gate_full = g.gate_mode == kGateFull;
  const bool gate_col = g.gate_mode == kGateChannel;
  const bool gate_row = g.gate_mode == kGateToken || g.gate_mode == kGateOne;
  Vec8 dw[kVec], dc[kVec];
  float dall = 0.0f;  // one gate in all: this block's rows
#pragma unroll
  for (int v = 0; v < kVec; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[v].v[i] = dc[v].v[i] = 0.0f;
  for (int64_t t = blockIdx.x; t < g.T; t += gridDim.x) {
    Vec8 d[kVec], y[kVec];
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      load8<kWide>(g.dout, t, v, g.H, d[v]);
      load8<kWide>(g.y, t, v, g.H, y[v]);
    }
    const float r = g.normalize ? g.rstd[t * g.rstd_s] : 1.0f;
    float rowv = 1.0f, rowslope = 1.0f;
    if (gate_row) {
      const float raw = scalar_at(g.gate, t * g.gate.s0);
      rowv = gate_value(raw, g.act);
      rowslope = gate_slope(raw, g.act);
    }
    float dot = 0.0f, gsum = 0.0f;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      Vec8 w, gt;
      load_weight<kWide>(g.w, v, g.H, w);
      if (gate_full || gate_col) load8<kWide>(g.gate, t, v, g.H, gt);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float yh = y[v].v[i] * r;
        const float dy0 = d[v].v[i] * yh;  // dout yh
        float a = rowv;
        if (gate_full || gate_col) {
          a = gate_value(gt.v[i], g.act);
          if (gate_full)
            gt.v[i] = dy0 * w.v[i] * gate_slope(gt.v[i], g.act);
          else
            dc[v].v[i] += dy0;  // w a'(g) of a column is the same in every row: applied at the end
        } else {
          gsum += dy0 * w.v[i];
        }
        y[v].v[i] = yh;
        dw[v].v[i] += a * dy0;
        d[v].v[i] *= a * w.v[i];
        dot += d[v].v[i] * yh;
      }
      if (gate_full && g.dgate.data) store8<kWide>(g.dgate, t, v, g.H, gt);
    }
    float c = 0.0f;
    if (g.normalize) c = block_sum(dot, scratch, turn) / static_cast<float>(g.H);
    if (gate_row && g.dgate.data) {
      const float s = block_sum(gsum, scratch, turn);
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
#pragma unroll
      for (int i = 0; i < 8; ++i) y[v].v[i] = r * (d[v].v[i] - y[v].v[i] * c);
      store8<kWide>(g.dy, t, v, g.H, y[v]);
    }
  }
  if (g.part) store_partial<kVec, kWide>(g.part, g.H, dw);
  if (g.part_gate) {
    if (gate_col)
      store_partial<kVec, kWide>(g.part_gate, g.H, dc);
    else if (threadIdx.x == 0)
      g.part_gate[blockIdx.x] = dall;
  }
}

// out[c] = sum of the partial rows, in row order within each of 32 strips and then over the
// strips; for a per-channel gate times w a'(g).  blockIdx.y = 0: dw, 1: the gate's sum.
constexpr int kStrips = 32;
__global__ void __launch_bounds__(32 * kStrips) column_sum_kernel(const ColumnSum g) {
  __shared__ float acc[kStrips][33];
  pdl_wait();
  pdl_launch_dependents();
  const bool gate = blockIdx.y == 1;
  const float* part = gate ? g.part_gate : g.part;
  if (!part) return;
  const RowView& out = gate ? g.dgate : g.dw;
  const int n = gate && g.gate_mode == kGateOne ? 1 : g.H;
  const int c = blockIdx.x * 32 + threadIdx.x;
  float s = 0.0f;
  if (c < n)
    for (int row = threadIdx.y; row < g.rows; row += kStrips) s += part[static_cast<int64_t>(row) * n + c];
  acc[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y != 0 || c >= n) return;
  s = 0.0f;
  for (int i = 0; i < kStrips; ++i) s += acc[i][threadIdx.x];
  if (gate) {
    const float raw = scalar_at(g.gate, g.gate_mode == kGateOne ? 0 : c * g.gate.s1);
    s *= gate_slope(raw, g.act);
    if (g.gate_mode == kGateChannel && g.w.data) s *= scalar_at(g.w, c * g.w.s1);
  }
  const int64_t off = c * out.s1;
  if (out.dtype == MOE_F32)
    static_cast<float*>(const_cast<void*>(out.data))[off] = s;
  else
    static_cast<__nv_bfloat16*>(const_cast<void*>(out.data))[off] = __float2bfloat16_rn(s);
}

// ---------------------------------------------------------------- launch

// Threads and 8-element slots of a block that holds one row of H elements.
struct Shape {
  int vec, threads;
};
Shape shape_of(int64_t H) {
  const int n = static_cast<int>((H + 7) / 8);
  const int vec = n <= 256 ? 1 : 2;
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

// Launches K<kVec, kWide, threads bound> for the row shape.
#define MOE_NORM_LAUNCH(K, g, wide, s, grid, st)                                                              \
  [&]() -> cudaError_t {                                                                                      \
    const dim3 gr(static_cast<unsigned>(grid)), bl(static_cast<unsigned>((s).threads));                       \
    if ((s).vec == 1) return (wide) ? launch_pdl(K<1, true, 256>, gr, bl, 0, st, g)                           \
                                    : launch_pdl(K<1, false, 256>, gr, bl, 0, st, g);                         \
    if ((s).threads <= 256) return (wide) ? launch_pdl(K<2, true, 256>, gr, bl, 0, st, g)                     \
                                          : launch_pdl(K<2, false, 256>, gr, bl, 0, st, g);                   \
    if ((s).threads <= 512) return (wide) ? launch_pdl(K<2, true, 512>, gr, bl, 0, st, g)                     \
                                          : launch_pdl(K<2, false, 512>, gr, bl, 0, st, g);                   \
    return (wide) ? launch_pdl(K<2, true, 1024>, gr, bl, 0, st, g)                                            \
                  : launch_pdl(K<2, false, 1024>, gr, bl, 0, st, g);                                          \
  }()

}  // namespace

int64_t norm_backward_rows(int64_t T, int64_t H, int num_sms) {
  return blocks_of(T, shape_of(H).threads, num_sms < kNormMaxSms ? num_sms : kNormMaxSms, 512);
}

cudaError_t launch_norm_before(const NormBefore& g, bool wide, int num_sms, cudaStream_t st) {
  const Shape s = shape_of(g.H);
  return MOE_NORM_LAUNCH(norm_before_kernel, g, wide, s, blocks_of(g.T, s.threads, num_sms, 2048), st);
}

cudaError_t launch_norm_after(const NormAfter& g, bool wide, int num_sms, cudaStream_t st) {
  const Shape s = shape_of(g.H);
  return MOE_NORM_LAUNCH(norm_after_kernel, g, wide, s, blocks_of(g.T, s.threads, num_sms, 2048), st);
}

cudaError_t launch_norm_before_backward(const NormBeforeBackward& g, bool wide, int num_sms, cudaStream_t st) {
  const Shape s = shape_of(g.H);
  return MOE_NORM_LAUNCH(norm_before_backward_kernel, g, wide, s, norm_backward_rows(g.T, g.H, num_sms), st);
}

cudaError_t launch_norm_after_backward(const NormAfterBackward& g, bool wide, int num_sms, cudaStream_t st) {
  const Shape s = shape_of(g.H);
  return MOE_NORM_LAUNCH(norm_after_backward_kernel, g, wide, s, norm_backward_rows(g.T, g.H, num_sms), st);
}

cudaError_t launch_column_sum(const ColumnSum& g, cudaStream_t st) {
  return launch_pdl(column_sum_kernel, dim3(static_cast<unsigned>((g.H + 31) / 32), g.part_gate ? 2 : 1),
                    dim3(32, kStrips), 0, st, g);
}

}  // namespace moe
