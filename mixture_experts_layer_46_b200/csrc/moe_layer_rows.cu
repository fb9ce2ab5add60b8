// The experts of a layer for a few tokens, bf16 weights: two kernels over the rows of the
// routed experts' matrices, each weight read once from memory and used from registers.
//
//   1. h[s, i] = silu(gate[e_s][i] . xn_t) (up[e_s][i] . xn_t)      s = slot (token t, column j)
//   2. out[t, o] = finish(sum_s w_s w2[e_s][o] . h[s])
//
// At these sizes a weight meets one or two tokens, so the work is the read of the weights (about
// 38 MB an expert of the Qwen3-235B shape) and fp32 multiply-adds keep up with it: a warp holds
// its 512 columns of xn (or h) in registers and takes row after row of its columns, with several
// rows' 16-byte loads in flight (64 to 128 KB a SM); the warps' sums meet in shared memory in a
// fixed order.  Tensor-core tiles stream the same bytes through shared memory with a hand-off for
// every tile; they are left to more tokens.  The second kernel starts while the first one's last
// blocks run and requests its first rows before it waits for h.  xn and h stay in fp32 here.
#include <atomic>

#include "../../include/moe.h"
#include "moe_block.h"
#include "moe_gate.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCols = 512;  // columns of a warp: 16 a lane
constexpr int kMaxSlots = 32;
constexpr int kGroup = 4;   // slots of an expert that share a read of its weights

struct Experts {
  int n;                      // distinct experts, in order of their first slot
  int e[kMaxSlots];
  unsigned slots[kMaxSlots];  // bit s: slot s
};

// warp 0: the distinct experts of the slots (ids outside [0, E) are left out)
__device__ __forceinline__ void find_experts(const View2& ids, int T, int k, int64_t E, Experts& x) {
  const int lane = threadIdx.x & 31, S = T * k;
  int64_t id = -1;
  if (lane < S) {
    const int64_t off = (lane / k) * ids.s0 + (lane % k) * ids.s1;
    // (from L2: the second kernel reads them before its wait)
    id = ids.dtype == MOE_I64 ? __ldcg(static_cast<const long long*>(ids.data) + off)
                              : static_cast<int64_t>(__ldcg(static_cast<const int*>(ids.data) + off));
  }
  const bool valid = id >= 0 && id < E;
  const int key = valid ? static_cast<int>(id) : -1 - lane;
  const unsigned same = __match_any_sync(0xffffffffu, key);
  const bool first = valid && __ffs(same) - 1 == lane;
  const unsigned firsts = __ballot_sync(0xffffffffu, first);
  if (first) {
    const int r = __popc(firsts & ((1u << lane) - 1u));
    x.e[r] = key;
    x.slots[r] = same;
  }
  if (lane == 0) x.n = __popc(firsts);
}

__device__ __forceinline__ uint4 load_weight(const __nv_bfloat16* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void fma8(float& acc, const uint4& w, const float* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc = fmaf(__uint_as_float(u[i] << 16), x[2 * i], acc);
    acc = fmaf(__uint_as_float(u[i] & 0xffff0000u), x[2 * i + 1], acc);
  }
}

// Sums of kN values over the warp, kN a power of two up to 32: lane l gets the sum of value
// l / (32 / kN).  The halves exchanged shrink with every step (kN - 1 shuffles and a few).
template <int kN>
__device__ __forceinline__ float sums(float (&v)[kN]) {
  const int lane = threadIdx.x & 31;
  int off = 16;
#pragma unroll
  for (int n = kN; n > 1; n >>= 1, off >>= 1) {
    const bool up = (lane & off) != 0;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float send = up ? v[i] : v[i + n / 2], keep = up ? v[i + n / 2] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
    }
  }
  float r = v[0];
  for (; off > 0; off >>= 1) r += __shfl_xor_sync(0xffffffffu, r, off);
  return r;
}

struct UpArgs {
  const float* xn;  // [T, H]
  View2 ids;
  int T, k, H, I;
  int64_t E;
  const __nv_bfloat16 *gate, *up;
  int64_t gs0, gs1, us0, us1;
  float* h;         // [T k, I]
  int rows_max;     // rows of an expert that part holds
};

// up to four slots of a mask, from its lowest on: their count, and the rest of the mask
struct Group {
  int n, slot[kGroup];
};
__device__ __forceinline__ Group take_group(unsigned& mask) {
  Group g;
  g.n = 0;
#pragma unroll
  for (int j = 0; j < kGroup; ++j) {
    g.slot[j] = mask ? __ffs(mask) - 1 : -1;
    if (mask) {
      ++g.n;
      mask &= mask - 1;
    }
  }
  return g;
}

// Rows [0, n) of gate and up from `gate` and `up` for kT slots: part [row][warp of the group][2 kT].
template <int kT, int kRows>
__device__ __forceinline__ void up_rows(const UpArgs& g, const Group& sl, const float* xs, const __nv_bfloat16* gate,
                                        const __nv_bfloat16* up, int n, int group, int groups, int chunk, int nc,
                                        float* part) {
  const int lane = threadIdx.x & 31, col = chunk * kCols + lane * 8;
  uint4 w[kRows][2][2];
  auto fetch = [&](int q) {
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int row = q + u * groups;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        w[u][0][j] = w[u][1][j] = make_uint4(0u, 0u, 0u, 0u);
        if (row < n && col + 256 * j < g.H) {
          w[u][0][j] = load_weight(gate + row * g.gs1 + col + 256 * j);
          w[u][1][j] = load_weight(up + row * g.us1 + col + 256 * j);
        }
      }
    }
  };
  fetch(group);
  float x[kT][16];
#pragma unroll
  for (int t = 0; t < kT; ++t)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = col + 256 * j;
      const bool in = t < sl.n && c < g.H;
      const float4* p = reinterpret_cast<const float4*>(xs + (in ? static_cast<size_t>(sl.slot[t] / g.k) * g.H + c : 0));
      const float4 lo = in ? p[0] : make_float4(0.0f, 0.0f, 0.0f, 0.0f), hi = in ? p[1] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float* o = x[t] + 8 * j;
      o[0] = lo.x; o[1] = lo.y; o[2] = lo.z; o[3] = lo.w;
      o[4] = hi.x; o[5] = hi.y; o[6] = hi.z; o[7] = hi.w;
    }
  for (int q = group; q < n; q += groups * kRows) {
    if (q != group) fetch(q);
    constexpr int kN = kRows * 2 * kT;
    float acc[kN];
#pragma unroll
    for (int u = 0; u < kRows; ++u)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int t = 0; t < kT; ++t) {
          float a = 0.0f;
          fma8(a, w[u][m][0], x[t]);
          fma8(a, w[u][m][1], x[t] + 8);
          acc[(u * 2 + m) * kT + t] = a;
        }
    const float s = sums<kN>(acc);
    const int v = lane / (32 / kN), u = v / (2 * kT), row = q + u * groups;
    if (lane % (32 / kN) == 0 && row < n) part[(row * nc + chunk) * 2 * kT + (v - u * 2 * kT)] = s;
  }
}

// Blocks take equal runs of the (expert, row) list; a block's warps are groups of ceil(H / 512),
// a group a row (gate and up) at a time.
__global__ void __launch_bounds__(kThreads, 1) layer_up_kernel(const UpArgs g) {
  extern __shared__ __align__(16) float smem[];
  float* xs = smem;                                        // [T, H]
  float* part = smem + static_cast<size_t>(g.T) * g.H;
  __shared__ Experts ex;
  const int warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_launch_dependents();  // (after the wait: the next kernel reads the ids before its own)
  if (warp == 0) find_experts(g.ids, g.T, g.k, g.E, ex);
  for (int i = threadIdx.x; i < g.T * g.H / 4; i += kThreads)
    reinterpret_cast<float4*>(xs)[i] = reinterpret_cast<const float4*>(g.xn)[i];
  __syncthreads();
  const int nc = (g.H + kCols - 1) / kCols, groups = kWarps / nc, group = warp / nc, chunk = warp % nc;
  const int64_t total = static_cast<int64_t>(ex.n) * g.I;
  const int64_t r1 = total * (blockIdx.x + 1) / gridDim.x;
  for (int64_t at = total * blockIdx.x / gridDim.x; at < r1;) {
    const int r = static_cast<int>(at / g.I), i0 = static_cast<int>(at - static_cast<int64_t>(r) * g.I);
    int n = g.I - i0;
    if (n > r1 - at) n = static_cast<int>(r1 - at);
    if (n > g.rows_max) n = g.rows_max;
    at += n;
    const int64_t e = ex.e[r];
    const __nv_bfloat16 *gate = g.gate + e * g.gs0 + i0 * g.gs1, *up = g.up + e * g.us0 + i0 * g.us1;
    for (unsigned mask = ex.slots[r]; mask;) {
      const Group sl = take_group(mask);
      if (group < groups) {
        if (sl.n == 1)
          up_rows<1, 4>(g, sl, xs, gate, up, n, group, groups, chunk, nc, part);
        else if (sl.n == 2)
          up_rows<2, 4>(g, sl, xs, gate, up, n, group, groups, chunk, nc, part);
        else
          up_rows<4, 2>(g, sl, xs, gate, up, n, group, groups, chunk, nc, part);
      }
      __syncthreads();
      const int kt = sl.n > 2 ? 4 : sl.n;
      for (int i = threadIdx.x; i < n * sl.n; i += kThreads) {
        const int t = i / n, row = i - t * n;
        float a = 0.0f, b = 0.0f;
        for (int c = 0; c < nc; ++c) {
          a += part[(row * nc + c) * 2 * kt + t];
          b += part[(row * nc + c) * 2 * kt + kt + t];
        }
        const int s = t == 0 ? sl.slot[0] : t == 1 ? sl.slot[1] : t == 2 ? sl.slot[2] : sl.slot[3];
        g.h[static_cast<int64_t>(s) * g.I + i0 + row] = a / (1.0f + expf(-a)) * b;
      }
      __syncthreads();
    }
  }
}

struct DownArgs {
  const float* h;  // [T k, I]
  View2 ids, wts;
  int T, k, H, I;
  int64_t E;
  const __nv_bfloat16* w2;
  int64_t ws0, ws1;
  __nv_bfloat16* out;
  int64_t os0, os1;
  Finish finish;
};

template <int kRows>
__device__ __forceinline__ void down_fetch(uint4 (&w)[8][2], const __nv_bfloat16* base, int64_t ld, int rows, int cols) {
#pragma unroll
  for (int u = 0; u < kRows; ++u)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      w[u][j] = make_uint4(0u, 0u, 0u, 0u);
      if (u < rows && 256 * j < cols) w[u][j] = load_weight(base + u * ld + 256 * j);
    }
}

// The rows of one expert's 512 columns for kT slots, added to mine [row][T].  base: the lane's
// columns of the block's first row, cols: columns of the matrix from the lane's first on.  w: the
// first rows' weights where `have`.
template <int kT, int kRows>
__device__ __forceinline__ void down_rows(const DownArgs& g, const Group& sl, int col, const __nv_bfloat16* base, int n,
                                          float* mine, uint4 (&w)[8][2], bool have) {
  const int lane = threadIdx.x & 31, cols = g.I - col;
  if (!have) down_fetch<kRows>(w, base, g.ws1, n, cols);
  float x[kT][16];
#pragma unroll
  for (int t = 0; t < kT; ++t) {
    const bool on = t < sl.n;
    const int s = on ? sl.slot[t] : 0, tok = s / g.k;
    const float f = on ? static_cast<const float*>(g.wts.data)[tok * g.wts.s0 + (s - tok * g.k) * g.wts.s1] : 0.0f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const bool in = on && 256 * j < cols;
      const float4* p = reinterpret_cast<const float4*>(g.h + (in ? static_cast<int64_t>(s) * g.I + col + 256 * j : 0));
      const float4 lo = in ? p[0] : make_float4(0.0f, 0.0f, 0.0f, 0.0f), hi = in ? p[1] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float* o = x[t] + 8 * j;
      o[0] = f * lo.x; o[1] = f * lo.y; o[2] = f * lo.z; o[3] = f * lo.w;
      o[4] = f * hi.x; o[5] = f * hi.y; o[6] = f * hi.z; o[7] = f * hi.w;
    }
  }
  for (int q = 0; q < n; q += kRows) {
    if (q > 0) down_fetch<kRows>(w, base + q * g.ws1, g.ws1, n - q, cols);
    constexpr int kN = kRows * kT;
    float acc[kN];
#pragma unroll
    for (int u = 0; u < kRows; ++u)
#pragma unroll
      for (int t = 0; t < kT; ++t) {
        float a = 0.0f;
        fma8(a, w[u][0], x[t]);
        fma8(a, w[u][1], x[t] + 8);
        acc[u * kT + t] = a;
      }
    const float s = sums<kN>(acc);
    const int v = lane / (32 / kN), row = q + v / kT, t = v % kT;
    if (lane % (32 / kN) == 0 && row < n && t < sl.n) {
      const int slot = t == 0 ? sl.slot[0] : t == 1 ? sl.slot[1] : t == 2 ? sl.slot[2] : sl.slot[3];
      mine[row * g.T + slot / g.k] += s;
    }
  }
}

// Blocks take equal runs of output rows; a block's warps take the (expert, 512 columns) pairs in
// turn, each over all the block's rows.  part: [warp][row][T]
// The first rows' weights (64 registers) live across the bodies for one, two and four slots: at 128
// registers a thread spills 444 bytes.
__global__ void __launch_bounds__(kThreads, 1) layer_down_kernel(const DownArgs g) {
  extern __shared__ __align__(16) float smem[];
  float* part = smem;
  __shared__ Experts ex;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) find_experts(g.ids, g.T, g.k, g.E, ex);
  const int o0 = static_cast<int>(static_cast<int64_t>(g.H) * blockIdx.x / gridDim.x);
  const int n = static_cast<int>(static_cast<int64_t>(g.H) * (blockIdx.x + 1) / gridDim.x) - o0;
  for (int i = threadIdx.x; i < kWarps * n * g.T; i += kThreads) part[i] = 0.0f;
  __syncthreads();
  const int nc = (g.I + kCols - 1) / kCols, tasks = ex.n * nc;
  auto base_of = [&](int task) {
    const int r = task / nc;
    return g.w2 + static_cast<int64_t>(ex.e[r]) * g.ws0 + static_cast<int64_t>(o0) * g.ws1 + (task - r * nc) * kCols + lane * 8;
  };
  uint4 first[8][2];
  if (warp < tasks)  // the weights do not depend on the kernel before
    down_fetch<8>(first, base_of(warp), g.ws1, n, g.I - (warp % nc) * kCols - lane * 8);
  pdl_wait();
  pdl_launch_dependents();
  float* mine = part + warp * n * g.T;
  bool have = true;
  for (int task = warp; task < tasks; task += kWarps) {
    const int r = task / nc, col = (task - r * nc) * kCols + lane * 8;
    for (unsigned mask = ex.slots[r]; mask;) {
      const Group sl = take_group(mask);
      if (sl.n == 1)
        down_rows<1, 8>(g, sl, col, base_of(task), n, mine, first, have);
      else if (sl.n == 2)
        down_rows<2, 8>(g, sl, col, base_of(task), n, mine, first, have);
      else
        down_rows<4, 4>(g, sl, col, base_of(task), n, mine, first, have);
      __syncwarp();
      have = false;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n * g.T; i += kThreads) {
    const int t = i / n, row = i - t * n, o = o0 + row;
    float a = 0.0f;
    for (int q = 0; q < kWarps; ++q) a += part[(q * n + row) * g.T + t];
    if (g.finish.mode == kFinishRows) {
      g.finish.y32[static_cast<int64_t>(t) * g.H + o] = a;
      continue;
    }
    if (g.finish.gate.data) a *= gate_value(view_float(g.finish.gate, t, o), g.finish.act);
    if (g.finish.alpha != 0.0f) a += g.finish.alpha * view_float(g.finish.residual, t, o);
    g.out[t * g.os0 + o * g.os1] = __float2bfloat16_rn(a);
  }
}

constexpr int kSmemMax = 200 << 10;

template <typename K>
cudaError_t raise_smem(K kernel, std::atomic<unsigned long long>& configured) {
  int dev = 0;
  cudaError_t rc = cudaGetDevice(&dev);
  if (rc != cudaSuccess) return rc;
  if (dev < 64 && (configured.load() & (1ull << dev))) return cudaSuccess;
  rc = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
  if (rc == cudaSuccess && dev < 64) configured.fetch_or(1ull << dev);
  return rc;
}

}  // namespace

// At most 32 slots (a warp finds the experts), rows of at most 16 x 512 columns, the normed rows in
// shared memory.  Up to four tokens an expert's weights are read once whatever the choice; with
// more, experts must not be shared by many, and large matrices gain nothing over the tensor-core
// tiles: Qwen3-235B shape T=1 61 us against 73, T=2 104 / 122, T=4 190 / 197; H=4096 I=1536, 4 of
// 128 experts, T=6 155 / 163; 4 of 64, T=8 202 / 185; H=2048 I=768, 4 of 16, T=8 58 / 73.
bool layer_by_rows(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k) {
  if (T > 8 || T * k > kMaxSlots || H > kCols * kWarps || T * H * 4 > (128 << 10)) return false;
  return T <= 4 || (T * k <= 2 * E && (T <= 6 || H * I <= (2 << 20)));
}

cudaError_t launch_layer_rows(const LayerRows& a, int num_sms, cudaStream_t st) {
  UpArgs u = {};
  u.xn = a.xn;
  u.ids = a.ids;
  u.T = a.T;
  u.k = a.k;
  u.H = a.H;
  u.I = a.I;
  u.E = a.E;
  u.gate = a.gate;
  u.up = a.up;
  u.gs0 = a.gs0;
  u.gs1 = a.gs1;
  u.us0 = a.us0;
  u.us1 = a.us1;
  u.h = a.h;
  static std::atomic<unsigned long long> up_configured{0}, down_configured{0};
  const int nc = (a.H + kCols - 1) / kCols;
  const size_t xs = static_cast<size_t>(a.T) * a.H * 4;
  const int64_t rows = (static_cast<int64_t>(a.T) * a.k * a.I + num_sms - 1) / num_sms;
  const int64_t row_bytes = static_cast<int64_t>(nc) * 2 * kGroup * 4, fit = (64 << 10) / row_bytes;
  u.rows_max = static_cast<int>(rows < fit ? rows : fit);
  cudaError_t rc = raise_smem(layer_up_kernel, up_configured);
  if (rc != cudaSuccess) return rc;
  rc = launch_pdl(layer_up_kernel, dim3(static_cast<unsigned>(num_sms)), dim3(kThreads), xs + u.rows_max * row_bytes, st, u);
  if (rc != cudaSuccess) return rc;
  DownArgs d = {};
  d.h = a.h;
  d.ids = a.ids;
  d.wts = a.wts;
  d.T = a.T;
  d.k = a.k;
  d.H = a.H;
  d.I = a.I;
  d.E = a.E;
  d.w2 = a.w2;
  d.ws0 = a.ws0;
  d.ws1 = a.ws1;
  d.out = a.out;
  d.os0 = a.os0;
  d.os1 = a.os1;
  d.finish = a.finish;
  const int64_t n = (a.H + num_sms - 1) / num_sms;
  rc = raise_smem(layer_down_kernel, down_configured);
  if (rc != cudaSuccess) return rc;
  return launch_pdl(layer_down_kernel, dim3(static_cast<unsigned>(num_sms)), dim3(kThreads),
                    static_cast<size_t>(kWarps) * n * a.T * 4, st, d);
}

}  // namespace moe
