// The way into a mixture-of-experts layer for a few tokens, in one launch: the norm of the
// token's row, the product with the router's rows, softmax and the choice of the k experts.
//
//   xn[t] = x[t] r w,  r = 1 / sqrt(mean x[t]^2 + eps)
//   l[t, e] = sum_h x[t, h] w[h] router[e, h] r
//   the k largest l, a tie going to the lower index; weights softmax(l) over all experts, or
//   over the chosen ones
//
// A cluster of eight CTAs takes a token: each CTA a share of the experts, a warp an expert at a
// time, and each warp hands its logit to all eight, so that every CTA ranks its experts against
// all of them without another launch or a counter in memory.  The logits are summed in 64 bits:
// x w (16 bits) times a bf16 router weight is exact in fp32, and the choice between two experts
// then does not hang on the order of additions.  One conversion an element bounds the time at
// one token (128 x 4096 router: 0.5 M conversions on 8 SMs, 2 us); it is spread over the SMs by
// the tokens as they become more.
#include <atomic>

#include "../../include/moe.h"
#include "moe_block.h"
#include "moe_internal.h"
#include "moe_pair.cuh"

namespace moe {
namespace {

constexpr int kCtas = 8;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float row_float(const RowView& t, int64_t row, int64_t c) {
  const int64_t off = row * t.s0 + c * t.s1;
  return t.dtype == MOE_F32
             ? static_cast<const float*>(t.data)[off]
             : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(t.data)[off]) << 16);
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void st_cluster_f64(uint32_t addr, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// a ranks before b (their indices i and j); NaN after every number
__device__ __forceinline__ bool before(double a, int i, double b, int j) {
  const bool an = a != a, bn = b != b;
  if (an || bn) return an == bn ? i < j : bn;
  return a > b || (a == b && i < j);
}

__global__ void __launch_bounds__(kThreads) __cluster_dims__(kCtas, 1, 1) route_kernel(const Route g) {
  extern __shared__ __align__(16) float xw[];  // [H]: x w
  __shared__ double logit[1024];
  __shared__ double red[kWarps];
  __shared__ int chosen[32];  // by rank (the first CTA's)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int64_t t = blockIdx.x / kCtas;
  const int H = g.H, E = g.E;
  // (all eight have to run before one writes into another's shared memory)
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  pdl_wait();
  pdl_launch_dependents();

  double ss = 0.0;
  for (int h = threadIdx.x; h < H; h += kThreads) {
    const float x = row_float(g.x, t, h);
    xw[h] = x * (g.w.data ? row_float(g.w, 0, h) : 1.0f);
    ss += static_cast<double>(x) * static_cast<double>(x);
  }
  ss = warp_sum(ss);
  if (lane == 0) red[warp] = ss;
  __syncthreads();
  ss = 0.0;
  for (int i = 0; i < kWarps; ++i) ss += red[i];
  const double r = 1.0 / sqrt(ss / H + static_cast<double>(g.eps));
  // this CTA's part of the normed row, rounded once
  const int per = (H + kCtas - 1) / kCtas, h0 = static_cast<int>(rank) * per;
  for (int h = h0 + threadIdx.x; h < H && h < h0 + per; h += kThreads)
    g.xn[t * H + h] = __float2bfloat16_rn(xw[h] * static_cast<float>(r));
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");

  for (int e = static_cast<int>(rank) * kWarps + warp; e < E; e += kCtas * kWarps) {
    double a0 = 0.0, a1 = 0.0;
    if (g.wide) {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(g.router.data) + e * g.router.s0);
#pragma unroll 4
      for (int c = lane; c < H / 8; c += 32) {
        const uint4 v = p[c];
        const float4 lo = *reinterpret_cast<const float4*>(xw + 8 * c), hi = *reinterpret_cast<const float4*>(xw + 8 * c + 4);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        const float f[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a0 += static_cast<double>(f[2 * i] * __uint_as_float(w[i] << 16));
          a1 += static_cast<double>(f[2 * i + 1] * __uint_as_float(w[i] & 0xffff0000u));
        }
      }
    } else {
      for (int h = lane; h < H; h += 32)
        a0 += static_cast<double>(xw[h]) * static_cast<double>(row_float(g.router, e, h));
    }
    const double l = warp_sum(a0 + a1) * r;
    if (lane < kCtas) st_cluster_f64(mapa_shared(smem_u32(&logit[e]), lane), l);
  }
  cluster_sync_all();

  // the rank of each of this CTA's experts: four threads an expert, a quarter of the others each
  const int share = (E + kCtas - 1) / kCtas, e0 = static_cast<int>(rank) * share;
  for (int base = 0; base < share; base += kThreads / 4) {
    const int i = base + (threadIdx.x >> 2), e = e0 + i;
    const bool mine = i < share && e < E;
    int n = 0;
    if (mine) {
      const double l = logit[e];
      for (int o = threadIdx.x & 3; o < E; o += 4) n += before(logit[o], o, l, e) ? 1 : 0;
    }
    n += __shfl_xor_sync(0xffffffffu, n, 1);
    n += __shfl_xor_sync(0xffffffffu, n, 2);
    if (mine && (threadIdx.x & 3) == 0 && n < g.k)
      st_cluster_u32(mapa_shared(smem_u32(&chosen[n]), 0), static_cast<uint32_t>(e));
  }
  cluster_sync_all();
  if (rank != 0 || warp != 0) return;
  const double m = logit[chosen[0]];
  const int id = lane < g.k ? chosen[lane] : 0;
  const double ex = lane < g.k ? exp(logit[id] - m) : 0.0;
  double part = ex;
  if (!g.renorm) {
    part = 0.0;
    for (int e = lane; e < E; e += 32) part += exp(logit[e] - m);
  }
  part = warp_sum(part);
  if (lane < g.k + (g.shared ? 1 : 0)) {
    const bool sh = lane == g.k;
    const int64_t io = t * g.ids.s0 + lane * g.ids.s1;
    const int out_id = sh ? E : id;
    if (g.ids.dtype == MOE_I64)
      static_cast<int64_t*>(const_cast<void*>(g.ids.data))[io] = out_id;
    else
      static_cast<int32_t*>(const_cast<void*>(g.ids.data))[io] = out_id;
    static_cast<float*>(const_cast<void*>(g.wts.data))[t * g.wts.s0 + lane * g.wts.s1] =
        sh ? 1.0f : static_cast<float>(ex / part);
  }
}

}  // namespace

cudaError_t launch_route(const Route& g, cudaStream_t st) {
  static std::atomic<unsigned long long> configured{0};
  int dev = 0;
  cudaError_t rc = cudaGetDevice(&dev);
  if (rc != cudaSuccess) return rc;
  if (dev >= 64 || !(configured.load() & (1ull << dev))) {
    rc = cudaFuncSetAttribute(route_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(kRouteMaxH * sizeof(float)));
    if (rc != cudaSuccess) return rc;
    if (dev < 64) configured.fetch_or(1ull << dev);
  }
  return launch_pdl(route_kernel, dim3(static_cast<unsigned>(g.T * kCtas)), dim3(kThreads),
                    static_cast<size_t>(g.H) * sizeof(float), st, g);
}

}  // namespace moe
