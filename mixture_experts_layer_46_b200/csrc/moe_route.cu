// The way into a mixture-of-experts layer for a few tokens, in one launch: the norm of the
// token's row, the product with the router's rows, softmax and the choice of the k experts.
//
//   xn[t] = x[t] r w,  r = 1 / sqrt(mean x[t]^2 + eps)
//   l[t, e] = sum_h x[t, h] w[h] router[e, h] r
//   the k largest l, a tie going to the lower index; weights softmax(l) over all experts, or
//   over the chosen ones
//
// A cluster of CTAs takes a token, each CTA a share of the experts, and hands its logits
// to all of them, so that every CTA ranks its experts against all others without another launch or
// a counter in memory.  The choice between two experts must not hang on the order of additions,
// so the sums carry their rounding errors along and meet in 64 bits; fp64 multiply-adds all the way
// took four times as long.  The terms are exact in fp32 (8 bits times 8 times 8) where pre_weight and
// the router are bf16; an f32 pre_weight leaves the roundings of x w and of its product, an f32 router
// takes the path in 64 bits.  Latency bounds the time otherwise: a warp takes 256 columns of eight
// experts at once, all loads in flight together.  128 x 4096 router, one token: 7.4 us.
#include <atomic>

#include "../../include/moe.h"
#include "moe_block.h"
#include "moe_internal.h"
#include "moe_pair.cuh"

namespace moe {
namespace {

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

// Two floats at a time (the pair's first in the low half).
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  return static_cast<uint64_t>(__float_as_uint(a)) | (static_cast<uint64_t>(__float_as_uint(b)) << 32);
}
__device__ __forceinline__ double lo_of(uint64_t p) { return static_cast<double>(__uint_as_float(static_cast<uint32_t>(p))); }
__device__ __forceinline__ double hi_of(uint64_t p) { return static_cast<double>(__uint_as_float(static_cast<uint32_t>(p >> 32))); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(b), "l"(0xbf800000bf800000ull), "l"(a));
  return r;
}
// sum + low += p, low taking what the rounding of sum leaves (the exact error of an addition,
// by six more: Knuth's two-sum)
__device__ __forceinline__ void add_exact(uint64_t& sum, uint64_t& low, uint64_t p) {
  const uint64_t s = add2(sum, p), b = sub2(s, sum);
  low = add2(low, add2(sub2(sum, sub2(s, b)), sub2(p, b)));
  sum = s;
}

// Sums of eight values over the warp: lane l gets the sum of value l / 4.
__device__ __forceinline__ double warp_sums8(double (&v)[8]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 8, off = 16; n > 1; n >>= 1, off >>= 1) {
    const bool up = (lane & off) != 0;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const double send = up ? v[i] : v[i + n / 2], keep = up ? v[i + n / 2] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
    }
  }
  v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

// A signed key that orders as the double it came from (-0 is +0), and back.  What is not finite comes back
// as NaN and is below every number: the compensated sums make NaN of an infinite term, and the sums
// in 64 bits, which would keep it, have to rank the same experts first.
__device__ __forceinline__ long long key_of(double v) {
  if (!isfinite(v)) return (-9223372036854775807ll - 1);
  const long long b = __double_as_longlong(v + 0.0);
  return b ^ ((b >> 63) & 0x7fffffffffffffffll);
}
__device__ __forceinline__ double of_key(long long k) { return __longlong_as_double(k ^ ((k >> 63) & 0x7fffffffffffffffll)); }

__device__ __forceinline__ void st_cluster_s64(uint32_t addr, long long v) {
  asm volatile("st.shared::cluster.s64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

template <int kCtas>
__global__ void __launch_bounds__(kThreads) route_kernel(const Route g) {
  extern __shared__ __align__(16) float xw[];  // [H]: x w
  __shared__ long long logit[1024];  // as keys
  __shared__ double red[kWarps];
  __shared__ int chosen[32];  // by rank (the first CTA's)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int64_t t = blockIdx.x / kCtas;
  const int H = g.H, E = g.E;
  // (all of them have to run before one writes into another's shared memory)
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  pdl_wait();
  pdl_launch_dependents();

  const int share = (E + kCtas - 1) / kCtas, e0 = static_cast<int>(rank) * share;
  const int mine_n = E - e0 < share ? E - e0 : share;  // (may be below 1)
  const int chunks = (H + 255) / 256, batches = (mine_n + 7) / 8;
  uint4 v[8];  // eight experts' weights in this lane's columns
  auto fetch = [&](int task) {
    const int chunk = task % chunks, first = task / chunks * 8, c = chunk * 256 + lane * 8;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      v[q] = make_uint4(0u, 0u, 0u, 0u);
      if (first + q < mine_n && c < H)
        v[q] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(g.router.data) + (e0 + first + q) * g.router.s0 + c);
    }
  };
  if (g.wide && warp < chunks * batches) fetch(warp);

  double ss = 0.0;
  if (g.x_wide) {
    for (int c = threadIdx.x * 8; c < H; c += kThreads * 8) {
      const uint4 xv = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(g.x.data) + t * g.x.s0 + c);
      uint4 wv = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);  // ones
      if (g.w.data) wv = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(g.w.data) + c);
      const uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w}, ws[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = __uint_as_float(xs[i] << 16), hi = __uint_as_float(xs[i] & 0xffff0000u);
        *reinterpret_cast<float2*>(xw + c + 2 * i) =
            make_float2(lo * __uint_as_float(ws[i] << 16), hi * __uint_as_float(ws[i] & 0xffff0000u));
        ss += static_cast<double>(lo) * static_cast<double>(lo);
        ss += static_cast<double>(hi) * static_cast<double>(hi);
      }
    }
  } else {
    for (int h = threadIdx.x; h < H; h += kThreads) {
      const float x = row_float(g.x, t, h);
      xw[h] = x * (g.w.data ? row_float(g.w, 0, h) : 1.0f);
      ss += static_cast<double>(x) * static_cast<double>(x);
    }
  }
  ss = warp_sum(ss);
  if (lane == 0) red[warp] = ss;
  __syncthreads();
  ss = warp_sum(lane < kWarps ? red[lane] : 0.0);
  const double r = 1.0 / sqrt(ss / H + static_cast<double>(g.eps));
  // this CTA's part of the normed row, rounded once
  const int per = (H + kCtas - 1) / kCtas, h0 = static_cast<int>(rank) * per;
  for (int h = h0 + threadIdx.x; h < H && h < h0 + per; h += kThreads)
    if (g.xn32)
      g.xn32[t * H + h] = xw[h] * static_cast<float>(r);
    else
      g.xn[t * H + h] = __float2bfloat16_rn(xw[h] * static_cast<float>(r));
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");

  if (g.wide) {
    // part [chunk of 256 columns][expert of this CTA]
    double* part = reinterpret_cast<double*>(xw + (H + 3) / 4 * 4);
    for (int task = warp; task < chunks * batches; task += kWarps) {
      const int chunk = task % chunks, first = task / chunks * 8, c = chunk * 256 + lane * 8;
      if (task != warp) fetch(task);
      uint64_t x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = c < H ? *reinterpret_cast<const uint64_t*>(xw + c + 2 * i) : 0ull;
      double acc[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint32_t w[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
        uint64_t sum = 0ull, low = 0ull;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          add_exact(sum, low, mul2(x[i], pair_of(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u))));
        acc[q] = (lo_of(sum) + lo_of(low)) + (hi_of(sum) + hi_of(low));
      }
      const double l = warp_sums8(acc);
      if ((lane & 3) == 0 && first + (lane >> 2) < mine_n) part[chunk * share + first + (lane >> 2)] = l;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < mine_n * kCtas; i += kThreads) {
      const int e = i / kCtas;
      double l = 0.0;
#pragma unroll 8
      for (int q = 0; q < chunks; ++q) l += part[q * share + e];
      st_cluster_s64(mapa_shared(smem_u32(&logit[e0 + e]), i % kCtas), key_of(l * r));
    }
  } else {
    for (int e = warp; e < mine_n; e += kWarps) {
      double a = 0.0;
      for (int h = lane; h < H; h += 32)
        a += static_cast<double>(xw[h]) * static_cast<double>(row_float(g.router, e0 + e, h));
      const double l = warp_sum(a) * r;
      if (lane < kCtas) st_cluster_s64(mapa_shared(smem_u32(&logit[e0 + e]), lane), key_of(l));
    }
  }
  cluster_sync_all();

  // the rank of each of this CTA's experts, a warp an expert: how many come before it
  for (int i = warp; i < mine_n; i += kWarps) {
    const int e = e0 + i;
    const long long l = logit[e];
    unsigned n = 0;
    for (int o = lane; o < E; o += 32) n += logit[o] > l || (logit[o] == l && o < e) ? 1u : 0u;
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0 && n < static_cast<unsigned>(g.k)) st_cluster_u32(mapa_shared(smem_u32(&chosen[n]), 0), static_cast<uint32_t>(e));
  }
  cluster_sync_all();
  if (rank != 0 || warp != 0) return;
  const double m = of_key(logit[chosen[0]]);
  const int id = lane < g.k ? chosen[lane] : 0;
  const double ex = lane < g.k ? exp(of_key(logit[id]) - m) : 0.0;
  double part = ex;
  if (!g.renorm) {
    part = 0.0;
    for (int e = lane; e < E; e += 32) part += exp(of_key(logit[e]) - m);
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

// x w, and the sums of every 256 columns of a CTA's experts
size_t route_smem(int64_t H, int64_t E, int ctas) {
  return static_cast<size_t>((H + 3) / 4 * 16 + (H + 255) / 256 * ((E + ctas - 1) / ctas) * 8);
}

template <int kCtas>
cudaError_t launch_clusters(const Route& g, cudaStream_t st) {
  static std::atomic<unsigned long long> configured{0};
  int dev = 0;
  cudaError_t rc = cudaGetDevice(&dev);
  if (rc != cudaSuccess) return rc;
  if (dev >= 64 || !(configured.load() & (1ull << dev))) {
    rc = cudaFuncSetAttribute(route_kernel<kCtas>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(route_smem(kRouteMaxH, kRouteMaxE, kCtas)));
    if (rc != cudaSuccess) return rc;
    rc = cudaFuncSetAttribute(route_kernel<kCtas>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (rc != cudaSuccess) return rc;
    if (dev < 64) configured.fetch_or(1ull << dev);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(g.T * kCtas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = route_smem(g.H, g.E, kCtas);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCtas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, route_kernel<kCtas>, g);
}

}  // namespace

// More CTAs a token are faster as long as the clusters find places at once: sixteen for up to four
// tokens (7.4 us at one token, 9.5 with eight), eight for up to eight (6.7 us at eight tokens of
// 2080 columns, 10.6 with sixteen; sixteen tokens 11.2), then four (20 to 28 tokens 6.9 us).
cudaError_t launch_route(const Route& g, cudaStream_t st) {
  if (g.T <= 4) return launch_clusters<16>(g, st);
  return g.T <= 8 ? launch_clusters<8>(g, st) : launch_clusters<4>(g, st);
}

}  // namespace moe
