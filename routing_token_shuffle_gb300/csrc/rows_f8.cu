// Rows in 8-bit floating point (e4m3) with a scale per row and 128 channels, and the SwiGLU
// activation that keeps its inputs so between the forward and the backward pass:
//   s = max |x| / 448 over a block (or the power of two that is not below it), q = rn(x / s);
//   h = g sig(g) u, keeping g and u as such blocks;
//   dg = dh u sig(g) (1 + g (1 - sig(g))), du = dh g sig(g), h again, from what was kept.
// Every element is read once and written once, so HBM is the bound. A block of 128 channels is
// 16 lanes of 8 values (16 bytes of bf16, 8 of the 8-bit values: full sectors both ways); its
// largest magnitude takes four shuffles, and nothing is kept in shared memory. A power-of-two
// scale costs no precision but at the smallest magnitudes (the format has its own exponent), its
// division is exact, and what it stands for is exact in bf16, so that a product of bf16 rows
// reads the kept values without another rounding.
// Measured: 131072 rows of 768, bf16, forward 140 us and backward 145 (6.4 TB/s); 16384 rows of 2048
// to 8 bits 23 us, 4.4 TB/s (16384 short blocks: start and end weigh).
#include <algorithm>
#include <cfloat>
#include <cuda_fp8.h>

#include "smoe_internal.cuh"

namespace smoe {
namespace {

constexpr int kRowsThreads = 256;                 // 16 blocks of 128 channels at a time
constexpr int kRowsGroups = kRowsThreads / 16;

__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* v) {
  unpack16(*reinterpret_cast<const uint4*>(p), v, (const __nv_bfloat16*)nullptr);
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* v) {
  *reinterpret_cast<uint4*>(p) = pack16(v, (const __nv_bfloat16*)nullptr);
}

// The block's 16 lanes hold 8 values each (zeros past the row's end). Magnitudes are compared as
// unsigned integers: a NaN is above every number, so its block does not pass for a finite one.
// A block whose scale would be subnormal gets scale 0 and zeros, one with an infinity or a NaN
// scale NaN and zeros.
template <bool POW2>
__device__ __forceinline__ uint2 quantise8(const float* v, float* scale) {
  uint32_t big = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) big = max(big, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
  for (int off = 8; off; off >>= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, off));
  const float amax = __uint_as_float(big);
  const bool finite = big <= 0x7f7fffffu;
  float s = amax / 448.0f;
  const bool zero = !finite || s < FLT_MIN;
  if (zero) s = finite ? 0.0f : __int_as_float(0x7fc00000);
  else if (POW2) s = __uint_as_float((__float_as_uint(s) + 0x7fffffu) & 0x7f800000u);
  *scale = s;
  uint2 q = make_uint2(0u, 0u);
  if (!zero) {
    const float inv = 1.0f / s;  // exact for a power of two (between 2^-126 and 2^120)
    float t[8];
    if (POW2) {
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = v[i] * inv;
    } else if (s >= 0x1p-90f) {
      // x / s from the rounded reciprocal: the product is off by at most a step, its residual
      // x - t s is exact (below |x| = s 2^-10 the result is zero either way, and above the residual's
      // last place is at least 2^-146), and one correction rounds as the division does (Markstein's
      // theorem on quotients from a correctly rounded reciprocal). (With divisions 16384 rows of 2048
      // took 30 us, against 26.)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        t[i] = v[i] * inv;
        t[i] = fmaf(fmaf(-t[i], s, v[i]), inv, t[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = v[i] / s;
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = __nv_cvt_float2_to_fp8x2(make_float2(t[2 * i], t[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    q = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
  }
  return q;
}

// 8 kept values times their block's scale
__device__ __forceinline__ void widen8(const uint2& q, float s, float* v) {
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2(
        (__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1)) & 0xffffu), __NV_E4M3));
    const float2 f = __half22float2(h);
    v[2 * i] = f.x * s;
    v[2 * i + 1] = f.y * s;
  }
}

// sig(x): for fp32 results with the accurate forms; for bf16 ones (and 8-bit ones, whose steps are
// larger) with the fast exponential, off by at most 2 + 1.2 |x| steps of 2^-23, and the fast division:
// (4 + 1.2 |x|) 2^-23 of sig in all, at most 2^-16 before sig leaves the normal numbers at x = -87,
// beside half a step of bf16, 2^-8
template <typename TE>
__device__ __forceinline__ float sigmoid(float x) {
  if (sizeof(TE) == 2) return __fdividef(1.0f, 1.0f + __expf(-x));
  return 1.0f / (1.0f + expf(-x));
}

// This thread's place: item `it` of `items` is 128 channels of a row. One item a thread: in the
// SwiGLU kernels, which load two or three vectors an item, many small blocks kept more loads in flight
// than two or four items of a thread with their loads first (131072 rows of 768, forward and backward: one
// 291 us, two 325, four 435). (rows_f8_kernel, one load an item, has the same form and was not measured
// with more.)
struct Place {
  bool in, lead;   // inside the row; the block's first lane
  size_t at, block;  // element and scale index
};
__device__ __forceinline__ Place place(uint32_t items, int cols, uint32_t nblk) {
  const uint32_t it = blockIdx.x * kRowsGroups + (threadIdx.x >> 4), row = it / nblk, b = it - row * nblk;
  const int l = threadIdx.x & 15, col = (int)b * 128 + l * 8;
  Place p;
  p.in = it < items && col < cols;
  p.lead = it < items && l == 0;
  p.at = (size_t)row * cols + col;
  p.block = (size_t)row * nblk + b;
  return p;
}

template <typename TE, bool POW2>
__global__ void __launch_bounds__(kRowsThreads)
rows_f8_kernel(const TE* x, uint2* q, float* scale, uint32_t items, int cols, uint32_t nblk) {
  pdl_wait_and_trigger();
  const Place p = place(items, cols, nblk);
  float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f}, s;
  if (p.in) load8(x + p.at, v);
  const uint2 w = quantise8<POW2>(v, &s);
  if (p.in) q[p.at >> 3] = w;
  if (p.lead) scale[p.block] = s;
}

template <typename TE>
struct SwigluArgs {
  const TE *g, *u;
  TE* h;               // each output nullable
  uint2 *h8, *g8, *u8;
  float *hs, *gs, *us;
  uint32_t items, nblk;
  int cols;
};

template <typename TE, bool POW2>
__global__ void __launch_bounds__(kRowsThreads)
swiglu_f8_kernel(const SwigluArgs<TE> a) {
  pdl_wait_and_trigger();
  const Place p = place(a.items, a.cols, a.nblk);
  float g[8], u[8], s;
#pragma unroll
  for (int i = 0; i < 8; ++i) g[i] = u[i] = 0.0f;
  if (p.in) {
    load8(a.g + p.at, g);
    load8(a.u + p.at, u);
  }
  if (a.g8) {
    const uint2 w = quantise8<POW2>(g, &s);
    if (p.in) a.g8[p.at >> 3] = w;
    if (p.lead) a.gs[p.block] = s;
  }
  if (a.u8) {
    const uint2 w = quantise8<POW2>(u, &s);
    if (p.in) a.u8[p.at >> 3] = w;
    if (p.lead) a.us[p.block] = s;
  }
  if (a.h == nullptr && a.h8 == nullptr) return;
  float h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = g[i] * sigmoid<TE>(g[i]) * u[i];
  if (a.h && p.in) store8(a.h + p.at, h);
  if (a.h8) {
    const uint2 w = quantise8<POW2>(h, &s);
    if (p.in) a.h8[p.at >> 3] = w;
    if (p.lead) a.hs[p.block] = s;
  }
}

template <typename TE>
struct SwigluGradArgs {
  const TE* dh;
  const uint2 *g8, *u8;
  const float *gs, *us;
  TE *dg, *du, *h;     // h nullable
  uint32_t items, nblk;
  int cols;
};

template <typename TE>
__global__ void __launch_bounds__(kRowsThreads)
swiglu_grad_f8_kernel(const SwigluGradArgs<TE> a) {
  pdl_wait_and_trigger();
  const Place p = place(a.items, a.cols, a.nblk);
  if (!p.in) return;
  float d[8], g[8], u[8], h[8];
  load8(a.dh + p.at, d);
  const uint2 g8 = a.g8[p.at >> 3], u8 = a.u8[p.at >> 3];
  const float gs = a.gs[p.block], us = a.us[p.block];
  widen8(g8, gs, g);
  widen8(u8, us, u);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float sig = sigmoid<TE>(g[i]), silu = g[i] * sig;
    h[i] = silu * u[i];
    g[i] = d[i] * u[i] * (sig * (1.0f + g[i] * (1.0f - sig)));
    u[i] = d[i] * silu;
  }
  store8(a.dg + p.at, g);
  store8(a.du + p.at, u);
  if (a.h) store8(a.h + p.at, h);
}

}  // namespace

cudaError_t launch_rows_f8(const smoe_desc& d, int rows, int cols, const void* x, int pow2, void* q,
                           float* scale, cudaStream_t s) {
  const uint32_t nblk = ceil_div(cols, 128), items = (uint32_t)rows * nblk;
  auto run = [&](auto* xt) -> cudaError_t {
    using TE = std::remove_const_t<std::remove_pointer_t<decltype(xt)>>;
    auto kern = pow2 ? rows_f8_kernel<TE, true> : rows_f8_kernel<TE, false>;
    SMOE_LAUNCH(kern, ceil_div(items, kRowsGroups), kRowsThreads, 0, s, xt, static_cast<uint2*>(q), scale,
                items, cols, nblk);
    return cudaGetLastError();
  };
  return d.dtype == SMOE_F32 ? run(static_cast<const float*>(x))
                             : run(static_cast<const __nv_bfloat16*>(x));
}

cudaError_t launch_swiglu_f8(const smoe_desc& d, int rows, int cols, const void* g, const void* u,
                             int pow2, void* h, const F8Rows& h8, const F8Rows& g8, const F8Rows& u8,
                             cudaStream_t s) {
  const uint32_t nblk = ceil_div(cols, 128), items = (uint32_t)rows * nblk;
  auto run = [&](auto* gt) -> cudaError_t {
    using TE = std::remove_const_t<std::remove_pointer_t<decltype(gt)>>;
    const SwigluArgs<TE> a{gt, static_cast<const TE*>(u), static_cast<TE*>(h),
                           static_cast<uint2*>(h8.q), static_cast<uint2*>(g8.q),
                           static_cast<uint2*>(u8.q), h8.scale, g8.scale, u8.scale,
                           items, nblk, cols};
    auto kern = pow2 ? swiglu_f8_kernel<TE, true> : swiglu_f8_kernel<TE, false>;
    SMOE_LAUNCH(kern, ceil_div(items, kRowsGroups), kRowsThreads, 0, s, a);
    return cudaGetLastError();
  };
  return d.dtype == SMOE_F32 ? run(static_cast<const float*>(g))
                             : run(static_cast<const __nv_bfloat16*>(g));
}

cudaError_t launch_swiglu_grad_f8(const smoe_desc& d, int rows, int cols, const void* dh,
                                  const void* g8, const float* gs, const void* u8, const float* us,
                                  void* dg, void* du, void* h, cudaStream_t s) {
  const uint32_t nblk = ceil_div(cols, 128), items = (uint32_t)rows * nblk;
  auto run = [&](auto* dt) -> cudaError_t {
    using TE = std::remove_const_t<std::remove_pointer_t<decltype(dt)>>;
    const SwigluGradArgs<TE> a{dt, static_cast<const uint2*>(g8), static_cast<const uint2*>(u8), gs, us,
                               static_cast<TE*>(dg), static_cast<TE*>(du), static_cast<TE*>(h),
                               items, nblk, cols};
    SMOE_LAUNCH((swiglu_grad_f8_kernel<TE>), ceil_div(items, kRowsGroups), kRowsThreads, 0, s, a);
    return cudaGetLastError();
  };
  return d.dtype == SMOE_F32 ? run(static_cast<const float*>(dh))
                             : run(static_cast<const __nv_bfloat16*>(dh));
}

}  // namespace smoe
