// Root-mean-square norm of the residual stream with the layer output's addition, in front
// of the router and the expert products:
//   h = r + y,   n = (h gamma) rsqrt(mean(h^2) + eps),
//   q = rint(n / s), s = max |n| / 127 (one scale per row).
// Each element is read once and every output written once: 4 + b bytes in and up to
// 4 + b + 1 out per element (b = bytes of the layer's dtype), so HBM is the bound. A row
// lives in registers between its loads and its stores; the sum of squares and the largest
// |h gamma| come from one pass over them and one block reduction, because rounding is
// monotonic: max over fl(fl(h gamma) rs) is fl(max |fl(h gamma)| rs).
#include <algorithm>
#include <cfloat>

#include "smoe_internal.cuh"

namespace smoe {
namespace {

// Rows of at most 1024 elements take one warp each (8 rows per block), longer ones a block.
constexpr int kWarpRowMax = 1024;

// An eps below this does not hide what a sum of squares below it has lost to underflow: such
// calls take a form of the kernel with a second pass over such rows (kNoEps). In every call its
// registers would cost 8192 rows of 5120 134 us, against 85.
constexpr float kNoEpsBelow = 0x1p-100f;

struct NormArgs {
  const float* r;
  const void* y;       // nullable
  const float* gamma;
  float* r_out;        // nullable
  void* x_out;         // nullable
  int8_t* q_out;       // nullable, with q_scale
  float* q_scale;
  int T, d;
  float eps;
};

// 8 consecutive elements as fp32
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

// One row per group of kThreads threads (a warp or the block); thread i holds the 8-element
// chunks i, i + kThreads, ... of it.
template <typename TE, int kChunks, bool kWarp, bool kNoEps>
__global__ void __launch_bounds__(1024)
add_rmsnorm_kernel(const NormArgs p) {
  pdl_wait_and_trigger();
  __shared__ float s_sum[32];
  __shared__ uint32_t s_max[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nthr = kWarp ? 32 : (int)blockDim.x, me = kWarp ? lane : (int)threadIdx.x;
  const int rows_per_block = kWarp ? (int)blockDim.x >> 5 : 1;
  const int nchunk = p.d >> 3;
  for (long long row = (long long)blockIdx.x * rows_per_block + (kWarp ? warp : 0); row < p.T;
       row += (long long)gridDim.x * rows_per_block) {
    const size_t base = (size_t)row * p.d;
    float h[kChunks][8];
    float sum, eps = p.eps, up = 1.0f;
    uint32_t big;
    const float* r = p.r;
    const void* y = p.y;
    // kNoEps: a row whose squares fp32 holds with few bits or not at all is taken twice, the
    // second time 2^100 times as large, which is exact (its values are below 2^-50). r_out has
    // been written by then and is read back, as it may be r.
#pragma unroll 1
    for (;;) {
      sum = 0.0f;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int ch = me + c * nthr;
        if (ch >= nchunk) continue;
        load8(r + base + ch * 8, h[c]);
        if (y) {
          float v[8];
          load8(static_cast<const TE*>(y) + base + ch * 8, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[c][i] += v[i];
        }
      }
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int ch = me + c * nthr;
        if (ch >= nchunk) continue;
        if (p.r_out && (!kNoEps || up == 1.0f)) store8(p.r_out + base + ch * 8, h[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (kNoEps) h[c][i] *= up;
          sum = fmaf(h[c][i], h[c][i], sum);
        }
      }
      // |h gamma| is compared as an unsigned integer: the order of the magnitudes, and a NaN
      // is above every number, so a row that holds one does not pass for a finite row
      big = 0;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int ch = me + c * nthr;
        if (ch >= nchunk) continue;
        float g[8];
        load8(p.gamma + ch * 8, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          h[c][i] *= g[i];
          big = max(big, __float_as_uint(h[c][i]) & 0x7fffffffu);
        }
      }
#pragma unroll
      for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      big = __reduce_max_sync(0xffffffffu, big);
      if (!kWarp) {
        __syncthreads();  // the previous sums have been read
        if (lane == 0) {
          s_sum[warp] = sum;
          s_max[warp] = big;
        }
        __syncthreads();
        sum = 0.0f;
        for (int w = 0; w < (int)blockDim.x >> 5; ++w) {
          sum += s_sum[w];
          big = max(big, s_max[w]);
        }
      }
      if (!kNoEps || up != 1.0f || !(sum < kNoEpsBelow)) break;
      up = 0x1p100f;
      eps = eps * 0x1p100f * 0x1p100f;
      if (p.r_out) {
        r = p.r_out;
        y = nullptr;
      }
    }
    // (a row of zeros without an eps: zeros)
    const float mean = sum / (float)p.d + eps;
    const float rs = kNoEps && mean == 0.0f ? 0.0f : 1.0f / sqrtf(mean);
    const float amax = __uint_as_float(big) * rs;
    // a row whose scale would be subnormal counts as zero; a row with an infinity or a NaN
    // gets the scale NaN and zeros, so that what is computed from it shows it
    const bool finite = amax <= FLT_MAX && sum <= FLT_MAX;
    float scale = amax / 127.0f;
    const bool zero = !finite || scale < FLT_MIN;
    if (zero) scale = finite ? 0.0f : __int_as_float(0x7fc00000);
    if (p.q_out && me == 0) p.q_scale[row] = scale;
    // n / s as a product (its own rounding is below the norm's), rounded to an integer, ties
    // to even, by adding 1.5 * 2^23: the sum's low byte is the integer in two's complement.
    // (With a division and a conversion per element 8192 rows of 5120 took 95 us; now 87,
    // 6.3 TB/s.)
    const float inv = 1.0f / scale;
    constexpr float kRound = 12582912.0f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int ch = me + c * nthr;
      if (ch >= nchunk) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] *= rs;
      if (p.x_out) store8(static_cast<TE*>(p.x_out) + base + ch * 8, h[c]);
      if (p.q_out) {
        uint2 w = make_uint2(0u, 0u);
        if (!zero) {
          uint32_t b[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(fmaf(h[c][i], inv, kRound));
          w.x = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
          w.y = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
        }
        *reinterpret_cast<uint2*>(p.q_out + base + ch * 8) = w;
      }
    }
  }
}

template <typename TE, bool kNoEps>
cudaError_t run_norm(const NormArgs& p, cudaStream_t s) {
  const int nchunk = p.d >> 3;
  if (p.d <= kWarpRowMax) {
    const int grid = ceil_div(p.T, 8);
    if (nchunk <= 32) SMOE_LAUNCH((add_rmsnorm_kernel<TE, 1, true, kNoEps>), grid, 256, 0, s, p);
    else SMOE_LAUNCH((add_rmsnorm_kernel<TE, 4, true, kNoEps>), grid, 256, 0, s, p);
    return cudaGetLastError();
  }
  // one chunk a thread: 3.6 us for 64 rows of 5120, against 4.4 with two; two where a block
  // of one would pass 768 threads (4096 rows of 8192: 79 us, against 84)
  const int per = p.d <= 6144 ? 1 : 2;
  const int threads = (ceil_div(nchunk, per) + 31) / 32 * 32;
  if (per == 1) SMOE_LAUNCH((add_rmsnorm_kernel<TE, 1, false, kNoEps>), p.T, threads, 0, s, p);
  else SMOE_LAUNCH((add_rmsnorm_kernel<TE, 2, false, kNoEps>), p.T, threads, 0, s, p);
  return cudaGetLastError();
}

template <typename TE>
cudaError_t run_norm_t(const NormArgs& p, cudaStream_t s) {
  return p.eps < kNoEpsBelow ? run_norm<TE, true>(p, s) : run_norm<TE, false>(p, s);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const smoe_desc& d, const float* r, const void* y,
                               const float* gamma, float eps, float* r_out, void* x_out,
                               int8_t* q_out, float* q_scale, cudaStream_t s) {
  const NormArgs p{r, y, gamma, r_out, x_out, q_out, q_scale, d.T, d.d, eps};
  return d.dtype == SMOE_F32 ? run_norm_t<float>(p, s) : run_norm_t<__nv_bfloat16>(p, s);
}

}  // namespace smoe
