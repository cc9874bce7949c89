// The experts' products and their gradients in fp32 layers, on the CUDA cores (the tensor cores'
// tf32 keeps 11 bits of an operand; large ones go to expert_planes.cu and expert_grad.cu):
//   kind 0  y[r, n] = sum_k x[r, k] w[e, n, k]            rows x n_out, over n_in
//   kind 1  dx[r, k] = sum_n dy[r, n] w[e, n, k] (twice)  rows x n_in, over n_out
//   kind 2  dw[e, n, k] = sum_r dy[r, n] x[r, k] (+ add)  n_out x n_in, over the rows
//
// Two forms. Where experts have few rows (kinds 0 and 1) the weights' stream from HBM is the
// work: up to eight rows of an expert are multiplied while each weight passes through registers
// once. Otherwise tiles of 64 x 128, 4 x 8 sums a thread, their operands through a ring of shared
// memory filled by asynchronous copies that run ahead across tiles, so that the short contractions of
// a weight gradient (an expert's rows) do not wait for memory tile by tile; FMAs bound it.
// Measured: 39 rows of 24 experts of 1000 to 1416 channels 23 us (4.8 TB/s of the weights that are
// touched); tiles at 39 TFLOP/s (8192 rows of 8 experts of 1024 to 2048 870 us, where planes take 232).
#include <algorithm>

#include "tc_common.cuh"

namespace smoe {
namespace {

struct F32Args {
  const float *a, *b, *a2, *b2, *add;
  float* out;
  const int32_t* expert_off;
  DeviceStatus* st;
  int E, TK, n_out, n_in;
  int slices;        // of the contraction (tiles): each slice's sums in a matrix of their own
  long long size;    // floats of such a matrix
};

// Row tiles of each expert (fixed > 0: that many for each; s_ts, prefix) and their first rows
// (s_off), by one warp. A bad expert_off schedules nothing.
__device__ __forceinline__ void f32_table(const F32Args& p, int rows_per_tile, int fixed, int32_t* s_ts,
                                          int32_t* s_off, int lane) {
  bool bad = false;
  for (int g = lane; g <= p.E; g += 32) {
    const int lo = p.expert_off[g], hi = g < p.E ? p.expert_off[g + 1] : lo;
    bad |= lo < 0 || hi < lo || hi > p.TK;
    s_off[g] = lo;
  }
  bad = __any_sync(0xffffffffu, bad);
  if (bad && lane == 0) record_error(p.st, kStatusData, kBadPairRow, -1);
  __syncwarp();
  int carry = 0;
  for (int g0 = 0; g0 < p.E; g0 += 32) {
    const int g = g0 + lane;
    int n = 0;
    if (!bad && g < p.E) n = fixed ? fixed : (s_off[g + 1] - s_off[g] + rows_per_tile - 1) / rows_per_tile;
    int incl = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    if (g < p.E) s_ts[g] = carry + incl - n;
    carry += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) s_ts[p.E] = carry;
}

// ------------------------------------------------------------------ few rows
constexpr int kFewRows = 8;      // rows of an expert that pass together
constexpr int kFewChan = 4;      // kind 0: channels of a warp at a time

__device__ __forceinline__ float dot4(const float4& a, const float4& b, float c) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}

// Kind 0: a warp takes four channels of an expert and its next R rows; the lanes share the
// contraction, 16 bytes each, and their sums meet by shuffles.
template <int R>
__device__ __forceinline__ void few_dot(const F32Args& p, int g, int row0, int rows, int n0, int lane) {
  float acc[R][kFewChan];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < kFewChan; ++c) acc[r][c] = 0.0f;
  const float* w = p.b + ((size_t)g * p.n_out + n0) * p.n_in;
  const float* x = p.a + (size_t)row0 * p.n_in;
#pragma unroll 2
  for (int k = lane * 4; k < p.n_in; k += 128) {
    float4 wv[kFewChan], xv[R];
#pragma unroll
    for (int c = 0; c < kFewChan; ++c) wv[c] = __ldcs(reinterpret_cast<const float4*>(w + (size_t)c * p.n_in + k));
#pragma unroll
    for (int r = 0; r < R; ++r) xv[r] = *reinterpret_cast<const float4*>(x + (size_t)min(r, rows - 1) * p.n_in + k);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < kFewChan; ++c) acc[r][c] = dot4(wv[c], xv[r], acc[r][c]);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int c = 0; c < kFewChan; ++c)
#pragma unroll
      for (int off = 16; off; off >>= 1) acc[r][c] += __shfl_xor_sync(0xffffffffu, acc[r][c], off);
    if (lane == 0 && r < rows)
      *reinterpret_cast<float4*>(p.out + (size_t)(row0 + r) * p.n_out + n0) =
          make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
  }
}

// (two blocks an SM: 39 rows of 24 experts of 1000 x 1416 23 us, one 31, three 27)
__global__ void __launch_bounds__(256, 2)
few_rows_kernel(const F32Args p) {
  __shared__ int32_t s_ts[kMaxGroups + 2], s_off[kMaxGroups + 2];
  pdl_wait_and_trigger();
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < 32) f32_table(p, kFewRows, 0, s_ts, s_off, lane);
  __syncthreads();
  const int nchan = p.n_out / kFewChan;
  const long long total = (long long)s_ts[p.E] * nchan;
  int g = 0;
  for (long long u = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); u < total; u += (long long)gridDim.x * 8) {
    while ((long long)s_ts[g + 1] * nchan <= u) ++g;
    // an expert's row passes follow one another for the same channels
    const int mt = s_ts[g + 1] - s_ts[g], local = (int)(u - (long long)s_ts[g] * nchan);
    const int n0 = local / mt * kFewChan, m0 = local % mt * kFewRows;
    const int row0 = s_off[g] + m0, rows = min(kFewRows, s_off[g + 1] - row0);
    if (rows == 1) few_dot<1>(p, g, row0, rows, n0, lane);
    else if (rows == 2) few_dot<2>(p, g, row0, rows, n0, lane);
    else if (rows <= 4) few_dot<4>(p, g, row0, rows, n0, lane);
    else few_dot<8>(p, g, row0, rows, n0, lane);
  }
}

// Kind 1: a block takes 128 columns of an expert's matrix and its next rows; each lane four
// columns, each warp every eighth matrix row, whose factors dy (all rows' side by side) come from
// shared memory; the warps' sums meet there too.
constexpr int kFewN = 512;  // matrix rows between two fills of shared memory

// Two blocks an SM, eight loads of a lane ahead. (Without the loads ahead and three blocks an SM: 128
// rows of 8 experts of 256 x 128, both pairs, 13.7 us, against 10.3; 39 of 24 of 1416 x 1000 41,
// against 30; 260 of 76 of 1392 x 304, both pairs, 101, against 68; but 216 of 152 of 936 x 432 42,
// against 49.)
__global__ void __launch_bounds__(256, 2)
few_rows_t_kernel(const F32Args p) {
  __shared__ int32_t s_ts[kMaxGroups + 2], s_off[kMaxGroups + 2];
  __shared__ alignas(16) float s_dy[kFewN][kFewRows];
  __shared__ alignas(16) float s_sum[8][4][128];
  pdl_wait_and_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < 32) f32_table(p, kFewRows, 0, s_ts, s_off, lane);
  __syncthreads();
  const int ntile = (p.n_in + 127) / 128;
  const int total = s_ts[p.E] * ntile;
  int g = 0;
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    while (s_ts[g + 1] * ntile <= u) ++g;
    const int mt = s_ts[g + 1] - s_ts[g], local = u - s_ts[g] * ntile;
    const int col = local / mt * 128 + lane * 4, m0 = local % mt * kFewRows;
    const int row0 = s_off[g] + m0, rows = min(kFewRows, s_off[g + 1] - row0);
    const bool in = col < p.n_in;
    float4 acc[kFewRows];
#pragma unroll
    for (int r = 0; r < kFewRows; ++r) acc[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int pair = 0; pair < (p.a2 ? 2 : 1); ++pair) {
      const float* dy = (pair ? p.a2 : p.a) + (size_t)row0 * p.n_out;
      const float* w = (pair ? p.b2 : p.b) + (size_t)g * p.n_out * p.n_in + (in ? col : 0);
      for (int n0 = 0; n0 < p.n_out; n0 += kFewN) {
        const int nn = min(kFewN, p.n_out - n0);
        // the next eight matrix rows are on their way while these are multiplied, the first ones
        // while dy is laid out
        float4 wv[2][8];
        auto fetch = [&](int n, float4 (&v)[8]) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            v[j] = in && n + 8 * j < nn ? __ldcs(reinterpret_cast<const float4*>(w + (size_t)(n0 + n + 8 * j) * p.n_in))
                                        : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        };
        auto multiply = [&](int n, const float4 (&v)[8]) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (n + 8 * j >= nn) break;
            const float* at = &s_dy[n + 8 * j][0];
            float f[kFewRows];
            *reinterpret_cast<float4*>(f) = *reinterpret_cast<const float4*>(at);
            if (rows > 4) *reinterpret_cast<float4*>(f + 4) = *reinterpret_cast<const float4*>(at + 4);
#pragma unroll
            for (int r = 0; r < kFewRows; ++r) {
              if (r >= 4 && rows <= 4) break;
              acc[r].x = fmaf(f[r], v[j].x, acc[r].x);
              acc[r].y = fmaf(f[r], v[j].y, acc[r].y);
              acc[r].z = fmaf(f[r], v[j].z, acc[r].z);
              acc[r].w = fmaf(f[r], v[j].w, acc[r].w);
            }
          }
        };
        fetch(warp, wv[0]);
        __syncthreads();
        {  // (all loads ahead of the stores)
          float f[kFewN / 256][kFewRows];
#pragma unroll
          for (int i = 0; i < kFewN / 256; ++i)
#pragma unroll
            for (int r = 0; r < kFewRows; ++r) {
              const int n = tid + 256 * i;
              f[i][r] = n < nn && r < rows ? dy[(size_t)r * p.n_out + n0 + n] : 0.0f;
            }
#pragma unroll
          for (int i = 0; i < kFewN / 256; ++i) {
            float4* to = reinterpret_cast<float4*>(&s_dy[tid + 256 * i][0]);
            to[0] = make_float4(f[i][0], f[i][1], f[i][2], f[i][3]);
            to[1] = make_float4(f[i][4], f[i][5], f[i][6], f[i][7]);
          }
        }
        __syncthreads();
        for (int n = warp; n < nn; n += 128) {
          fetch(n + 64, wv[1]);
          multiply(n, wv[0]);
          if (n + 64 >= nn) break;
          fetch(n + 128, wv[0]);
          multiply(n + 64, wv[1]);
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // four rows at a time
      if (4 * h >= rows) break;
      __syncthreads();
#pragma unroll
      for (int r = 0; r < 4; ++r) *reinterpret_cast<float4*>(&s_sum[warp][r][lane * 4]) = acc[4 * h + r];
      __syncthreads();
      const int r = tid >> 6, c = (tid & 63) * 2, c0 = local / mt * 128;
      if (4 * h + r < rows && c0 + c < p.n_in) {
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 v = *reinterpret_cast<const float2*>(&s_sum[k][r][c]);
          sum.x += v.x;
          sum.y += v.y;
        }
        *reinterpret_cast<float2*>(p.out + (size_t)(row0 + 4 * h + r) * p.n_in + c0 + c) = sum;
      }
    }
  }
}

// ------------------------------------------------------------------ tiles
constexpr int kBM = 64, kBN = 128, kBK = 16, kRing = 4;
// An operand contiguous along the contraction is staged row by row (pitch 20 floats), one
// contiguous across it as it lies: reads of 16 bytes without bank conflicts either way.
constexpr int kPitchK = kBK + 4;
template <int KIND>
struct TileSmem {
  static constexpr int kA = KIND == 2 ? kBK * (kBM + 4) : kBM * kPitchK;
  static constexpr int kB = KIND == 0 ? kBN * kPitchK : kBK * (kBN + 4);
  static constexpr size_t kBytes = (size_t)kRing * (kA + kB) * 4 + 8 * (kMaxGroups + 2);
};

struct F32Tile {
  int g, m0, n0, row0, M, K1, nk1, nk;
  int k0, slice;     // the slice's first stage, and its number
};

template <int KIND>
__device__ __forceinline__ F32Tile f32_decode(const F32Args& p, const int32_t* ts, const int32_t* off,
                                              int ntile, int t, int& g) {
  const int slice = t % p.slices;
  t /= p.slices;
  while (ts[g + 1] * ntile <= t) ++g;
  const int mt = ts[g + 1] - ts[g], local = t - ts[g] * ntile;
  const int n_tile = local / mt;
  F32Tile r;
  r.g = g;
  r.n0 = n_tile * kBN;
  r.m0 = (local - n_tile * mt) * kBM;
  r.row0 = off[g];
  const int rows = off[g + 1] - off[g];
  r.M = KIND == 2 ? p.n_out : rows;
  r.K1 = KIND == 0 ? p.n_in : KIND == 1 ? p.n_out : rows;
  r.nk1 = (r.K1 + kBK - 1) / kBK;
  const int nk = KIND == 1 && p.a2 ? 2 * r.nk1 : r.nk1, step = (nk + p.slices - 1) / p.slices;
  r.slice = slice;
  r.k0 = min(nk, slice * step);
  r.nk = min(nk - r.k0, step);
  return r;
}

template <int KIND>
__global__ void __launch_bounds__(256, 3)
tiled_f32_kernel(const F32Args p) {
  using S = TileSmem<KIND>;
  extern __shared__ __align__(16) float smem[];
  float* sA = smem;
  float* sB = sA + kRing * S::kA;
  int32_t* s_ts = reinterpret_cast<int32_t*>(sB + kRing * S::kB);
  int32_t* s_off = s_ts + kMaxGroups + 2;
  pdl_wait_and_trigger();
  const int tid = threadIdx.x;
  if (tid < 32) f32_table(p, kBM, KIND == 2 ? (p.n_out + kBM - 1) / kBM : 0, s_ts, s_off, tid);
  __syncthreads();
  const int N = KIND == 0 ? p.n_out : p.n_in, ntile = (N + kBN - 1) / kBN;
  const int total = s_ts[p.E] * ntile * p.slices;
  const int tx = tid & 15, ty = tid >> 4;  // columns tx * 4 + {0, 64}; rows ty * 4 + {0 .. 3}

  // the copies' own walk over (tile, 16 of the contraction), ahead of the sums'
  int lt = blockIdx.x, lg = 0, lk = 0, lslot = 0;
  F32Tile ld{};
  bool fresh = true;
  auto copy_next = [&] {
    while (lt < total) {
      if (fresh) {
        ld = f32_decode<KIND>(p, s_ts, s_off, ntile, lt, lg);
        fresh = false;
        lk = 0;
      }
      if (lk < ld.nk) break;
      lt += gridDim.x;
      fresh = true;
    }
    if (lt < total) {
      const bool second = ld.k0 + lk >= ld.nk1;
      const float* a = second ? p.a2 : p.a;
      const float* b = second ? p.b2 : p.b;
      const int k0 = (ld.k0 + lk - (second ? ld.nk1 : 0)) * kBK;
      {
        const float* from = a;
        bool in;
        float* to = sA + lslot * S::kA;
        if (KIND == 2) {  // [row][n_out]
          const int k = tid >> 4, m = (tid & 15) * 4;
          in = k0 + k < ld.K1 && ld.m0 + m < ld.M;
          if (in) from = a + (size_t)(ld.row0 + k0 + k) * p.n_out + ld.m0 + m;
          to += k * (kBM + 4) + m;
        } else {
          const int m = tid >> 2, k = (tid & 3) * 4;
          in = ld.m0 + m < ld.M && k0 + k < ld.K1;
          if (in) from = a + (size_t)(ld.row0 + ld.m0 + m) * ld.K1 + k0 + k;
          to += m * kPitchK + k;
        }
        tc::cp_async16(tc::smem_u32(to), from, in ? 16u : 0u);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int v = tid + i * 256;
        const float* from = b;
        bool in;
        float* to = sB + lslot * S::kB;
        if (KIND == 0) {  // [n_out][n_in]
          const int n = v >> 2, k = (v & 3) * 4;
          in = ld.n0 + n < N && k0 + k < ld.K1;
          if (in) from = b + ((size_t)ld.g * p.n_out + ld.n0 + n) * p.n_in + k0 + k;
          to += n * kPitchK + k;
        } else {
          const int k = v >> 5, n = (v & 31) * 4;
          in = k0 + k < ld.K1 && ld.n0 + n < N;
          const size_t row = KIND == 1 ? (size_t)ld.g * p.n_out + k0 + k : (size_t)ld.row0 + k0 + k;
          if (in) from = b + row * p.n_in + ld.n0 + n;
          to += k * (kBN + 4) + n;
        }
        tc::cp_async16(tc::smem_u32(to), from, in ? 16u : 0u);
      }
      ++lk;
      if (++lslot == kRing) lslot = 0;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) copy_next();

  int g = 0, slot = 0;
  for (int t = blockIdx.x; t < total; t += gridDim.x) {
    const F32Tile tl = f32_decode<KIND>(p, s_ts, s_off, ntile, t, g);
    float acc[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
    for (int kb = 0; kb < tl.nk; ++kb) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
      __syncthreads();  // this stage has landed, the one before it has been read by all
      copy_next();
      const float* A = sA + slot * S::kA;
      const float* B = sB + slot * S::kB;
      if (++slot == kRing) slot = 0;
#pragma unroll
      for (int k = 0; k < kBK; k += 4) {
        if (KIND == 2 && (tl.k0 + kb) * kBK + k >= tl.K1) break;  // short contractions end inside a stage
        float a[4][4], b[4][8];  // [k][row], [k][column]
        if (KIND == 2) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const float4 f = *reinterpret_cast<const float4*>(A + (k + kk) * (kBM + 4) + ty * 4);
            a[kk][0] = f.x; a[kk][1] = f.y; a[kk][2] = f.z; a[kk][3] = f.w;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 f = *reinterpret_cast<const float4*>(A + (ty * 4 + i) * kPitchK + k);
            a[0][i] = f.x; a[1][i] = f.y; a[2][i] = f.z; a[3][i] = f.w;
          }
        }
        if (KIND == 0) {
          // (columns tx + 16 j: neighbouring lanes read neighbouring rows of the stage)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 f = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * kPitchK + k);
            b[0][j] = f.x; b[1][j] = f.y; b[2][j] = f.z; b[3][j] = f.w;
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float4 f = *reinterpret_cast<const float4*>(B + (k + kk) * (kBN + 4) + tx * 4 + 64 * j);
              b[kk][4 * j] = f.x; b[kk][4 * j + 1] = f.y; b[kk][4 * j + 2] = f.z; b[kk][4 * j + 3] = f.w;
            }
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[i][j] = fmaf(a[kk][i], b[kk][j], acc[i][j]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = tl.m0 + ty * 4 + i;
      if (m >= tl.M) continue;
      float* out = p.out + tl.slice * p.size + ((KIND == 2 ? (size_t)tl.g * p.n_out : (size_t)tl.row0) + m) * N;
      if (KIND == 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int n = tl.n0 + tx + 16 * j;
          if (n < N) out[n] = acc[i][j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int n = tl.n0 + tx * 4 + 64 * j;
          if (n >= N) continue;
          float4 o = make_float4(acc[i][4 * j], acc[i][4 * j + 1], acc[i][4 * j + 2], acc[i][4 * j + 3]);
          if (KIND == 2 && p.add) {
            const float4 f = *reinterpret_cast<const float4*>(p.add + (out - p.out) + n);
            o.x += f.x; o.y += f.y; o.z += f.z; o.w += f.w;
          }
          *reinterpret_cast<float4*>(out + n) = o;
        }
      }
    }
  }
  tc::cp_async_wait_all();
}

template <int KIND>
cudaError_t run_tiled(F32Args p, long long tiles, long long stages, void* ws, const ProductLayout& L,
                      cudaStream_t s) {
  // (500 rows of one expert, 5120 to 256 channels: one slice 377 us)
  const int row_len = KIND == 0 ? p.n_out : p.n_in;
  const long long rows = KIND == 2 ? (long long)p.E * p.n_out : p.TK;
  p.size = rows * row_len;
  p.slices = slices_of(tiles, device_sms() * 3LL, stages / 4, p.size);
  float* const out = p.out;
  const float* const add = p.add;
  if (p.slices > 1) {
    p.out = ws_ptr<float>(ws, L.parts);
    p.add = nullptr;
  }

  auto kern = tiled_f32_kernel<KIND>;
  const int smem = (int)TileSmem<KIND>::kBytes;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int grid = (int)std::min<long long>(std::max<long long>(tiles * p.slices, 1), (long long)device_sms() * 3);
  SMOE_LAUNCH(kern, grid, 256, smem, s, p);
  if (p.slices == 1) return cudaGetLastError();
  return launch_sum_slices(p.out, p.slices, rows, row_len, KIND != 2, p.expert_off, p.E, p.TK, add, out, s);
}

// Rows an expert on average from which the tiles take over. Measured (us, tiles and streaming): 24
// experts of 1000 to 1416 channels, 8 rows: 188 and 54, 24: 189 and 115, 48: 192 and 202; their row
// gradients 24: 175 and 99, 48: 244 and 173; 8 experts of 2048 to 1024, 48: 153 and 88, and 122
// and 75.
constexpr int kTileRows = 56;
// ... and from which, with so many multiply-adds, products of bf16 planes on the tensor cores
// (expert_planes.cu) do, the planes' making included. Measured (us, planes and CUDA cores): 24 experts
// of 1000 to 1416, 32 rows: 164 and 139, 64: 167 and 197, 256: 224 and 580, 1024: 517 and 2024; 8 of
// 2048 to 1024, 64: 87 and 134, 1024: 232 and 994; 4 of 512 to 512, 128: 24 and 21, 256: 26 and 30,
// 1024: 33 and 99; one of 5120 to 256, 64: 27 and 32, 1024: 43 and 84; row gradients alike.
constexpr int kPlaneRows = kPlaneRowsMin;
constexpr double kPlaneMacs = 1.5e8;

}  // namespace

cudaError_t launch_expert_rows_f32(const smoe_desc& d, int n_out, int n_in, const float* a,
                                   const float* w, const float* a2, const float* w2, bool transposed,
                                   const int32_t* expert_off, float* out, void* ws, cudaStream_t s) {
  ProductLayout L;
  product_ws_layout(d, &L);
  const int TK = d.T * d.K;
  const F32Args p{a, w, a2, w2, nullptr, out, expert_off, ws_ptr<DeviceStatus>(ws, L.status), d.E, TK, n_out, n_in, 1, 0};
  if (has_weight_planes(d) && n_out <= std::max(d.d, d.F) && n_in <= std::max(d.d, d.F) &&
      (long long)n_out * n_in <= (long long)d.d * d.F && 3LL * TK < 1LL << 30 &&
      (long long)TK >= (long long)kPlaneRows * d.E && (double)TK * n_out * n_in * (a2 ? 2 : 1) >= kPlaneMacs)
    return launch_expert_rows_planes(d, n_out, n_in, a, w, a2, w2, transposed, expert_off, out, ws, s);
  if ((long long)TK >= (long long)kTileRows * d.E) {
    const long long tiles = ((long long)ceil_div(TK, kBM) + std::min(TK, d.E)) * ceil_div(transposed ? n_in : n_out, kBN);
    return transposed ? run_tiled<1>(p, tiles, ceil_div(n_out, kBK) * (a2 ? 2 : 1), ws, L, s)
                      : run_tiled<0>(p, tiles, ceil_div(n_in, kBK), ws, L, s);
  }
  const long long passes = (long long)ceil_div(TK, kFewRows) + std::min(TK, d.E), most = (long long)device_sms() * 4;
  if (transposed) {
    SMOE_LAUNCH(few_rows_t_kernel, (int)std::min(most, passes * ceil_div(n_in, 128)), 256, 0, s, p);
  } else {
    SMOE_LAUNCH(few_rows_kernel, (int)std::min(most, (passes * (n_out / kFewChan) + 7) / 8), 256, 0, s, p);
  }
  return cudaGetLastError();
}

cudaError_t launch_expert_dw_f32(const smoe_desc& d, int n_out, int n_in, const float* dy,
                                 const float* x, const int32_t* expert_off, const float* add, float* dw,
                                 void* ws, cudaStream_t s) {
  ProductLayout L;
  product_ws_layout(d, &L);
  const int TK = d.T * d.K;
  const F32Args p{dy, x, nullptr, nullptr, add, dw, expert_off, ws_ptr<DeviceStatus>(ws, L.status), d.E, TK, n_out, n_in, 1, 0};
  return run_tiled<2>(p, (long long)d.E * ceil_div(n_out, kBM) * ceil_div(n_in, kBN), TK / d.E / kBK, ws, L, s);
}

}  // namespace smoe
