// Expert products in 8-bit integers with a scale per row (token) and per output channel:
//   out[r, n] = xs[r] ws[e(r), n] sum_k xq[r, k] wq[e(r), n, k],
// and the SwiGLU FFN made of three of them, its hidden rows requantised in between.
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "smoe_internal.cuh"

namespace smoe {
namespace {

constexpr int kRows = 64, kCols = 64;  // output tile of a block
constexpr int kStep = 64;              // contraction bytes per step

// Group g < E: rows expert_off[g] .. expert_off[g+1]; group E + j: shared expert j, T rows.
// tile_start[g] = first row tile of group g. A bad expert_off schedules nothing.
__global__ void i8_tiles_kernel(const int32_t* __restrict__ expert_off, int E, int n_shared, int T,
                                int TK, int bm, int32_t* __restrict__ tile_start, DeviceStatus* st) {
  pdl_wait_and_trigger();
  const int lane = threadIdx.x, G = E + n_shared;
  bool bad = false;
  for (int g = lane; g < E; g += 32) {
    const int lo = expert_off[g], hi = expert_off[g + 1];
    bad |= lo < 0 || hi < lo || hi > TK;
  }
  bad = __any_sync(0xffffffffu, bad);
  if (bad && lane == 0) record_error(st, kStatusData, kBadPairRow, -1);
  int carry = 0;
  for (int g0 = 0; g0 < G; g0 += 32) {
    const int g = g0 + lane;
    int rows = 0;
    if (!bad && g < E) rows = expert_off[g + 1] - expert_off[g];
    else if (!bad && g < G) rows = T;
    const int n = (rows + bm - 1) / bm;
    int incl = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    if (g < G) tile_start[g] = carry + incl - n;
    carry += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) tile_start[G] = carry;
}

struct I8Args {
  const int8_t* x;            // rows: [n_src, KD] (read through map), or [TK (+ S T), KD]
  const float* xs;            // [n_src] or [TK (+ S T)]
  const int32_t* map;         // nullable: source row of each dispatched row
  const int32_t* expert_off;
  const int32_t* tile_start;
  const int8_t *wa, *wb;      // [G, N, KD]; wb: the W3 of the up product
  const float *sa, *sb;       // [G, N]
  void* out;                  // routed rows [TK, N]; up: all rows [TK + S T, N] fp32
  void* out_sh;               // down: shared rows [S T, N]
  DeviceStatus* st;
  int E, G, T, TK, N, KD, n_src;
};

__device__ __forceinline__ float silu(float v) { return v / (1.0f + expf(-v)); }

template <bool UP, typename TO>
__global__ void __launch_bounds__(256)
i8_product_kernel(const I8Args p) {
  pdl_wait_and_trigger();
  __shared__ int sx[kRows][kStep / 4 + 1], sw[UP ? 2 : 1][kCols][kStep / 4 + 1];
  __shared__ int s_src[kRows];
  const int total = p.tile_start[p.G];
  for (int t = blockIdx.y; t < total; t += gridDim.y) {
    int lo = 0, hi = p.G - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.tile_start[mid] <= t) lo = mid; else hi = mid - 1;
    }
    const int g = lo, r0 = (t - p.tile_start[g]) * kRows, n0 = blockIdx.x * kCols;
    const bool shared = g >= p.E;
    const int first = shared ? 0 : p.expert_off[g];
    const int rows = shared ? p.T : p.expert_off[g + 1] - first;
    // rows of the operand and of the output: shared expert j's follow the T K routed ones
    const long long orow = (shared ? (long long)p.TK + (long long)(g - p.E) * p.T : first) + r0;
    __syncthreads();
    if (threadIdx.x < kRows) {
      int src = -1;
      if (r0 + (int)threadIdx.x < rows) {
        if (p.map || (shared && UP)) {  // the tokens' rows
          src = shared ? r0 + threadIdx.x : p.map[orow + threadIdx.x];
          if ((unsigned)src >= (unsigned)p.n_src) {
            record_error(p.st, kStatusData, kBadPerm, orow + threadIdx.x);
            src = -1;
          }
        } else {
          src = (int)(orow + threadIdx.x);
        }
      }
      s_src[threadIdx.x] = src;
    }
    int acc[UP ? 2 : 1][4][4] = {};
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int k0 = 0; k0 < p.KD; k0 += kStep) {
      __syncthreads();
      for (int i = threadIdx.x; i < kRows * (kStep / 4); i += 256) {
        const int rr = i / (kStep / 4), kk = i % (kStep / 4);
        const bool in = k0 + 4 * kk < p.KD;
        sx[rr][kk] = in && s_src[rr] >= 0
                         ? *reinterpret_cast<const int*>(p.x + (size_t)s_src[rr] * p.KD + k0 + 4 * kk)
                         : 0;
        const bool inw = in && n0 + rr < p.N;
        const size_t wo = ((size_t)g * p.N + n0 + rr) * p.KD + k0 + 4 * kk;
        sw[0][rr][kk] = inw ? *reinterpret_cast<const int*>(p.wa + wo) : 0;
        if (UP) sw[1][rr][kk] = inw ? *reinterpret_cast<const int*>(p.wb + wo) : 0;
      }
      __syncthreads();
#pragma unroll 4
      for (int kk = 0; kk < kStep / 4; ++kk)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[0][i][j] = __dp4a(sx[ty + 16 * i][kk], sw[0][tx + 16 * j][kk], acc[0][i][j]);
            if (UP) acc[UP][i][j] = __dp4a(sx[ty + 16 * i][kk], sw[UP][tx + 16 * j][kk], acc[UP][i][j]);
          }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int rr = ty + 16 * i;
      if (r0 + rr >= rows) continue;
      const float xs = s_src[rr] >= 0 ? p.xs[s_src[rr]] : 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + tx + 16 * j;
        if (n >= p.N) continue;
        float v = (float)acc[0][i][j] * xs * p.sa[(size_t)g * p.N + n];
        if (UP) v = silu(v) * ((float)acc[UP][i][j] * xs * p.sb[(size_t)g * p.N + n]);
        TO* out = static_cast<TO*>(!UP && shared ? p.out_sh : p.out);
        const long long ro = !UP && shared ? orow - p.TK : orow;
        out[(size_t)(ro + rr) * p.N + n] = Elem<TO>::from_f32(v);
      }
    }
  }
}

// hq = rint(h / s), s = max |h| / 127 of the row (0 for a row that is zero or whose scale
// would be subnormal, NaN for a row that is not finite).
__global__ void __launch_bounds__(256)
i8_quantise_rows_kernel(const float* __restrict__ h, int8_t* __restrict__ q, float* __restrict__ s,
                        int rows, int F) {
  pdl_wait_and_trigger();
  __shared__ uint32_t red[8];
  for (int r = blockIdx.x; r < rows; r += gridDim.x) {
    const float* row = h + (size_t)r * F;
    uint32_t big = 0;
    for (int i = threadIdx.x; i < F; i += 256) big = max(big, __float_as_uint(row[i]) & 0x7fffffffu);
    big = __reduce_max_sync(0xffffffffu, big);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = big;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) big = max(big, red[w]);
    const float amax = __uint_as_float(big);
    const bool finite = amax <= FLT_MAX;
    float scale = amax / 127.0f;
    const bool zero = !finite || scale < FLT_MIN;
    if (zero) scale = finite ? 0.0f : __int_as_float(0x7fc00000);
    if (threadIdx.x == 0) s[r] = scale;
    for (int i = threadIdx.x; i < F; i += 256)
      q[(size_t)r * F + i] = zero ? (int8_t)0 : (int8_t)__float2int_rn(row[i] / scale);
  }
}

template <bool UP, typename TO>
cudaError_t run_product(const I8Args& p, int n_shared, cudaStream_t s) {
  const long long bound = (long long)ceil_div(p.TK, kRows) + p.E + (long long)n_shared * ceil_div(p.T, kRows);
  SMOE_LAUNCH((i8_product_kernel<UP, TO>), dim3(ceil_div(p.N, kCols), (int)std::min(bound, 32768LL)), 256, 0, s, p);
  return cudaGetLastError();
}

}  // namespace

void i8_ws_layout(const smoe_desc& d, I8Layout* L) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) / 256 * 256;
    return o;
  };
  const size_t rows = (size_t)d.T * d.K + (size_t)d.n_shared * d.T;
  L->status = take(256);
  L->tiles = take(4 * ((size_t)d.E + d.n_shared + 1));
  L->h = take(rows * d.F * 4);
  L->hq = take(rows * d.F);
  L->hs = take(rows * 4);
  L->total = off;
}

cudaError_t launch_expert_matmul_i8(const smoe_desc& d, int n_out, int n_in, const int8_t* xq,
                                    const float* xs, const int32_t* row_src,
                                    const int32_t* expert_off, const int8_t* wq, const float* ws_n,
                                    void* out, void* ws, cudaStream_t s) {
  I8Layout L;
  i8_ws_layout(d, &L);
  int32_t* tiles = ws_ptr<int32_t>(ws, L.tiles);
  DeviceStatus* st = ws_ptr<DeviceStatus>(ws, L.status);
  const int TK = d.T * d.K;
  SMOE_LAUNCH(i8_tiles_kernel, 1, 32, 0, s, expert_off, d.E, 0, d.T, TK, kRows, tiles, st);
  const I8Args p{xq, xs, row_src, expert_off, tiles, wq, nullptr, ws_n, nullptr, out, nullptr, st,
                 d.E, d.E, d.T, TK, n_out, n_in, row_src ? d.T : TK};
  return d.dtype == SMOE_F32 ? run_product<false, float>(p, 0, s)
                             : run_product<false, __nv_bfloat16>(p, 0, s);
}

cudaError_t launch_expert_ffn_i8(const smoe_desc& d, const int8_t* xq, const float* xs,
                                 const int32_t* row_src, const int32_t* expert_off,
                                 const smoe_i8_weights& W, void* y_disp, void* y_sh, void* ws,
                                 cudaStream_t s) {
  I8Layout L;
  i8_ws_layout(d, &L);
  int32_t* tiles = ws_ptr<int32_t>(ws, L.tiles);
  DeviceStatus* st = ws_ptr<DeviceStatus>(ws, L.status);
  const int TK = d.T * d.K, G = d.E + d.n_shared, rows = TK + d.n_shared * d.T;
  float* h = ws_ptr<float>(ws, L.h);
  int8_t* hq = ws_ptr<int8_t>(ws, L.hq);
  float* hs = ws_ptr<float>(ws, L.hs);
  SMOE_LAUNCH(i8_tiles_kernel, 1, 32, 0, s, expert_off, d.E, d.n_shared, d.T, TK, kRows, tiles, st);
  const I8Args up{xq, xs, row_src, expert_off, tiles, W.w1, W.w3, W.s1, W.s3, h, nullptr, st,
                  d.E, G, d.T, TK, d.F, d.d, row_src ? d.T : TK};
  cudaError_t e = run_product<true, float>(up, d.n_shared, s);
  if (e != cudaSuccess) return e;
  SMOE_LAUNCH(i8_quantise_rows_kernel, std::min(rows, 4096), 256, 0, s, h, hq, hs, rows, d.F);
  const I8Args dn{hq, hs, nullptr, expert_off, tiles, W.w2, nullptr, W.s2, nullptr, y_disp, y_sh,
                  st, d.E, G, d.T, TK, d.d, d.F, rows};
  return d.dtype == SMOE_F32 ? run_product<false, float>(dn, d.n_shared, s)
                             : run_product<false, __nv_bfloat16>(dn, d.n_shared, s);
}

}  // namespace smoe
