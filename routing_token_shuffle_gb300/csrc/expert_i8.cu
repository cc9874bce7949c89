// Expert products in 8-bit integers with a scale per row (token) and per output channel:
//   out[r, n] = xs[r] ws[e(r), n] sum_k xq[r, k] wq[e(r), n, k],
// and the SwiGLU FFN made of three of them, its hidden rows requantised in between.
//
// GB300's tensor cores have no fast 8-bit integer rate, but every int8 value is exact in
// fp16, every product of two is at most 2^14, and the accumulator is fp32: the fp16 products
// give the integer sum exactly while it stays within 2^24. So the rows are widened to fp16
// once (they are small), the weights travel and are staged as bytes (what bounds a decode
// batch is their stream from HBM) and are widened on the way into the tensor core: warps
// read the staged bytes, turn them into fp16 pairs (1.25 instructions a value: the byte with
// its sign bit flipped, under the exponent of 1024, is 1152 + value) and write them to
// TMEM, from where tcgen05.mma takes its A operand. Shared memory holds no widened copy.
//
// One persistent CTA per SM walks the tiles (group, 128-channel tile, row tile), row tiles
// fastest so that neighbours share the weights through L2:
//   warp 0      TMA: weight bytes (128 channels x 128)
//   warp 3      TMA: fp16 rows (NT rows x 128); or three warps gather them with 16-byte
//               asynchronous copies (see kGatherChannels) and warp 2 hands them over
//   warps 8-15  widen a weight stage into a TMEM operand stage
//   warp 1      tcgen05.mma, M = 128 channels (256 on a pair of CTAs), N = the tile's rows
//   warps 4-7   epilogue: scales, SwiGLU, stores (up: fp32 hidden rows and their largest
//               magnitude, by an integer atomicMax, whose result has no order)
// The up product's A tile is 64 channels of W1 and the same 64 of W3.
//
// Measured: 384 rows over 160 experts of 5120 x 1536 184 to 187 us (6.2 TB/s of weights); 131072
// rows of 2048 over 128 experts of 768 channels 326 us, 1.26 PFLOP/s of fp16; the FFN of 8192
// tokens (6 of 160 experts and two shared ones, 5120 x 1536) 2.26 to 2.4 ms with the clock that
// the power cap allows, 1.29 to 1.37 PFLOP/s; of 1001 tokens (2 of 8 experts of 4096 x 14336)
// 547 to 580 us, 1.22 to 1.29 PFLOP/s.
#include <algorithm>
#include <cfloat>
#include <cuda_fp16.h>

#include "tc_common.cuh"

namespace smoe {
namespace {

constexpr int kI8Threads = 512;
constexpr int kCopyWarps = 3;        // that gather rows: warp 3 and two more
constexpr int kStageW = 128 * 128;   // weight stage: 128 channels x 128 bytes
constexpr int kXchPitch = 20;        // floats: 16 of a thread; 16-byte accesses without bank conflicts
constexpr int kMaxGroupTab = 2 * (kMaxGroups + 2);

// NT: most rows of a tile. TMEM holds two accumulators of NT columns, then the widened
// operand stages (64 columns: 128 contraction values), kOp of them.
// 64: weight streaming. A deep weight ring; the rows of an operand stage (two 64-value
//     halves) sit beside it under the same barrier, so that the MMA warp waits once and
//     commits once per 128 values: with separate barriers for the halves it was the
//     bottleneck (1190 clocks a stage, against 780 at the HBM rate).
// 160, 192: batches whose experts fill them, on pairs of CTAs (a cluster on the two SMs of a
//     TPC): 256 channels, each CTA widening its own 128, and half of the rows in each CTA's
//     shared memory, in a ring of their own. One CTA alone moves 155 bytes a clock through
//     shared memory at the MMAs' rate (rows written and read, weight bytes written and
//     read), the pair 97; the limit is 128. 160 leaves TMEM for three operand stages, so
//     that widening does not wait for the MMAs of the stage before last; 192 issues fewer
//     MMAs a row (see kTallRows), and serves the gathering products, whose copies take as
//     long for fewer rows (328 us, against 347 with 160).
template <int NT> struct I8Cfg;
template <> struct I8Cfg<64> { static constexpr int kW = 8, kOp = 4, kB = 0, kRows = 64; };
template <> struct I8Cfg<160> { static constexpr int kW = 6, kOp = 3, kB = 5, kRows = 80; };
template <> struct I8Cfg<192> { static constexpr int kW = 6, kOp = 2, kB = 4, kRows = 96; };

template <int NT>
constexpr size_t i8_smem() {
  using C = I8Cfg<NT>;
  return 1024 + (size_t)C::kW * kStageW + (size_t)2 * (C::kB ? C::kB : C::kOp) * C::kRows * 128 +
         4 * (2 * 128 * kXchPitch + NT) + 8 * (2 * (C::kW + C::kB + C::kOp) + C::kB + 5) + 16 + 4 * (kMaxGroupTab + C::kRows);
}

// What the product's fp16 rows [rows, KD] and their scales are made from: token rows (xq,
// read through map) or fp32 hidden rows with their largest magnitudes (h, row_max).
struct RowSource {
  const int8_t* xq;
  const float* xs;
  const int32_t* map;       // nullable
  const float* h;           // nullable
  const uint32_t* row_max;
  uint4* out;
  float* out_s;
  int rows, TK, n_src;
};

// Kept small: with another 110 bytes of parameters beside the five tensor maps consecutive
// calls no longer overlapped (a decode batch's product 188 -> 202 us).
struct I8Args {
  const int32_t* expert_off;
  const float* xs;          // scale of each row of the operand (routed rows, then shared)
  const float *sa, *sb;     // [G, N] channel scales (sb: W3)
  void* out;                // [TK, N]; up: [TK + S T, N] fp32
  void* out_sh;             // shared rows of the down product [S T, N]
  uint32_t* row_max;        // up: largest |h| of each row, as bits
  DeviceStatus* st;
  int E, G, T, TK, N, KD;
  int shared_rows;          // first operand row of shared expert j: TK + (down ? j T : 0)
  // pairs, token rows: the fp16 tokens [T + 1, KD], the last one zero, and the token of each
  // dispatched row (NULL: the operand's rows are in place)
  const char* tok;
  const int32_t* row_tok;
};

struct I8Tile {
  int g, n0, r0, rows;      // group, first channel, first row of the tile in its group, rows
  int brow;                 // first operand row
  long long orow;           // first output row
  bool shared;
};

// Row tiles per group from expert_off (s_ts, prefix; s_off a copy), by one warp. A bad
// expert_off (or none) schedules nothing.
template <int NT>
__device__ __forceinline__ void group_table(const I8Args& p, int32_t* s_ts, int32_t* s_off, int lane) {
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
  for (int g0 = 0; g0 < p.G; g0 += 32) {
    const int g = g0 + lane;
    int rows = 0;
    if (!bad && g < p.E) rows = s_off[g + 1] - s_off[g];
    else if (!bad && g < p.G) rows = p.T;
    const int n = (rows + NT - 1) / NT;
    int incl = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    if (g < p.G) s_ts[g] = carry + incl - n;
    carry += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) s_ts[p.G] = carry;
}

// Tile t of this CTA's walk, whose tiles ascend; g: the last one's group. A group's row tiles
// are equally long, not NT rows and a rest.
template <bool UP, int NT>
__device__ __forceinline__ I8Tile decode(const I8Args& p, const int32_t* ts, const int32_t* off,
                                         int ntile, int t, uint32_t rank, int& g) {
  constexpr int kRound = I8Cfg<NT>::kB ? 32 : 16;
  while (ts[g + 1] * ntile <= t) ++g;
  const int mt = ts[g + 1] - ts[g], local = t - ts[g] * ntile;
  const int n_tile = local / mt, m_tile = local - n_tile * mt;
  I8Tile r;
  r.g = g;
  r.n0 = (n_tile * (I8Cfg<NT>::kB ? 2 : 1) + (int)rank) * (UP ? 64 : 128);
  r.shared = g >= p.E;
  const int j = g - p.E;
  const int rows = r.shared ? p.T : off[g + 1] - off[g];
  const int step = ((rows + mt - 1) / mt + kRound - 1) & ~(kRound - 1);
  r.r0 = m_tile * step;
  r.rows = min(step, rows - r.r0);
  // the up product reads the tokens' own rows for every shared expert
  r.brow = (r.shared ? p.shared_rows + (UP ? 0 : j * p.T) : off[g]) + r.r0;
  r.orow = (r.shared ? (UP ? (long long)p.TK : 0LL) + (long long)j * p.T : (long long)off[g]) + r.r0;
  return r;
}

// MMA columns of a tile: its rows rounded up to 16 (to 32 on a pair, half for each CTA)
template <int NT>
__device__ __forceinline__ int tile_n(int rows) {
  return I8Cfg<NT>::kB ? min(NT, (rows + 31) & ~31) : min(NT, (rows + 15) & ~15);
}

// 4 signed bytes to 4 fp16
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
  const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), bias);
  const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), bias);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

// (What an earlier kernel of the stream may still be writing when a kernel here starts is read
// through L2: loads through the read-only path may be moved above the wait for that kernel.)
// One row of the product's operand, by a warp. Token rows: row r < TK is xq[map[r]] (or
// xq[r]), row TK + t the token t (shared experts); rows outside the segments [begin, end)
// belong to nobody. Hidden rows: s = max |h| / 127, rint(h / s), an integer that fp16 holds;
// s is 0 for a row that is zero or whose scale would be subnormal, NaN for a row that is not
// finite.
__device__ __forceinline__ void make_row(const RowSource& p, int r, int begin, int end, int KD,
                                         DeviceStatus* st, int lane) {
  if (p.h == nullptr) {
    if ((r < begin || r >= end) && r < p.TK) return;
    const int src = r >= p.TK ? r - p.TK : p.map ? p.map[r] : r;
    const bool in = (unsigned)src < (unsigned)p.n_src;
    if (lane == 0) {
      if (!in) record_error(st, kStatusData, kBadPerm, r);
      p.out_s[r] = in ? p.xs[src] : 0.0f;
    }
    const int vecs = KD >> 3;  // 8 values: a warp's stores are 512 bytes in a row
    const uint2* from = reinterpret_cast<const uint2*>(p.xq) + (size_t)src * vecs;
    uint4* to = p.out + (size_t)r * vecs;
    for (int v = lane; v < vecs; v += 32 * 8) {  // eight loads ahead of the stores
      uint2 b[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        b[u] = in && v + 32 * u < vecs ? __ldcg(from + v + 32 * u) : make_uint2(0u, 0u);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        uint4 o;
        widen4(b[u].x, o.x, o.y);
        widen4(b[u].y, o.z, o.w);
        if (v + 32 * u < vecs) to[v + 32 * u] = o;
      }
    }
    return;
  }
  const float amax = __uint_as_float(p.row_max[r]);
  const bool finite = amax <= FLT_MAX;
  float scale = amax / 127.0f;
  const bool zero = !finite || scale < FLT_MIN;
  if (zero) scale = finite ? 0.0f : __int_as_float(0x7fc00000);
  if (lane == 0) p.out_s[r] = scale;
  const float inv = zero ? 0.0f : 1.0f / scale;
  const int vecs = KD >> 2;
  const float4* in = reinterpret_cast<const float4*>(p.h) + (size_t)r * vecs;
  uint2* out = reinterpret_cast<uint2*>(p.out) + (size_t)r * vecs;
  for (int v = lane; v < vecs; v += 32 * 4) {  // 4 values a lane, four loads ahead
    float4 a[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      a[u] = v + 32 * u < vecs ? __ldcs(in + v + 32 * u) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const __half2 lo = __floats2half2_rn(rintf(a[u].x * inv), rintf(a[u].y * inv));
      const __half2 hi = __floats2half2_rn(rintf(a[u].z * inv), rintf(a[u].w * inv));
      if (v + 32 * u < vecs)
        out[v + 32 * u] = zero ? make_uint2(0u, 0u)
                               : make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                            *reinterpret_cast<const uint32_t*>(&hi));
    }
  }
}

// For gathered rows: the tokens in fp16 and a zero row behind them, with their scales, and the
// token of each dispatched row, the zero row where it is out of range. Also clears the maxima
// of the hidden rows that the product will write.
__global__ void __launch_bounds__(256)
i8_tokens_kernel(const RowSource p, const int32_t* expert_off, int E, int KD,
                 int32_t* row_tok, uint32_t* clear, int nclear,
                 DeviceStatus* st) {
  pdl_wait_and_trigger();
  const int begin = expert_off[0], end = expert_off[E], T = p.n_src;
  for (int i = blockIdx.x * 256 + threadIdx.x; i < max(nclear, p.TK); i += gridDim.x * 256) {
    if (i < nclear) clear[i] = 0u;
    if (i < p.TK) {
      const bool used = i >= begin && i < end;
      const int t = used ? p.map[i] : T;
      const bool in = (unsigned)t < (unsigned)T;
      if (!in && used) record_error(st, kStatusData, kBadPerm, i);
      row_tok[i] = in ? t : T;
    }
  }
  const int lane = threadIdx.x & 31;
  for (int r = blockIdx.x * 8 + (threadIdx.x >> 5); r <= T; r += gridDim.x * 8) {
    if (r < T) {
      RowSource one = p;
      one.map = nullptr;
      make_row(one, r, 0, T, KD, st, lane);
    } else {
      for (int v = lane; v < KD / 8; v += 32) p.out[(size_t)T * (KD / 8) + v] = make_uint4(0, 0, 0, 0);
      if (lane == 0) p.out_s[T] = 0.0f;
    }
  }
}

// The rows put in place, by a kernel of their own. (Made inside the product by spare warps,
// behind completion counters, 131072 rows of 2048 took 401 us with their product, against
// 376.) Also clears the maxima of the hidden rows that the product will write.
__global__ void __launch_bounds__(256)
i8_rows_kernel(const RowSource p, const int32_t* expert_off, int E, int KD,
               uint32_t* clear, int nclear, DeviceStatus* st) {
  pdl_wait_and_trigger();
  for (int i = blockIdx.x * 256 + threadIdx.x; i < nclear; i += gridDim.x * 256) clear[i] = 0u;
  const int begin = p.h ? 0 : expert_off[0], end = p.h ? p.rows : expert_off[E];
  for (int r = blockIdx.x * 8 + (threadIdx.x >> 5); r < p.rows; r += gridDim.x * 8)
    make_row(p, r, begin, end, KD, st, threadIdx.x & 31);
}

// GATHER (pairs): the token rows are gathered by the product itself.
template <bool UP, int NT, typename TO, bool GATHER>
__global__ void __launch_bounds__(GATHER ? kI8Threads + 32 * (kCopyWarps - 1) : kI8Threads, 1)
i8_gemm_kernel(const __grid_constant__ CUtensorMap tmWa,   // weights as 16-bit pairs; up: 64-row box
               const __grid_constant__ CUtensorMap tmWb,   // (W3), else 128-row box
               const __grid_constant__ CUtensorMap tmX16,  // fp16 rows, boxes of 16, 48 and kRows
               const __grid_constant__ CUtensorMap tmX48,
               const __grid_constant__ CUtensorMap tmX, const I8Args p) {
  // The kernel before this one in the stream writes the rows and has itself waited for what
  // is before it, so the weights and expert_off are read without waiting for it: the weight
  // ring fills while it runs. The rows' producer and the epilogue wait.
  pdl_trigger();
  using C = I8Cfg<NT>;
  constexpr uint32_t kHalf = C::kRows * 128;  // rows x 64 values
  constexpr bool kOwnB = C::kB > 0;           // a ring of their own for the rows, on CTA pairs
  constexpr bool kPair = kOwnB;
  constexpr int kOpCol = 2 * NT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sW = base;
  uint8_t* sB = sW + C::kW * kStageW;
  float* s_xch = reinterpret_cast<float*>(sB + 2 * (kOwnB ? C::kB : C::kOp) * kHalf);  // [2][128][20]
  float* s_xs = s_xch + 2 * 128 * kXchPitch;             // [NT] row scales of the tile
  uint64_t* wfull = reinterpret_cast<uint64_t*>(s_xs + NT);
  uint64_t* wempty = wfull + C::kW;
  uint64_t* bfull = wempty + C::kW;
  uint64_t* bempty = bfull + C::kB;
  uint64_t* afull = bempty + C::kB;
  uint64_t* aempty = afull + C::kOp;
  uint64_t* dfull = aempty + C::kOp;
  uint64_t* dempty = dfull + 2;
  uint64_t* drain = dempty + 2;
  uint64_t* rfull = drain + 1;  // pairs: this CTA's gathered rows of a stage
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(rfull + C::kB);
  int* s_abort = reinterpret_cast<int*>(s_tmem + 1);
  int32_t* s_ts = reinterpret_cast<int32_t*>(s_abort + 1);
  int32_t* s_off = s_ts + kMaxGroups + 2;
  int32_t* s_row = s_off + kMaxGroups + 2;               // pairs: the tokens of this CTA's rows

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = kPair ? tc::cluster_rank() : 0u;
  const int first = kPair ? blockIdx.x >> 1 : blockIdx.x, stride = kPair ? gridDim.x >> 1 : gridDim.x;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kW; ++s) {
      tc::mbar_init(&wfull[s], 1);
      tc::mbar_init(&wempty[s], 8);
    }
    for (int s = 0; s < C::kB; ++s) {
      tc::mbar_init(&bfull[s], GATHER ? 2 : 1);  // both CTAs' gathered rows, or the copies' bytes
      tc::mbar_init(&bempty[s], 1);
      tc::mbar_init(&rfull[s], 32 * kCopyWarps);
    }
    for (int s = 0; s < C::kOp; ++s) {
      tc::mbar_init(&afull[s], kPair ? 16 : 9);  // both CTAs' widening warps; or with the rows' copy
      tc::mbar_init(&aempty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      tc::mbar_init(&dfull[a], 1);
      tc::mbar_init(&dempty[a], kPair ? 256 : 128);
    }
    tc::mbar_init(drain, 1);
    *s_abort = 0;
    tc::mbar_init_fence();
    tc::tma_prefetch_map(&tmWa);
    tc::tma_prefetch_map(&tmWb);
    tc::tma_prefetch_map(&tmX16);
    tc::tma_prefetch_map(&tmX48);
    tc::tma_prefetch_map(&tmX);
  }
  __syncwarp();
  if (kPair) tc::cluster_arrive();
  if (warp == 3) group_table<NT>(p, s_ts, s_off, lane);
  __syncwarp();
  // the peer runs, and both CTAs' barriers are initialised before a remote signal
  if (kPair) tc::cluster_wait();
  if (warp == 2) {
    if (kPair) {
      tc::tmem_alloc_pair(s_tmem, 512);
      tc::tmem_relinquish_pair();
    } else {
      tc::tmem_alloc(s_tmem, 512);
      tc::tmem_relinquish();
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *s_tmem;
  constexpr int kChan = (UP ? 64 : 128) * (kPair ? 2 : 1);
  const int ntile = (p.N + kChan - 1) / kChan;
  const int total = s_ts[p.G] * ntile;
  const int nk = (p.KD + 127) / 128, nb = (p.KD + 63) / 64;
  volatile int* abort = s_abort;

  if (warp == 0) {
    // ---------------------------------------------------------------- weight producer
    const bool lead = tc::elect_one();
    uint32_t ws = 0, wph = 1, wit = 0;
    bool ok = true;
    int g = 0;
    for (int t = first; t < total && ok; t += stride) {
      const I8Tile tl = decode<UP, NT>(p, s_ts, s_off, ntile, t, rank, g);
      const int wrow = tl.g * p.N + tl.n0;
      for (int kb = 0; kb < nk; ++kb) {
        ok = tc::mbar_wait_warp(&wempty[ws], wph, abort);
        if (!ok) break;
        if (lead) {
          tc::mbar_expect_tx(&wfull[ws], kStageW);
          tc::tma_load_2d(sW + ws * kStageW, &tmWa, &wfull[ws], kb * 64, wrow);
          if (UP) tc::tma_load_2d(sW + ws * kStageW + kStageW / 2, &tmWb, &wfull[ws], kb * 64, wrow);
        }
        __syncwarp();
        ++wit;
        if (++ws == C::kW) { ws = 0; wph ^= 1u; }
      }
    }
    if (lead) {
      if (!ok) {
        *abort = 1;
        record_error(p.st, kStatusTimeout, kTimeoutGemm, blockIdx.x);
      }
      // the copies in flight land before the CTA's shared memory goes away, also where it was
      // another role that gave up
      volatile int never = 0;
      for (uint32_t j = wit > C::kW ? wit - C::kW : 0; j < wit; ++j)
        tc::mbar_wait(&wfull[j % C::kW], (j / C::kW) & 1u, &never);
    }
    __syncwarp();
  } else if (GATHER && (warp >= 16 || warp == 3)) {
    // ---------------------------------------------------------------- row producer: gather
    // Two rows of 256 bytes (128 values) an instruction, into the two 128-byte-swizzled
    // halves of the stage.
    // The copying warps take groups of 16 rows in turn (six of them for 192 MMA columns).
    pdl_wait();
    const int cw = warp == 3 ? 0 : warp - 15;
    uint32_t bs = 0, bph = 1;
    bool ok = true;
    int g = 0;
    const int c = lane & 15;
    const uint32_t half = (uint32_t)(c >> 3) * kHalf;
    for (int t = first; t < total && ok; t += stride) {
      const I8Tile tl = decode<UP, NT>(p, s_ts, s_off, ntile, t, rank, g);
      const int mine = tile_n<NT>(tl.rows) / 2;  // a multiple of 16
      __syncwarp();
      for (int i = 16 * cw + lane; i < mine && lane < 16; i += 16 * kCopyWarps) {
        const int r = (int)rank * mine + i;  // row of the tile
        s_row[i] = r >= tl.rows ? p.T : tl.shared ? tl.r0 + r : __ldcg(p.row_tok + tl.brow + r);
      }
      __syncwarp();
      for (int kb = 0; kb < nk; ++kb) {
        ok = tc::mbar_wait_warp(&bempty[bs], bph, abort);
        if (!ok) break;
        const uint32_t dst = tc::smem_u32(sB + 2 * bs * kHalf) + half;
        const int left = p.KD * 2 - kb * 256 - c * 16;
        const uint32_t valid = left > 0 ? 16u : 0u;
        const char* src = p.tok + (left > 0 ? kb * 256 + c * 16 : 0);
        for (int i0 = 16 * cw + (lane >> 4); i0 < mine; i0 += 16 * kCopyWarps) {
          const char* from[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) from[u] = src + (size_t)s_row[i0 + 2 * u] * (2 * p.KD);
#pragma unroll
          for (int u = 0; u < 8; ++u)
            tc::cp_async16(dst + (i0 + 2 * u) * 128 + (((c & 7) ^ ((i0 + 2 * u) & 7)) << 4), from[u], valid);
        }
        tc::cp_async_arrive(&rfull[bs]);
        if (++bs == C::kB) { bs = 0; bph ^= 1u; }
      }
    }
    tc::cp_async_wait_all();
    if (!ok && lane == 0) {
      *abort = 1;
      record_error(p.st, kStatusTimeout, kTimeoutGemm, blockIdx.x);
    }
    __syncwarp();
  } else if (GATHER && warp == 2) {
    // ---------------------------------------------------------------- gathered rows' signal
    // The copies wrote through the generic proxy, the MMA reads through the async proxy, and the
    // leader issues it for both CTAs' rows: the proxy fence, then a release at cluster scope of
    // what is in shared memory, which the MMA warp acquires. (131072 rows of 2048 to 768
    // channels: 327 us, 324 without the order. A release of everything waits for the epilogue's
    // stores: 446 us, and 356 with a warp for each stage of the ring.)
    const int stages = total > first ? (total - first + stride - 1) / stride * nk : 0;
    uint32_t bs = 0, ph = 0;
    bool ok = true;
    for (int i = 0; i < stages; ++i) {
      ok = tc::mbar_wait_warp(&rfull[bs], ph, abort);
      if (!ok) break;
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_cluster_shared(tc::cluster_addr(&bfull[bs], 0));
      if (++bs == C::kB) { bs = 0; ph ^= 1u; }
    }
    if (!ok && lane == 0) {
      *abort = 1;
      record_error(p.st, kStatusTimeout, kTimeoutGemm, blockIdx.x);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ---------------------------------------------------------------- row producer: in place
    pdl_wait();
    const bool lead = tc::elect_one();
    constexpr uint32_t kRing = kOwnB ? C::kB : C::kOp;
    uint64_t* bar = kOwnB ? bfull : afull;
    uint64_t* free = kOwnB ? bempty : aempty;
    uint32_t bs = 0, bph = 1, bit = 0;
    bool ok = true;
    int g = 0;
    for (int t = first; t < total && ok; t += stride) {
      const I8Tile tl = decode<UP, NT>(p, s_ts, s_off, ntile, t, rank, g);
      // this CTA's rows: all of the tile's, or its half of the MMA's columns
      const int mine = kPair ? tile_n<NT>(tl.rows) / 2 : tl.rows;
      const int box = mine <= 16 ? 16 : mine <= 48 ? 48 : C::kRows;
      const CUtensorMap* xmap = box == 16 ? &tmX16 : box == 48 ? &tmX48 : &tmX;
      const int brow = tl.brow + (kPair ? (int)rank * mine : 0);
      for (int kb = 0; kb < nk; ++kb) {
        ok = tc::mbar_wait_warp(&free[bs], bph, abort);
        if (!ok) break;
        if (lead) {
          const int halves = min(2, nb - 2 * kb);
          uint8_t* dst = sB + 2 * bs * kHalf;
          if (kPair) {  // both CTAs' bytes complete on the leader's barrier
            const uint32_t on = tc::cluster_addr(&bar[bs], 0);
            if (rank == 0) tc::mbar_expect_tx(&bar[bs], 2 * box * 128 * halves);
            tc::tma_load_2d_pair(dst, xmap, on, 2 * kb * 64, brow);
            if (halves == 2) tc::tma_load_2d_pair(dst + kHalf, xmap, on, (2 * kb + 1) * 64, brow);
          } else {
            tc::mbar_expect_tx(&bar[bs], box * 128 * halves);
            tc::tma_load_2d(dst, xmap, &bar[bs], 2 * kb * 64, brow);
            if (halves == 2) tc::tma_load_2d(dst + kHalf, xmap, &bar[bs], (2 * kb + 1) * 64, brow);
          }
        }
        __syncwarp();
        ++bit;
        if (++bs == kRing) { bs = 0; bph ^= 1u; }
      }
    }
    if (lead) {
      if (!ok) {
        *abort = 1;
        record_error(p.st, kStatusTimeout, kTimeoutGemm, blockIdx.x);
      }
      // as above, the leader for both CTAs' copies; a barrier that others share may never
      // complete: then the limit is waited out once. So does a peer where a role gave up: its
      // copies may be of stages that the leader did not get to.
      volatile int never = 0;
      if (rank == 0) {
        for (uint32_t j = bit > kRing ? bit - kRing : 0; j < bit; ++j)
          if (!tc::mbar_wait(&bar[j % kRing], (j / kRing) & 1u, &never)) break;
      } else if (*abort) {
        tc::wait_out();
      }
    }
    __syncwarp();
  } else if (warp == 1 && rank == 0) {
    // ---------------------------------------------------------------- MMA issuer (of the pair)
    const bool lead = tc::elect_one();
    uint32_t bs = 0, bph = 0, as = 0, aph = 0, d = 0, dph = 1;
    bool ok = true, a_in = false, b_in = false;
    int g = 0;
    for (int t = first; t < total && ok; t += stride) {
      const I8Tile tl = decode<UP, NT>(p, s_ts, s_off, ntile, t, rank, g);
      const uint32_t idesc = tc::instr_desc_f16(kPair ? 256 : 128, tile_n<NT>(tl.rows));
      if (!tc::mbar_wait_warp(&dempty[d], dph, abort)) { ok = false; break; }
      tc::fence_after_sync();
      const uint32_t acc = tmem + d * NT;
      for (int kb = 0; kb < nk; ++kb) {
        if (!a_in) ok = tc::mbar_wait_warp(&afull[as], aph, abort);
        if (kOwnB && !b_in && ok)
          ok = GATHER ? tc::mbar_wait_warp_shared(&bfull[bs], bph, abort)
                      : tc::mbar_wait_warp(&bfull[bs], bph, abort);
        if (!ok) break;
        tc::fence_after_sync();
        const uint32_t a0 = tmem + kOpCol + as * 64;
        const uint64_t bdesc = tc::sw128_kmajor_desc(tc::smem_u32(sB + 2 * (kOwnB ? bs : as) * kHalf));
        uint64_t *a_free = &aempty[as], *b_free = &bempty[bs];
        if (++as == C::kOp) { as = 0; aph ^= 1u; }
        if (kOwnB && ++bs == C::kB) { bs = 0; bph ^= 1u; }
        // look at the next stage's barriers while this stage's MMAs are issued: asking costs
        // over 100 clocks even when they have completed
        const bool a_next = tc::mbar_test(&afull[as], aph);
        const bool b_next = kOwnB && (GATHER ? tc::mbar_test_shared(&bfull[bs], bph)
                                             : tc::mbar_test(&bfull[bs], bph));
        if (lead) {
          const int n = 4 * min(2, nb - 2 * kb);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (k >= n) break;
            const uint64_t b = bdesc + (k >> 2) * (kHalf >> 4) + 2 * (k & 3);
            if (kPair) tc::mma_f16_tmem_a_pair(acc, a0 + k * 8, b, idesc, kb > 0 || k > 0);
            else tc::mma_f16_tmem_a(acc, a0 + k * 8, b, idesc, kb > 0 || k > 0);
          }
          if (kPair) {
            tc::commit_pair(b_free, 0x3);
            tc::commit_pair(a_free, 0x3);
          } else {
            tc::commit(a_free);
          }
        }
        a_in = __all_sync(0xffffffffu, a_next);
        b_in = __all_sync(0xffffffffu, b_next);
      }
      if (!ok) break;
      if (lead) {
        if (kPair) tc::commit_pair(&dfull[d], 0x3);
        else tc::commit(&dfull[d]);
      }
      __syncwarp();
      if (++d == 2) { d = 0; dph ^= 1u; }
    }
    if (lead) {
      if (!ok) {
        *abort = 1;
        record_error(p.st, kStatusTimeout, kTimeoutGemm, blockIdx.x);
      }
      // wait for every MMA this thread issued before TMEM is released
      volatile int never = 0;
      if (kPair) tc::commit_pair(drain, 0x1);
      else tc::commit(drain);
      tc::mbar_wait(drain, 0, &never);
    }
    __syncwarp();
  } else if (warp >= 8) {
    // ---------------------------------------------------------------- widen the weights
    const int q = warp & 3, half = (warp - 8) >> 2, row = q * 32 + lane;
    uint32_t ws = 0, wph = 0, as = 0, aph = 1;
    bool ok = true, w_in = false;
    for (int t = first; t < total && ok; t += stride)
      for (int kb = 0; kb < nk; ++kb) {
        if (!w_in) ok = tc::mbar_wait_warp(&wfull[ws], wph, abort);
        if (!ok) break;
        // the operand stage is asked for while the bytes are read, the next bytes while they
        // are widened: each asking costs over 100 of the stage's 600 to 850 clocks
        const bool a_free = tc::mbar_test(&aempty[as], aph);
        const uint8_t* src = sW + ws * kStageW + row * 128;
        uint4 v[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          v[c] = *reinterpret_cast<const uint4*>(src + (((4 * half + c) ^ (row & 7)) << 4));
        uint64_t* w_done = &wempty[ws];
        if (++ws == C::kW) { ws = 0; wph ^= 1u; }
        const bool w_next = tc::mbar_test(&wfull[ws], wph);
        uint32_t r[32];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          widen4(v[c].x, r[8 * c], r[8 * c + 1]);
          widen4(v[c].y, r[8 * c + 2], r[8 * c + 3]);
          widen4(v[c].z, r[8 * c + 4], r[8 * c + 5]);
          widen4(v[c].w, r[8 * c + 6], r[8 * c + 7]);
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(w_done);
        if (!__all_sync(0xffffffffu, a_free)) ok = tc::mbar_wait_warp(&aempty[as], aph, abort);
        if (!ok) break;
        tc::fence_after_sync();
        tc::tmem_st32(tmem + ((uint32_t)(q * 32) << 16) + kOpCol + as * 64 + half * 32, r);
        w_in = __all_sync(0xffffffffu, w_next);
        tc::tmem_st_wait();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if (kPair) tc::mbar_arrive_remote(tc::cluster_addr(&afull[as], 0));
          else tc::mbar_arrive(&afull[as]);
        }
        if (++as == C::kOp) { as = 0; aph ^= 1u; }
      }
    if (!ok && lane == 0) {
      *abort = 1;
      record_error(p.st, kStatusTimeout, kTimeoutGemm, blockIdx.x);
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- epilogue
    pdl_wait();
    const int q = warp & 3, row = q * 32 + lane;
    const int fr = row & 63, tq = row >> 6;  // up: this thread's feature and half of 32 tokens
    uint32_t d = 0, dph = 0;
    int g = 0;
    for (int t = first; t < total; t += stride) {
      const I8Tile tl = decode<UP, NT>(p, s_ts, s_off, ntile, t, rank, g);
      const int nt = min(NT, tl.rows), n32 = (nt + 31) >> 5;
      const int chan = tl.n0 + (UP ? fr : row);  // this thread's channel
      const bool has = chan < p.N;
      // the tile's scales, ahead of its accumulator
      for (int i = row; i < NT; i += 128) {
        int r = tl.brow + i;
        if (GATHER && i < nt) r = tl.shared ? tl.r0 + i : __ldcg(p.row_tok + r);
        s_xs[i] = i < nt ? __ldcg(p.xs + r) : 0.0f;
      }
      const float sc = has ? __ldg(p.sa + (size_t)tl.g * p.N + chan) : 0.0f;
      const float sc3 = UP && has ? __ldg(p.sb + (size_t)tl.g * p.N + chan) : 0.0f;
      const bool ok = tc::mbar_wait_warp(&dfull[d], dph, abort);
      // one outcome for the four warps, which meet at barriers
      uint32_t all;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
          "barrier.cta.red.and.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}\n"
          : "=r"(all) : "r"((uint32_t)ok) : "memory");
      if (!all) {
        *abort = 1;
        record_error(p.st, kStatusTimeout, kTimeoutGemm, blockIdx.x);
        break;
      }
      tc::fence_after_sync();
      const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + d * NT;
      TO* out = static_cast<TO*>(!UP && tl.shared ? p.out_sh : p.out) + (size_t)tl.orow * p.N + chan;
#pragma unroll 1
      for (int c = 0; c < n32; ++c) {
        __syncwarp();  // TMEM loads are a whole warp's: lanes that split (atomics, barriers) join
        auto read_out = [&] {  // after the last chunk another tile's MMAs may start
          if (c != n32 - 1) return;
          tc::fence_before_sync();
          if (kPair) tc::mbar_arrive_remote(tc::cluster_addr(&dempty[d], 0));
          else tc::mbar_arrive(&dempty[d]);
        };
        if (UP) {
          // Lanes 0-63 hold gates, 64-127 the same features' up values. A thread keeps 16 of
          // its 32 tokens and gives the other 16 to its counterpart; the largest magnitudes of
          // 16 rows leave in one atomic instruction. This work overlaps the next tile's MMAs
          // and still takes shared memory, issue slots and power from them: with both values
          // through shared memory and an atomic for each row, 1001 tokens of 8 wide experts
          // took 635 us, now 578; 8192 tokens of 160 experts 2.57 ms, now 2.48.
          float keep[16], give[16], other[16];
          tc::tmem_ld16(taddr + 32 * c + 16 * tq, keep);
          tc::tmem_ld16(taddr + 32 * c + 16 * (tq ^ 1), give);
          read_out();
          float* xch = s_xch + (c & 1) * 128 * kXchPitch;
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<float4*>(xch + row * kXchPitch + i) =
                make_float4(give[i], give[i + 1], give[i + 2], give[i + 3]);
          asm volatile("barrier.cta.sync %0, 64;" ::"r"(2 + (q & 1)) : "memory");
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 f = *reinterpret_cast<const float4*>(xch + (row ^ 64) * kXchPitch + i);
            other[i] = f.x; other[i + 1] = f.y; other[i + 2] = f.z; other[i + 3] = f.w;
          }
          const int at = 32 * c + 16 * tq, left = nt - at;
          auto hidden = [&](const float (&gate)[16], const float (&up)[16]) {
            const int stop = has ? left : 0;
            TO* o = out + (size_t)at * p.N;
            uint32_t most = 0;
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const float4 x4 = *reinterpret_cast<const float4*>(s_xs + at + i);
              const float x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
              for (int j = 0; j < 4; ++j, o += p.N) {
                const float g = gate[i + j] * x[j] * sc;
                const float u = up[i + j] * x[j] * sc3;
                // (the fast division: 2 units in the last place, and 7 bits are kept of h)
                const float h = has ? __fdividef(g, 1.0f + expf(-g)) * u : 0.0f;
                if (i + j < stop) *o = Elem<TO>::from_f32(h);
                const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(h) & 0x7fffffffu);
                if (lane == i + j) most = m;
              }
            }
            if (lane < 16 && lane < left) atomicMax(p.row_max + tl.orow + at + lane, most);
          };
          if (left > 0) {
            if (tq == 0) hidden(keep, other);
            else hidden(other, keep);
          }
        } else {
          uint32_t v[32];
          tc::tmem_ld32(taddr + 32 * c, v);
          tc::tmem_ld_wait();
          read_out();
          const int stop = has ? nt - 32 * c : 0;
          TO* o = out + (size_t)(32 * c) * p.N;
#pragma unroll
          for (int i = 0; i < 32; i += 4) {  // (scales read one by one: FFN prefill 2.50 ms, by four 2.38)
            const float4 x = *reinterpret_cast<const float4*>(s_xs + 32 * c + i);
            const float y[4] = {__uint_as_float(v[i]) * x.x * sc, __uint_as_float(v[i + 1]) * x.y * sc,
                                __uint_as_float(v[i + 2]) * x.z * sc, __uint_as_float(v[i + 3]) * x.w * sc};
#pragma unroll
            for (int j = 0; j < 4; ++j, o += p.N)
              if (i + j < stop) *o = Elem<TO>::from_f32(y[j]);
          }
        }
      }
      asm volatile("barrier.cta.sync 1, 128;" ::: "memory");  // s_xs has been read
      if (++d == 2) { d = 0; dph ^= 1u; }
    }
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  if (kPair) tc::cluster_sync();  // no signal or copy of the other CTA is on its way here
  tc::fence_after_sync();
  if (warp == 2) {
    if (kPair) tc::tmem_dealloc_pair(tmem, 512);
    else tc::tmem_dealloc(tmem, 512);
  }
}

// From this many rows per expert on average the wide tiles win: they read a weight byte once
// per 160 rows and issue fewer MMAs for them; below, the weights' stream is the work, and the
// narrow tiles keep more of it in flight. Measured (FFN, narrow and wide, at 24, 40 and 64 rows):
// 160 experts of 5120 x 1536 633 and 628, 670 and 647, 784 and 684 us; 8 experts of
// 4096 x 14336 256 and 258, 264 and 263, 322 and 268; 128 experts of 2048 x 768 126 and 138,
// 140 and 144, 166 and 159.
constexpr int kWideRows = 40;
// From this many on, 192-row tiles instead of 160 where the rows are in place: fewer MMAs a
// row, against a third operand stage (FFN, 160 and 192 rows, 8 experts of 4096 x 14336: 100
// rows an expert 288 and 309 us, 250: 535 and 569, 512: 975 and 980, 1024: 1706 and 1659; 160 of
// 5120 x 1536, 307 rows: 2134 and 2156; 16 of 2048 x 2048, 512 rows: 211 and 204).
constexpr int kTallRows = 400;
bool wide(const smoe_desc& d) { return (long long)d.T * d.K >= (long long)kWideRows * d.E; }

int i8_sm_count() {
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n > 0 ? n : 148;
}

template <bool UP, int NT, typename TO, bool GATHER = false>
cudaError_t run_gemm(const I8Args& p, const int8_t* wa, const int8_t* wb, const void* x16,
                     long long xrows, cudaStream_t s) {
  alignas(64) CUtensorMap ta, tb, x1, x4, xn;
  const uint64_t wrows = (uint64_t)p.G * p.N;
  if (!encode_tmap_2d(&ta, wa, false, wrows, p.KD / 2, UP ? 64 : 128, 64) ||
      !encode_tmap_2d(&tb, UP ? wb : wa, false, wrows, p.KD / 2, UP ? 64 : 128, 64) ||
      !encode_tmap_2d(&x1, x16, false, xrows, p.KD, 16, 64) ||
      !encode_tmap_2d(&x4, x16, false, xrows, p.KD, 48, 64) ||
      !encode_tmap_2d(&xn, x16, false, xrows, p.KD, I8Cfg<NT>::kRows, 64))
    return cudaErrorInvalidValue;
  auto kern = i8_gemm_kernel<UP, NT, TO, GATHER>;
  const int smem = (int)i8_smem<NT>();
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(I8Cfg<NT>::kB ? i8_sm_count() / 2 * 2 : i8_sm_count());
  cfg.blockDim = dim3(GATHER ? kI8Threads + 32 * (kCopyWarps - 1) : kI8Threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = I8Cfg<NT>::kB ? 2 : 1;
  SMOE_COUNT_LAUNCH(1);
  return cudaLaunchKernelEx(&cfg, kern, ta, tb, x1, x4, xn, p);
}

template <bool UP, typename TO>
cudaError_t run_product(const smoe_desc& d, const I8Args& p, const int8_t* wa, const int8_t* wb,
                        const void* x16, long long xrows, cudaStream_t s) {
  if (p.row_tok) return run_gemm<UP, 192, TO, true>(p, wa, wb, x16, xrows, s);
  if ((long long)d.T * d.K >= (long long)kTallRows * d.E)
    return run_gemm<UP, 192, TO>(p, wa, wb, x16, xrows, s);
  if (wide(d)) return run_gemm<UP, 160, TO>(p, wa, wb, x16, xrows, s);
  return run_gemm<UP, 64, TO>(p, wa, wb, x16, xrows, s);
}

cudaError_t run_rows(const RowSource& r, const int32_t* expert_off, int E, int KD, uint32_t* clear,
                     int nclear, DeviceStatus* st, cudaStream_t s) {
  const int grid = std::max(1, std::min(std::max(ceil_div(r.rows, 8), ceil_div(nclear, 256)), 152 * 8));
  SMOE_LAUNCH(i8_rows_kernel, grid, 256, 0, s, r, expert_off, E, KD, clear, nclear, st);
  return cudaGetLastError();
}

// Up to this many output channels a product of wide tiles gathers its rows from the widened
// tokens; above, a kernel puts them in place and TMA loads them. Gathering spares writing
// every row (K times the tokens) and slows the product by about a tenth, which more channels
// make dearer. Measured (in place, gathered): 131072 rows of 2048: 256 channels 230, 129 us;
// 768: 372, 326; 1536: 628, 616; 2048: 813, 816. 49152 rows of 5120: 768 channels 383, 340; 1536:
// 647, 646; 2048: 819, 844. 16384 rows of 4096: 768 channels 96, 92; 1536: 152, 158; 2048: 185, 197.
constexpr int kGatherChannels = 1536;

// Token rows for the product `p`: gathered by it (wide tiles), or put in place for it.
cudaError_t run_token_rows(const smoe_desc& d, I8Args* p, const RowSource& r, uint32_t* clear,
                           int nclear, int32_t* row_tok, int channels, cudaStream_t s) {
  if (!wide(d) || r.map == nullptr || channels > kGatherChannels)
    return run_rows(r, p->expert_off, d.E, p->KD, clear, nclear, p->st, s);
  const int grid = std::min(std::max(ceil_div(d.T + 1, 8), ceil_div(std::max(nclear, r.TK), 256)), 152 * 8);
  SMOE_LAUNCH(i8_tokens_kernel, grid, 256, 0, s, r, p->expert_off, d.E, p->KD, row_tok, clear, nclear,
              p->st);
  p->tok = reinterpret_cast<const char*>(r.out);
  p->row_tok = row_tok;
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
  const size_t TK = (size_t)d.T * d.K, rows = TK + (size_t)d.n_shared * d.T;
  // rows in place, or the tokens and a zero row
  const size_t xrows = std::max(TK + (d.n_shared ? d.T : 0), (size_t)d.T + 1);
  L->status = take(256);
  L->x16 = take(xrows * std::max(d.d, d.F) * 2);
  L->x16_s = take(xrows * 4);
  L->h = take(rows * d.F * 4);
  L->h16 = take(rows * d.F * 2);
  L->h16_s = take(rows * 4);
  L->row_max = take(rows * 4);
  L->row_tok = take(TK * 4);
  L->total = off;
}

cudaError_t launch_expert_matmul_i8(const smoe_desc& d, int n_out, int n_in, const int8_t* xq,
                                    const float* xs, const int32_t* row_src,
                                    const int32_t* expert_off, const int8_t* wq, const float* ws_n,
                                    void* out, void* ws, cudaStream_t s) {
  I8Layout L;
  i8_ws_layout(d, &L);
  DeviceStatus* st = ws_ptr<DeviceStatus>(ws, L.status);
  const int TK = d.T * d.K;
  uint4* x16 = ws_ptr<uint4>(ws, L.x16);
  float* x16_s = ws_ptr<float>(ws, L.x16_s);
  const RowSource r{xq, xs, row_src, nullptr, nullptr, x16, x16_s, TK, TK, row_src ? d.T : TK};
  I8Args p{expert_off, x16_s, ws_n, nullptr, out, nullptr, nullptr, st,
           d.E, d.E, d.T, TK, n_out, n_in, TK, nullptr, nullptr};
  const cudaError_t e = run_token_rows(d, &p, r, nullptr, 0, ws_ptr<int32_t>(ws, L.row_tok), n_out, s);
  if (e != cudaSuccess) return e;
  return d.dtype == SMOE_F32 ? run_product<false, float>(d, p, wq, nullptr, x16, TK, s)
                             : run_product<false, __nv_bfloat16>(d, p, wq, nullptr, x16, TK, s);
}

cudaError_t launch_expert_ffn_i8(const smoe_desc& d, const int8_t* xq, const float* xs,
                                 const int32_t* row_src, const int32_t* expert_off,
                                 const smoe_i8_weights& W, void* y_disp, void* y_sh, void* ws,
                                 cudaStream_t s) {
  I8Layout L;
  i8_ws_layout(d, &L);
  DeviceStatus* st = ws_ptr<DeviceStatus>(ws, L.status);
  const int TK = d.T * d.K, G = d.E + d.n_shared, rows = TK + d.n_shared * d.T;
  const int xrows = TK + (d.n_shared ? d.T : 0);
  uint4 *x16 = ws_ptr<uint4>(ws, L.x16), *h16 = ws_ptr<uint4>(ws, L.h16);
  float *x16_s = ws_ptr<float>(ws, L.x16_s), *h = ws_ptr<float>(ws, L.h);
  float* h16_s = ws_ptr<float>(ws, L.h16_s);
  uint32_t* row_max = ws_ptr<uint32_t>(ws, L.row_max);
  const RowSource rx{xq, xs, row_src, nullptr, nullptr, x16, x16_s, xrows, TK, row_src ? d.T : TK};
  const RowSource rh{nullptr, nullptr, nullptr, h, row_max, h16, h16_s, rows, TK, 0};
  I8Args up{expert_off, x16_s, W.s1, W.s3, h, nullptr, row_max, st,
            d.E, G, d.T, TK, d.F, d.d, TK, nullptr, nullptr};
  cudaError_t e = run_token_rows(d, &up, rx, row_max, rows, ws_ptr<int32_t>(ws, L.row_tok), 2 * d.F, s);
  if (e != cudaSuccess) return e;
  e = run_product<true, float>(d, up, W.w1, W.w3, x16, xrows, s);
  if (e != cudaSuccess) return e;
  e = run_rows(rh, expert_off, d.E, d.F, nullptr, 0, st, s);
  if (e != cudaSuccess) return e;
  const I8Args dn{expert_off, h16_s, W.s2, nullptr, y_disp, y_sh, nullptr, st,
                  d.E, G, d.T, TK, d.d, d.F, TK, nullptr, nullptr};
  return d.dtype == SMOE_F32 ? run_product<false, float>(d, dn, W.w2, nullptr, h16, rows, s)
                             : run_product<false, __nv_bfloat16>(d, dn, W.w2, nullptr, h16, rows, s);
}

}  // namespace smoe
