// Weight gradients of the experts' products, each over its expert's ragged rows,
//   dw[e, n, k] = add[e, n, k] + sum_{r of e} dy[r, n] x[r, k]   (fp32),
// x as it is or widened from 8-bit rows first.
//
// bf16: the contraction runs over rows, which neither operand is contiguous in, so both are
// staged by TMA as they lie (boxes of 64 channels x 64 rows) and read MN-major by tcgen05.mma:
// nothing is transposed. A segment ends anywhere: an MMA takes 16 rows, those of the last one
// that belong to the next expert (or to nobody) are set to zero in shared memory, in both
// operands, before it runs, so that neither their values nor their infinities reach the sum.
// A persistent pair of CTAs (a cluster on the two SMs of a TPC) walks 256 x 256 tiles of the
// gradients: each CTA stages 128 channels of dy and 128 of x for each 64 rows, holds 128 x 256 sums
// and stores them. (128 x 256 tiles of single CTAs stage half as much again, and the L2's
// bandwidth bounded them at large row counts.)
//   warp 0  TMA;  warp 1  the last rows' zeros, and on the leader tcgen05.mma into one of two
//   TMEM accumulators;  warps 4-11  add and store, while the next tile's MMAs run.
// An expert's R rows give 2 R flops per element of 4 bytes (8 with add): below about 550 rows an
// expert the stores bound it, not the tensor cores.
#include <algorithm>
#include <cuda_fp8.h>

#include "tc_common.cuh"

namespace smoe {
namespace {

constexpr int kDwStages = 5, kDwWarps = 8, kDwThreads = 128 + 32 * kDwWarps;
constexpr int kDwCols = 1024 / kDwWarps;  // columns of an epilogue warp
constexpr int kDwHalf = 128 * 128;  // bytes of an operand's stage in a CTA: 64 rows of 128 channels
constexpr size_t kDwSmem = 1024 + kDwStages * 2 * kDwHalf + kDwWarps * 4096 +
                           8 * (3 * kDwStages + 2 * 2 + 1) + 16 + 4 * (kMaxGroups + 2);

struct DwArgs {
  const int32_t* expert_off;
  const float* add;   // nullable
  float* dw;
  DeviceStatus* st;
  int E, TK, M, N;    // M = n_out, N = n_in
  int mt, nt;         // tiles of each
};

struct DwTile {
  int e, m0, n0, row0, rows;
};

__device__ __forceinline__ DwTile dw_decode(const DwArgs& p, const int32_t* off, int t) {
  DwTile r;
  const int per = p.mt * p.nt;
  r.e = t / per;
  const int in = t - r.e * per, m = in / p.nt;
  r.m0 = m * 256;
  r.n0 = (in - m * p.nt) * 256;
  r.row0 = off[r.e];
  r.rows = off[r.e + 1] - r.row0;
  return r;
}

// The rows [left, the next multiple of 16) of a stage become zeros, by a warp.
__device__ __forceinline__ void dw_clear(uint8_t* a, uint8_t* b, int left, int lane) {
  for (int i = left * 8 + lane; i < ((left + 15) & ~15) * 8; i += 32)  // 16 bytes each
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      *reinterpret_cast<uint4*>(a + j * 8192 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
      *reinterpret_cast<uint4*>(b + j * 8192 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
}

__global__ void __launch_bounds__(kDwThreads, 1)
dw_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
          const DwArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sA = base;
  uint8_t* sB = sA + kDwStages * kDwHalf;
  uint8_t* sE = sB + kDwStages * kDwHalf;
  uint64_t* full = reinterpret_cast<uint64_t*>(sE + kDwWarps * 4096);
  uint64_t* empty = full + kDwStages;
  uint64_t* last = empty + kDwStages;  // the peer's copies of a segment's last stage
  uint64_t* dfull = last + kDwStages;
  uint64_t* dempty = dfull + 2;
  uint64_t* drain = dempty + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(drain + 1);
  int* s_abort = reinterpret_cast<int*>(s_tmem + 1);
  int* s_bad = s_abort + 1;
  int32_t* s_off = s_bad + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = tc::cluster_rank();
  const int first = blockIdx.x >> 1, stride = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kDwStages; ++s) {
      tc::mbar_init(&full[s], 2);  // on the leader: each CTA's word, and the copies' bytes
      tc::mbar_init(&empty[s], 1);
      tc::mbar_init(&last[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      tc::mbar_init(&dfull[a], 1);
      tc::mbar_init(&dempty[a], 2 * kDwWarps);
    }
    tc::mbar_init(drain, 1);
    *s_abort = 0;
    tc::mbar_init_fence();
    tc::tma_prefetch_map(&tmA);
    tc::tma_prefetch_map(&tmB);
  }
  pdl_wait_and_trigger();
  __syncwarp();
  tc::cluster_arrive();
  if (warp == 3) {  // a bad expert_off schedules nothing
    bool bad = false;
    for (int g = lane; g <= p.E; g += 32) {
      const int lo = p.expert_off[g], hi = g < p.E ? p.expert_off[g + 1] : lo;
      bad |= lo < 0 || hi < lo || hi > p.TK;
      s_off[g] = lo;
    }
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
      *s_bad = bad;
      if (bad) record_error(p.st, kStatusData, kBadPairRow, -1);
    }
  }
  __syncwarp();
  // the peer runs, and both CTAs' barriers are initialised before any remote signal
  tc::cluster_wait();
  if (warp == 2) {
    tc::tmem_alloc_pair(s_tmem, 512);
    tc::tmem_relinquish_pair();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *s_tmem;
  const int total = *s_bad ? 0 : p.E * p.mt * p.nt;
  volatile int* abort = s_abort;
  // A tile's columns: 256, or 128 where the matrix has no more; half of them staged by each CTA.

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA
    // The leader's barrier of a stage counts both CTAs' bytes. A segment's last stage, where it
    // holds rows that are cleared first, is different on the peer: its copies complete on a barrier
    // of its own, and its warp 1 gives the leader its word once the rows are cleared.
    const bool lead = tc::elect_one();
    uint32_t s = 0, ph = 1, it = 0, lph = 0;  // lph: bits of `last`'s phases
    uint32_t own = 0;                         // stages whose copies are counted by `last`
    bool ok = true;
    for (int t = first; t < total && ok; t += stride) {
      const DwTile tl = dw_decode(p, s_off, t);
      const int nb = tl.n0 + 128 < p.N ? 2 : 1, m0 = tl.m0 + (int)rank * 128, n0 = tl.n0 + (int)rank * 64 * nb;
      for (int r = 0; r < tl.rows; r += 64) {
        ok = tc::mbar_wait_warp(&empty[s], ph, abort);
        if (!ok) break;
        const bool cut = tl.rows - r < 64 && ((tl.rows - r) & 15) != 0;
        if (lead) {
          const uint32_t bytes = (2 + nb) * 8192, leader = tc::cluster_addr(&full[s], 0);
          uint32_t on = leader;
          if (rank == 0) {
            tc::mbar_expect_tx(&full[s], cut ? bytes : 2 * bytes);
          } else if (cut) {
            tc::mbar_expect_tx(&last[s], bytes);
            on = tc::cluster_addr(&last[s], 1);
          } else {
            tc::mbar_arrive_remote(leader);
          }
          for (int j = 0; j < 2; ++j)
            tc::tma_load_2d_pair(sA + s * kDwHalf + j * 8192, &tmA, on, m0 + 64 * j, tl.row0 + r);
          for (int j = 0; j < nb; ++j)
            tc::tma_load_2d_pair(sB + s * kDwHalf + j * 8192, &tmB, on, n0 + 64 * j, tl.row0 + r);
        }
        __syncwarp();
        own &= ~(1u << s);
        if (cut && rank == 1) {
          own |= 1u << s;
          lph ^= 1u << s;  // the phase that these copies complete is the one before
        }
        ++it;
        if (++s == kDwStages) { s = 0; ph ^= 1u; }
      }
    }
    if (lead) {
      if (!ok) {
        *abort = 1;
        record_error(p.st, kStatusTimeout, kTimeoutGemm, blockIdx.x);
      }
      // The copies in flight land before shared memory goes away, whichever role gave up: the
      // leader waits for both CTAs' (a barrier that the peer did not get to never completes: then
      // the limit is waited out once), the peer sees only its last stages' complete.
      volatile int never = 0;
      if (rank == 0) {
        for (uint32_t j = it > kDwStages ? it - kDwStages : 0; j < it; ++j)
          if (!tc::mbar_wait(&full[j % kDwStages], (j / kDwStages) & 1u, &never)) break;
      } else {
        for (int j = 0; j < kDwStages; ++j)
          if (own >> j & 1u) tc::mbar_wait(&last[j], (lph >> j & 1u) ^ 1u, &never);
        if (*abort) tc::wait_out();
      }
    }
    __syncwarp();
  } else if (warp == 1 && rank == 0) {
    // ---------------------------------------------------------------- MMA issuer (of the pair)
    const bool lead = tc::elect_one();
    uint32_t s = 0, ph = 0, d = 0, dph = 1;
    bool ok = true, in = false;
    for (int t = first; t < total && ok; t += stride) {
      const DwTile tl = dw_decode(p, s_off, t);
      if (tl.rows == 0) continue;
      const uint32_t idesc = tc::instr_desc(false, 256, tl.n0 + 128 < p.N ? 256 : 128) |
                             tc::kIdescTransA | tc::kIdescTransB;
      ok = tc::mbar_wait_warp(&dempty[d], dph, abort);
      if (!ok) break;
      tc::fence_after_sync();
      const uint32_t acc = tmem + d * 256;
      for (int r = 0; r < tl.rows; r += 64) {
        const int left = min(64, tl.rows - r);
        if (left & 15) {
          // the peer's zeros are acquired with its word
          ok = tc::mbar_wait_warp_shared(&full[s], ph, abort);
          if (!ok) break;
          dw_clear(sA + s * kDwHalf, sB + s * kDwHalf, left, lane);
        } else if (!in) {
          ok = tc::mbar_wait_warp(&full[s], ph, abort);
          if (!ok) break;
        }
        tc::fence_after_sync();
        const uint64_t ad = tc::sw128_mnmajor_desc(tc::smem_u32(sA + s * kDwHalf));
        const uint64_t bd = tc::sw128_mnmajor_desc(tc::smem_u32(sB + s * kDwHalf));
        uint64_t* e_bar = &empty[s];
        if (++s == kDwStages) { s = 0; ph ^= 1u; }
        const bool in_next = tc::mbar_test(&full[s], ph);
        if (lead) {
          const int steps = (left + 15) >> 4;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < steps) tc::mma_bf16_pair(acc, ad + 128 * k, bd + 128 * k, idesc, r > 0 || k > 0);
          tc::commit_pair(e_bar, 0x3);
        }
        in = __all_sync(0xffffffffu, in_next);
      }
      if (!ok) break;
      if (lead) tc::commit_pair(&dfull[d], 0x3);
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
      tc::commit_pair(drain, 0x1);
      tc::mbar_wait(drain, 0, &never);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- the peer's last rows
    uint32_t it = 0, lph = 0;
    bool ok = true;
    for (int t = first; t < total && ok; t += stride) {
      const DwTile tl = dw_decode(p, s_off, t);
      it += (tl.rows + 63) >> 6;
      if ((tl.rows & 15) == 0) continue;
      const uint32_t s = (it - 1) % kDwStages;
      ok = tc::mbar_wait_warp(&last[s], lph >> s & 1u, abort);
      if (!ok) break;
      lph ^= 1u << s;
      dw_clear(sA + s * kDwHalf, sB + s * kDwHalf, tl.rows & 63, lane);
      if (lane == 0) tc::mbar_arrive_cluster_shared(tc::cluster_addr(&full[s], 0));
    }
    if (!ok && lane == 0) {
      *abort = 1;
      record_error(p.st, kStatusTimeout, kTimeoutGemm, blockIdx.x);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- epilogue
    // Each warp 32 rows of kDwCols columns, in windows of 32 columns through 4 KB of its own
    // (16-byte chunks swizzled by row: no bank conflicts), added to and stored as whole lines. What
    // is added is loaded a window ahead.
    const int q = warp & 3, part = (warp - 4) >> 2;
    constexpr int kWins = kDwCols / 32;
    uint8_t* buf = sE + (warp - 4) * 4096;
    const int ch = lane & 7, sub = lane >> 3;
    uint32_t d = 0, dph = 0;
    bool ok = true;
    for (int t = first; t < total && ok; t += stride) {
      const DwTile tl = dw_decode(p, s_off, t);
      const int m0 = tl.m0 + (int)rank * 128 + q * 32, n0 = tl.n0 + part * kDwCols;
      const int mrows = min(32, p.M - m0), ncols = min(kDwCols, p.N - n0);  // may be below 1
      const size_t at = ((size_t)tl.e * p.M + m0 + sub) * p.N + n0 + ch * 4;
      const int nwin = mrows > 0 && ncols > 0 ? (ncols + 31) >> 5 : 0;
      float4 add[8];
      auto load = [&](int w) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          add[i] = i * 4 + sub < mrows && w * 32 + ch * 4 < ncols
                       ? __ldcs(reinterpret_cast<const float4*>(p.add + at + (size_t)(i * 4) * p.N + w * 32))
                       : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      };
      if (p.add) load(0);
      if (tl.rows > 0) {
        ok = tc::mbar_wait_warp(&dfull[d], dph, abort);
        if (!ok) break;
        tc::fence_after_sync();
      }
      const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + d * 256 + part * kDwCols;
#pragma unroll
      for (int w = 0; w < kWins; ++w) {
        if (w >= nwin) break;
        __syncwarp();  // TMEM loads are a whole warp's
        uint32_t v[32];
        if (tl.rows > 0) {
          tc::tmem_ld32(taddr + 32 * w, v);
          tc::tmem_ld_wait(v);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0u;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<uint4*>(buf + lane * 128 + ((j ^ (lane & 7)) << 4)) =
              make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        __syncwarp();
        float4 o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rr = i * 4 + sub;
          o[i] = *reinterpret_cast<const float4*>(buf + rr * 128 + ((ch ^ (rr & 7)) << 4));
          if (p.add) {
            o[i].x += add[i].x; o[i].y += add[i].y; o[i].z += add[i].z; o[i].w += add[i].w;
          }
        }
        if (p.add && w + 1 < kWins) load(w + 1);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i * 4 + sub < mrows && w * 32 + ch * 4 < ncols)
            __stcs(reinterpret_cast<float4*>(p.dw + at + (size_t)(i * 4) * p.N + w * 32), o[i]);
      }
      if (tl.rows > 0) {
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_remote(tc::cluster_addr(&dempty[d], 0));
        if (++d == 2) { d = 0; dph ^= 1u; }
      }
    }
    if (!ok && lane == 0) {
      *abort = 1;
      record_error(p.st, kStatusTimeout, kTimeoutGemm, blockIdx.x);
    }
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();  // no signal or copy of the other CTA is on its way here
  tc::fence_after_sync();
  if (warp == 2) tc::tmem_dealloc_pair(tmem, 512);
}

// ------------------------------------------------------------------ kept rows
// dst[r] = q[map[r]] times its scales, in the layer's type, for the rows of the segments; a map
// entry out of range gives a row of zeros. A warp a row, 8 values a lane at a time (stores of 512
// bytes in a row for bf16), eight loads ahead of their use.
// (The product can read its rows through map itself, by asynchronous copies, and none is written:
// its stores, which fill the load and store units' queues, then hold the copies up: 160 experts of
// 1536 x 5120, 49152 rows of 8192 tokens 1293 us, against 1040 with this copy.)
template <typename TE>
__global__ void __launch_bounds__(256)
widen_rows_kernel(const uint2* q, const float* scale, const int32_t* map, const int32_t* expert_off,
                  int E, int rows, int n_src, int cols, TE* dst, DeviceStatus* st) {
  pdl_wait_and_trigger();
  const int vecs = cols >> 3, nblk = (cols + 127) >> 7, lane = threadIdx.x & 31;
  const int begin = max(expert_off[0], 0), end = min(expert_off[E], rows);
  for (int r = begin + blockIdx.x * 8 + (threadIdx.x >> 5); r < end; r += gridDim.x * 8) {
    const int src = map ? map[r] : r;
    const bool in = (unsigned)src < (unsigned)n_src;
    if (!in && lane == 0) record_error(st, kStatusData, kBadPerm, r);
    const uint2* from = q + (in ? (size_t)src * vecs : 0);
    const float* sc = scale + (in ? (size_t)src * nblk : 0);
    for (int v0 = lane; v0 < vecs; v0 += 32 * 8) {
      uint2 w[8];
      float s[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int v = v0 + 32 * u;
        const bool has = in && v < vecs;
        w[u] = has ? __ldcg(from + v) : make_uint2(0u, 0u);
        s[u] = has ? __ldcg(sc + (v >> 4)) : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int v = v0 + 32 * u;
        if (v >= vecs) break;
        float f[8];
        const uint32_t b[2] = {w[u].x, w[u].y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 h = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(
              (__nv_fp8x2_storage_t)(b[i >> 1] >> (16 * (i & 1)) & 0xffffu), __NV_E4M3)));
          f[2 * i] = h.x * s[u];
          f[2 * i + 1] = h.y * s[u];
        }
        uint4* out = reinterpret_cast<uint4*>(dst + (size_t)r * cols + v * 8);
        constexpr int kVec = 16 / (int)sizeof(TE);
#pragma unroll
        for (int i = 0; i < 8 / kVec; ++i) out[i] = pack16(f + i * kVec, (const TE*)nullptr);
      }
    }
  }
}

// ------------------------------------------------------------------ fp32
// fp32 layers multiply in fp32 on the CUDA cores (the tensor cores' tf32 keeps 11 bits):
//   kind 0  y[r, n] = sum_k x[r, k] w[e, n, k]           rows x n_out, over n_in
//   kind 1  dx[r, k] = sum_n dy[r, n] w[e, n, k] (twice) rows x n_in, over n_out
//   kind 2  dw[e, n, k] = sum_r dy[r, n] x[r, k] (+ add)  n_out x n_in, over the rows
// Tiles of BM x 128, 256 threads with BM / 16 x 8 sums each (16 x 128: 2 x 4), 16 of the contraction at
// a time through shared memory, the next 16 in registers meanwhile.
struct F32Args {
  const float *a, *b, *a2, *b2, *add;
  float* out;
  const int32_t* expert_off;
  DeviceStatus* st;
  int E, TK, n_out, n_in;
};

template <int KIND, int BM>
__global__ void __launch_bounds__(256)
grouped_f32_kernel(const F32Args p) {
  constexpr int BN = 128, BK = 16, TM = BM == 16 ? 2 : BM / 16, TN = BM == 16 ? 4 : 8;
  constexpr int kTx = BN / TN;                  // threads along N
  __shared__ alignas(16) float As[BK][BM + 4];
  __shared__ alignas(16) float Bs[BK][BN + 4];
  __shared__ int32_t s_ts[kMaxGroups + 2], s_off[kMaxGroups + 2];
  pdl_wait_and_trigger();
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid < 32) {
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
      if (!bad && g < p.E) n = KIND == 2 ? (p.n_out + BM - 1) / BM : (s_off[g + 1] - s_off[g] + BM - 1) / BM;
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
  __syncthreads();
  const int N = KIND == 0 ? p.n_out : p.n_in, ntile = (N + BN - 1) / BN;
  const int total = s_ts[p.E] * ntile;
  const int tx = tid % kTx, ty = tid / kTx;
  int g = 0;
  for (int t = blockIdx.x; t < total; t += gridDim.x) {
    while (s_ts[g + 1] * ntile <= t) ++g;
    const int mt = s_ts[g + 1] - s_ts[g], local = t - s_ts[g] * ntile;
    const int n_tile = local / mt, n0 = n_tile * BN, m0 = (local - n_tile * mt) * BM;
    const int row0 = s_off[g], rows = s_off[g + 1] - row0;
    const int M = KIND == 2 ? p.n_out : rows;
    const int K1 = KIND == 0 ? p.n_in : KIND == 1 ? p.n_out : rows;
    const int nk1 = (K1 + BK - 1) / BK, nk = KIND == 1 && p.a2 ? 2 * nk1 : nk1;
    float acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = 0.0f;

    constexpr int kA = (BM * BK / 4 + 255) / 256, kB = BN * BK / 4 / 256;
    float4 ra[kA], rb[kB];
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto fetch = [&](int kb) {
      const bool second = kb >= nk1;
      const float* a = second ? p.a2 : p.a;
      const float* b = second ? p.b2 : p.b;
      const int k0 = (second ? kb - nk1 : kb) * BK;
#pragma unroll
      for (int i = 0; i < kA; ++i) {
        const int v = tid + i * 256;
        ra[i] = zero;
        if (v >= BM * BK / 4) continue;
        if (KIND == 2) {  // [row][n_out]
          const int k = v / (BM / 4), m = (v - k * (BM / 4)) * 4;
          if (k0 + k < K1 && m0 + m < M)
            ra[i] = *reinterpret_cast<const float4*>(a + (size_t)(row0 + k0 + k) * p.n_out + m0 + m);
        } else {
          const int m = v >> 2, k = (v & 3) * 4;
          if (m0 + m < M && k0 + k < K1)
            ra[i] = *reinterpret_cast<const float4*>(a + (size_t)(row0 + m0 + m) * K1 + k0 + k);
        }
      }
#pragma unroll
      for (int i = 0; i < kB; ++i) {
        const int v = tid + i * 256;
        rb[i] = zero;
        if (KIND == 0) {  // [n_out][n_in]
          const int n = v >> 2, k = (v & 3) * 4;
          if (n0 + n < N && k0 + k < K1)
            rb[i] = *reinterpret_cast<const float4*>(b + ((size_t)g * p.n_out + n0 + n) * p.n_in + k0 + k);
        } else {
          const int k = v >> 5, n = (v & 31) * 4;
          const size_t row = KIND == 1 ? (size_t)g * p.n_out + k0 + k : (size_t)row0 + k0 + k;
          if (k0 + k < K1 && n0 + n < N)
            rb[i] = *reinterpret_cast<const float4*>(b + row * p.n_in + n0 + n);
        }
      }
    };
    if (nk > 0) fetch(0);
    for (int kb = 0; kb < nk; ++kb) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kA; ++i) {
        const int v = tid + i * 256;
        if (v >= BM * BK / 4) continue;
        const float f[4] = {ra[i].x, ra[i].y, ra[i].z, ra[i].w};
        if (KIND == 2) {
          const int k = v / (BM / 4), m = (v - k * (BM / 4)) * 4;
          *reinterpret_cast<float4*>(&As[k][m]) = ra[i];
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) As[(v & 3) * 4 + j][v >> 2] = f[j];
        }
      }
#pragma unroll
      for (int i = 0; i < kB; ++i) {
        const int v = tid + i * 256;
        const float f[4] = {rb[i].x, rb[i].y, rb[i].z, rb[i].w};
        if (KIND == 0) {
#pragma unroll
          for (int j = 0; j < 4; ++j) Bs[(v & 3) * 4 + j][v >> 2] = f[j];
        } else {
          *reinterpret_cast<float4*>(&Bs[v >> 5][(v & 31) * 4]) = rb[i];
        }
      }
      __syncthreads();
      if (kb + 1 < nk) fetch(kb + 1);
#pragma unroll
      for (int k = 0; k < BK; ++k) {
        float a[TM], b[TN];
#pragma unroll
        for (int i = 0; i < TM; ++i) a[i] = As[k][ty * TM + i];
#pragma unroll
        for (int j = 0; j < TN; j += 4) {
          const float4 f = *reinterpret_cast<const float4*>(&Bs[k][tx * 4 + j * kTx]);
          b[j] = f.x; b[j + 1] = f.y; b[j + 2] = f.z; b[j + 3] = f.w;
        }
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
      }
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int m = m0 + ty * TM + i;
      if (m >= M) continue;
      const size_t row = (KIND == 2 ? (size_t)g * p.n_out : (size_t)row0) + m;
#pragma unroll
      for (int j = 0; j < TN; j += 4) {
        const int n = n0 + tx * 4 + j * kTx;
        if (n >= N) continue;
        float4 o = make_float4(acc[i][j], acc[i][j + 1], acc[i][j + 2], acc[i][j + 3]);
        if (KIND == 2 && p.add) {
          const float4 f = *reinterpret_cast<const float4*>(p.add + row * N + n);
          o.x += f.x; o.y += f.y; o.z += f.z; o.w += f.w;
        }
        *reinterpret_cast<float4*>(p.out + row * N + n) = o;
      }
    }
  }
}

template <int KIND, int BM>
cudaError_t run_f32(const F32Args& p, long long tiles, cudaStream_t s) {
  const int grid = (int)std::min<long long>(std::max<long long>(tiles, 1), (long long)device_sms() * 4);
  SMOE_LAUNCH((grouped_f32_kernel<KIND, BM>), grid, 256, 0, s, p);
  return cudaGetLastError();
}

// Rows an expert from which the 64-row tiles take over from the 16-row ones.
constexpr int kF32Rows = 24;

}  // namespace

int device_sms() {
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n > 0 ? n : 148;
}

void product_ws_layout(const smoe_desc& d, ProductLayout* L) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) / 256 * 256;
    return o;
  };
  L->status = take(256);
  L->tiles = take(4 * (kMaxGroups + 2));
  L->rows = take((size_t)d.T * d.K * std::max(d.d, d.F) * elem_size(d));
  L->total = off;
}

cudaError_t launch_expert_rows(const smoe_desc& d, int n_out, int n_in, const void* a, const void* w,
                               const void* a2, const void* w2, bool transposed,
                               const int32_t* expert_off, void* out, void* ws, cudaStream_t s) {
  if (d.dtype != SMOE_F32)
    return launch_expert_rows_bf16(d, n_out, n_in, a, w, a2, w2, transposed, expert_off, out, ws, s);
  const int TK = d.T * d.K;
  const F32Args p{static_cast<const float*>(a), static_cast<const float*>(w),
                  static_cast<const float*>(a2), static_cast<const float*>(w2), nullptr,
                  static_cast<float*>(out), expert_off, static_cast<DeviceStatus*>(ws), d.E, TK, n_out, n_in};
  const bool few = (long long)TK < (long long)kF32Rows * d.E;
  const long long tiles = ((long long)ceil_div(TK, few ? 16 : 64) + std::min(TK, d.E)) *
                          ceil_div(transposed ? n_in : n_out, 128);
  if (transposed) return few ? run_f32<1, 16>(p, tiles, s) : run_f32<1, 64>(p, tiles, s);
  return few ? run_f32<0, 16>(p, tiles, s) : run_f32<0, 64>(p, tiles, s);
}

cudaError_t launch_expert_dw(const smoe_desc& d, int n_out, int n_in, const void* dy, const void* x,
                             const int32_t* expert_off, const float* add, float* dw, void* ws,
                             cudaStream_t s) {
  const int TK = d.T * d.K;
  DeviceStatus* st = static_cast<DeviceStatus*>(ws);
  if (d.dtype == SMOE_F32) {
    const F32Args p{static_cast<const float*>(dy), static_cast<const float*>(x), nullptr, nullptr, add,
                    dw, expert_off, st, d.E, TK, n_out, n_in};
    return run_f32<2, 64>(p, (long long)d.E * ceil_div(n_out, 64) * ceil_div(n_in, 128), s);
  }
  alignas(64) CUtensorMap A, B;
  if (!encode_tmap_2d(&A, dy, false, TK, n_out, 64, 64) || !encode_tmap_2d(&B, x, false, TK, n_in, 64, 64))
    return cudaErrorInvalidValue;
  const cudaError_t e = cudaFuncSetAttribute(dw_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kDwSmem);
  if (e != cudaSuccess) return e;
  const DwArgs p{expert_off, add, dw, st, d.E, TK, n_out, n_in, ceil_div(n_out, 256), ceil_div(n_in, 256)};
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(2 * (int)std::min<long long>(device_sms() / 2, (long long)d.E * p.mt * p.nt));
  cfg.blockDim = dim3(kDwThreads);
  cfg.dynamicSmemBytes = kDwSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  SMOE_COUNT_LAUNCH(1);
  return cudaLaunchKernelEx(&cfg, dw_kernel, A, B, p);
}

cudaError_t launch_widen_rows(const smoe_desc& d, int cols, const void* xq, const float* scale,
                              const int32_t* row_src, const int32_t* expert_off, void* ws,
                              const void** rows_out, cudaStream_t s) {
  ProductLayout L;
  product_ws_layout(d, &L);
  const int TK = d.T * d.K;
  DeviceStatus* st = ws_ptr<DeviceStatus>(ws, L.status);
  void* dst = ws_ptr<char>(ws, L.rows);
  *rows_out = dst;
  const int grid = std::min(ceil_div(TK, 8), 152 * 8);
  auto run = [&](auto* out) -> cudaError_t {
    using TE = std::remove_pointer_t<decltype(out)>;
    SMOE_LAUNCH((widen_rows_kernel<TE>), grid, 256, 0, s, static_cast<const uint2*>(xq), scale, row_src,
                expert_off, d.E, TK, row_src ? d.T : TK, cols, out, st);
    return cudaGetLastError();
  };
  return d.dtype == SMOE_F32 ? run(static_cast<float*>(dst)) : run(static_cast<__nv_bfloat16*>(dst));
}

}  // namespace smoe
