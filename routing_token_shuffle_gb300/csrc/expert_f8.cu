// Expert products in 8-bit floating point (e4m3) with a scale for each block of 128 contraction
// channels, one per row on the token side and one per 128 output channels on the weight side:
//   out[r, n] = sum_b xs[s(r), b] ws[e(r), n / 128, b] sum_{k in b} xq[s(r), k] wq[e(r), n, k].
//
// The scales are fp32 of any value, so a block's sum leaves the tensor core before it is
// scaled: tcgen05.mma (kind::f8f6f4) gives each block of 128 in a TMEM buffer of its own, and
// the epilogue warps multiply it by its two scales and add it to accumulators in registers
// while the next blocks' MMAs run into the other buffers. One block costs the epilogue one TMEM
// read and one FMA a value, less than the MMAs' own time.
//
// One persistent CTA per SM walks the tiles (expert, channel tile, row tile), row tiles fastest
// so that neighbours share the weights through L2. The token rows are gathered through row_src by
// 16-byte asynchronous copies, so no dispatched copy of them is made; weights come by TMA.
//   wide   128 rows x 256 channels: the rows are the MMA's M, so that a thread of the epilogue
//          holds one row and a block's scale is one number for it
//   narrow 128 channels x at most 64 rows: for batches that do not fill an expert's tile the
//          weights' stream is the work; the channels are the MMA's M, its N the rows rounded up
//          to 16, and the row scales are read from shared memory
//
// Measured: 384 rows over 160 experts of 5120 to 1536 channels (narrow) 181 us, 6.3 TB/s of
// weights; 131072 rows over 128 experts of 2048 to 768 (wide) 229 us, 1.80 PFLOP/s; 2002 rows over
// 8 experts of 4096 to 14336, fp32 out, 152 us. What bounds the wide form: without its stores the
// prefill product took 205 us, without the epilogue's FMAs and TMEM loads besides 170, without the
// gathering and the weights' loads besides 125: the work of each of the three overlaps the MMAs (96 us
// at the nominal rate) and still takes from them, and a block's way from the MMAs to the epilogue and
// back (two TMEM buffers of 256 columns are all there is) takes longer than its four MMAs.
#include <algorithm>

#include "tc_common.cuh"

namespace smoe {
namespace {

template <bool WIDE> struct F8Cfg;
// Registers hold the accumulators: 128 a thread in the wide form (8 epilogue warps), 64 in the
// narrow one (4 warps).
template <> struct F8Cfg<true> {
  static constexpr int kThreads = 512, kGather = 4, kStages = 3, kChan = 256, kRows = 128, kBufs = 2, kCols = 256;
  static constexpr int kStage = 48 * 1024, kEpiWarps = 8, kEpiSmem = 8 * 8192;
  static constexpr int kScale = 2 * 2 * 128 * 16;  // scales: two slots of four blocks, both halves
};
template <> struct F8Cfg<false> {
  static constexpr int kThreads = 256, kGather = 2, kStages = 8, kChan = 128, kRows = 64, kBufs = 8, kCols = 64;
  static constexpr int kStage = 24 * 1024, kEpiWarps = 4, kEpiSmem = 4 * 256, kScale = 0;
};

template <bool WIDE>
constexpr size_t f8_smem() {
  using C = F8Cfg<WIDE>;
  return 1024 + (size_t)C::kStages * C::kStage + C::kEpiSmem + C::kScale +
         8 * (2 * C::kStages + 2 * C::kBufs + 5) + 16 +
         4 * 2 * (kMaxGroups + 2);
}

struct F8Args {
  const uint8_t* xq;
  const float* xs;
  const int32_t* row_src;     // nullable
  const int32_t* expert_off;
  const float* ws;
  void* out;
  DeviceStatus* st;
  int E, TK, n_src, N, KD;    // n_src: rows of xq
};

struct F8Tile {
  int g, n0, rows;            // expert, first channel, rows of the tile
  int row0;                   // first dispatched row
};

// Row tiles of each expert (s_ts, prefix) and their first rows (s_off), by one warp. A bad
// expert_off schedules nothing.
template <int ROWS>
__device__ __forceinline__ void f8_table(const F8Args& p, int32_t* s_ts, int32_t* s_off, int lane) {
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
    const int n = !bad && g < p.E ? (s_off[g + 1] - s_off[g] + ROWS - 1) / ROWS : 0;
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

// Tile t of a walk whose tiles ascend; g: the last one's expert. Narrow: an expert's row tiles
// are equally long, not 64 rows and a rest.
template <bool WIDE>
__device__ __forceinline__ F8Tile f8_decode(const F8Args& p, const int32_t* ts, const int32_t* off,
                                            int ntile, int t, int& g) {
  using C = F8Cfg<WIDE>;
  while (ts[g + 1] * ntile <= t) ++g;
  const int mt = ts[g + 1] - ts[g], local = t - ts[g] * ntile;
  const int n_tile = local / mt, m_tile = local - n_tile * mt;
  const int rows = off[g + 1] - off[g];
  const int step = WIDE ? C::kRows : ((rows + mt - 1) / mt + 15) & ~15;
  F8Tile r;
  r.g = g;
  r.n0 = n_tile * C::kChan;
  r.rows = min(step, rows - m_tile * step);
  r.row0 = off[g] + m_tile * step;
  return r;
}

template <bool WIDE, typename TO>
__global__ void __launch_bounds__(F8Cfg<WIDE>::kThreads, 1)
f8_gemm_kernel(const __grid_constant__ CUtensorMap tmW,  // weights as 16-bit pairs, 128-row box
               const __grid_constant__ CUtensorMap tmO,  // wide: the output, boxes of 32 rows x 128 bytes
               const F8Args p) {
  using C = F8Cfg<WIDE>;
  constexpr int kWBytes = C::kChan * 128, kXBytes = C::kRows * 128;
  constexpr int kGatherWarps = C::kGather, kGatherRows = C::kRows / kGatherWarps;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sW = base;                                  // [kStages][kChan x 128 bytes]
  uint8_t* sX = sW + C::kStages * kWBytes;             // [kStages][kRows x 128 bytes]
  uint8_t* sE = sX + C::kStages * kXBytes;             // epilogue warps' own space
  float4* sS = reinterpret_cast<float4*>(sE + C::kEpiSmem);  // wide: [slot][half][row]
  uint64_t* full = reinterpret_cast<uint64_t*>(sE + C::kEpiSmem + C::kScale);
  uint64_t* empty = full + C::kStages;
  uint64_t* dfull = empty + C::kStages;
  uint64_t* dempty = dfull + C::kBufs;
  uint64_t* drain = dempty + C::kBufs;
  uint64_t* sfull = drain + 1;
  uint64_t* sempty = sfull + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(sempty + 2);
  int* s_abort = reinterpret_cast<int*>(s_tmem + 1);
  int32_t* s_ts = reinterpret_cast<int32_t*>(s_abort + 3);
  int32_t* s_off = s_ts + kMaxGroups + 2;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      tc::mbar_init(&full[s], 1 + 32 * kGatherWarps);
      tc::mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      tc::mbar_init(&dfull[b], 1);
      tc::mbar_init(&dempty[b], C::kEpiWarps);
    }
    tc::mbar_init(drain, 1);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sfull[i], 2);
      tc::mbar_init(&sempty[i], C::kEpiWarps);
    }
    *s_abort = 0;
    tc::mbar_init_fence();
    tc::tma_prefetch_map(&tmW);
    if (WIDE) tc::tma_prefetch_map(&tmO);
  }
  pdl_wait_and_trigger();
  __syncwarp();
  if (warp == 3) f8_table<C::kRows>(p, s_ts, s_off, lane);
  if (warp == 2) {
    tc::tmem_alloc(s_tmem, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *s_tmem;
  const int ntile = (p.N + C::kChan - 1) / C::kChan;
  const int total = s_ts[p.E] * ntile;
  const int nk = (p.KD + 127) / 128;
  volatile int* abort = s_abort;
  // Wide: 512 threads of 128 registers at launch, 2 x 72 + 2 x 184 = 4 x 128 from here on.
  if (warp < (WIDE ? 8 : 4)) {
  if (WIDE) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  if (warp == 0) {
    // ---------------------------------------------------------------- weights
    const bool lead = tc::elect_one();
    uint32_t s = 0, ph = 1, it = 0;
    bool ok = true;
    int g = 0;
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
      const F8Tile tl = f8_decode<WIDE>(p, s_ts, s_off, ntile, t, g);
      const int wrow = tl.g * p.N + tl.n0;
      // the tile's second 128 channels, where the matrix has them
      const bool two = WIDE && tl.n0 + 128 < p.N;
      for (int kb = 0; kb < nk; ++kb) {
        ok = tc::mbar_wait_warp(&empty[s], ph, abort);
        if (!ok) break;
        if (lead) {
          tc::mbar_expect_tx(&full[s], two ? 2 * 128 * 128 : 128 * 128);
          tc::tma_load_2d(sW + s * kWBytes, &tmW, &full[s], kb * 64, wrow);
          if (two) tc::tma_load_2d(sW + s * kWBytes + 128 * 128, &tmW, &full[s], kb * 64, wrow + 128);
        }
        __syncwarp();
        ++it;
        if (++s == C::kStages) { s = 0; ph ^= 1u; }
      }
    }
    if (lead) {
      if (!ok) {
        *abort = 1;
        record_error(p.st, kStatusTimeout, kTimeoutGemm, blockIdx.x);
      }
      // The copies in flight land before shared memory goes away, whichever role gave up. A
      // stage that the gathering warps did not get to never completes: then the limit is
      // waited out once.
      volatile int never = 0;
      for (uint32_t j = it > C::kStages ? it - C::kStages : 0; j < it; ++j)
        if (!tc::mbar_wait(&full[j % C::kStages], (j / C::kStages) & 1u, &never)) break;
    }
    __syncwarp();
  } else if (WIDE && (warp == 2 || warp == 3)) {
    // ---------------------------------------------------------------- scales
    // The product of both scales, for four blocks at a time and both halves of the channels. (Loaded
    // by the epilogue warps, whose load instructions then queue behind the gathering warps'
    // copies, 131072 rows of 2048 to 768 channels took 269 us; now 246.)
    uint32_t slot = 0, ph = 1;
    bool ok = true;
    int g = 0;
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
      const F8Tile tl = f8_decode<WIDE>(p, s_ts, s_off, ntile, t, g);
      const int nblk = (p.N + 127) / 128, r0 = (warp - 2) * 64 + lane;
      const float* ws = p.ws + ((size_t)tl.g * nblk + tl.n0 / 128) * nk;
      const int second = tl.n0 + 128 < p.N ? nk : 0;
      int src[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int r = r0 + 32 * u;
        src[u] = r >= tl.rows ? -1 : p.row_src ? __ldcg(p.row_src + tl.row0 + r) : tl.row0 + r;
      }
      auto four = [&](const float* f, int k0, bool in) {
        if ((nk & 3) == 0)
          return in ? __ldcg(reinterpret_cast<const float4*>(f + k0)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float4 v;
        v.x = in ? __ldcg(f + k0) : 0.0f;
        v.y = in && k0 + 1 < nk ? __ldcg(f + k0 + 1) : 0.0f;
        v.z = in && k0 + 2 < nk ? __ldcg(f + k0 + 2) : 0.0f;
        v.w = in && k0 + 3 < nk ? __ldcg(f + k0 + 3) : 0.0f;
        return v;
      };
      for (int k0 = 0; k0 < nk; k0 += 4) {
        float4 x[2], w[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const bool in = (unsigned)src[u] < (unsigned)p.n_src;
          x[u] = four(p.xs + (in ? (size_t)src[u] * nk : 0), k0, in);
          w[u] = four(ws + u * second, k0, true);
        }
        ok = tc::mbar_wait_warp(&sempty[slot], ph, abort);
        if (!ok) break;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            sS[(slot * 2 + h) * 128 + r0 + 32 * u] =
                make_float4(x[u].x * w[h].x, x[u].y * w[h].y, x[u].z * w[h].z, x[u].w * w[h].w);
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sfull[slot]);
        if (++slot == 2) { slot = 0; ph ^= 1u; }
      }
    }
    if (!ok && lane == 0) {
      *abort = 1;
      record_error(p.st, kStatusTimeout, kTimeoutGemm, blockIdx.x);
    }
    __syncwarp();
  } else if (WIDE ? warp >= 4 : warp >= 2) {
    // ---------------------------------------------------------------- rows
    // Four rows of 128 bytes an instruction, into the 128-byte-swizzled stage. Rows past the
    // tile's are zeros (narrow: up to the MMA's columns).
    const int c = lane & 7, sub = (warp - (WIDE ? 4 : 2)) * kGatherRows + (lane >> 3);
    constexpr int kIter = kGatherRows / 4;
    uint32_t s = 0, ph = 1;
    bool ok = true;
    int g = 0;
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
      const F8Tile tl = f8_decode<WIDE>(p, s_ts, s_off, ntile, t, g);
      const int used = WIDE ? C::kRows : (tl.rows + 15) & ~15;
      // (all loads before the first check: one latency a tile, not one a row)
      int id[kIter];
#pragma unroll
      for (int i = 0; i < kIter; ++i) {
        const int r = sub + 4 * i;
        id[i] = r >= tl.rows ? -1 : p.row_src ? __ldcg(p.row_src + tl.row0 + r) : tl.row0 + r;
      }
#pragma unroll
      for (int i = 0; i < kIter; ++i)
        if ((unsigned)id[i] >= (unsigned)p.n_src) {
          if (sub + 4 * i < tl.rows && tl.n0 == 0 && c == 0)
            record_error(p.st, kStatusData, kBadPerm, tl.row0 + sub + 4 * i);
          id[i] = -1;
        }
      for (int kb = 0; kb < nk; ++kb) {
        ok = tc::mbar_wait_warp(&empty[s], ph, abort);
        if (!ok) break;
        const uint32_t dst = tc::smem_u32(sX + s * kXBytes);
        const int at = kb * 128 + c * 16;
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
          const int r = sub + 4 * i;
          const bool in = id[i] >= 0 && at < p.KD;
          if (r < used)
            tc::cp_async16(dst + r * 128 + ((c ^ (r & 7)) << 4),
                           p.xq + (in ? (size_t)id[i] * p.KD + at : 0), in ? 16u : 0u);
        }
        tc::cp_async_arrive(&full[s]);
        if (++s == C::kStages) { s = 0; ph ^= 1u; }
      }
    }
    tc::cp_async_wait_all();
    if (!ok && lane == 0) {
      *abort = 1;
      record_error(p.st, kStatusTimeout, kTimeoutGemm, blockIdx.x);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    // (The halves of a tile's channels as MMAs of N = 128 into buffers of their own, so that one
    // half is read while the other's run: 131072 rows of 2048 to 768 channels 306 us, against 274.)
    const bool lead = tc::elect_one();
    uint32_t s = 0, ph = 0, b = 0, bph = 1;
    bool ok = true, in = false, free = false;
    int g = 0;
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
      const F8Tile tl = f8_decode<WIDE>(p, s_ts, s_off, ntile, t, g);
      const uint32_t idesc =
          WIDE ? tc::instr_desc_f8(128, tl.n0 + 128 < p.N ? 256 : 128) : tc::instr_desc_f8(128, (tl.rows + 15) & ~15);
      for (int kb = 0; kb < nk; ++kb) {
        if (!in) ok = tc::mbar_wait_warp(&full[s], ph, abort);
        if (!ok) break;
        // the gathered rows were written through the generic proxy
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        const uint64_t wd = tc::sw128_kmajor_desc(tc::smem_u32(sW + s * kWBytes));
        const uint64_t xd = tc::sw128_kmajor_desc(tc::smem_u32(sX + s * kXBytes));
        const uint32_t acc = tmem + b * C::kCols;
        uint64_t *e_bar = &empty[s], *d_bar = &dfull[b];
        // (last before the MMAs: the hand-over of a buffer is what this loop waits for)
        if (!free) ok = tc::mbar_wait_warp(&dempty[b], bph, abort);
        if (!ok) break;
        tc::fence_after_sync();
        if (lead) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc::mma_f8(acc, (WIDE ? xd : wd) + 2 * k, (WIDE ? wd : xd) + 2 * k, idesc, k > 0);
          tc::commit(d_bar);
          tc::commit(e_bar);
        }
        __syncwarp();
        if (++s == C::kStages) { s = 0; ph ^= 1u; }
        if (++b == C::kBufs) { b = 0; bph ^= 1u; }
        const bool in_next = tc::mbar_test(&full[s], ph), free_next = tc::mbar_test(&dempty[b], bph);
        in = __all_sync(0xffffffffu, in_next);
        free = __all_sync(0xffffffffu, free_next);
      }
    }
    if (lead) {
      if (!ok) {
        *abort = 1;
        record_error(p.st, kStatusTimeout, kTimeoutGemm, blockIdx.x);
      }
      // wait for every MMA this thread issued before TMEM is released
      volatile int never = 0;
      tc::commit(drain);
      tc::mbar_wait(drain, 0, &never);
    }
    __syncwarp();
  }
  } else if (WIDE) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    // ---------------------------------------------------------------- epilogue, wide
    // warps 8-11 the tile's first 128 channels, 12-15 the other 128; a thread holds one row.
    // (A tile's last channels may lie past the matrix: they are not stored. A half that has none
    // reads what its TMEM holds, and stores nothing.)
    // (In pairs, by fma.rn.f32x2, 131072 rows of 2048 to 768 channels took 297 us, against 269.)
    const int q = warp & 3, half = (warp - 8) >> 2, r = q * 32 + lane;
    uint8_t* buf = sE + (warp - 8) * 8192;
    uint32_t b = 0, bph = 0, slot = 0, sph = 0;
    bool ok = true;
    int g = 0;
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
      F8Tile tl = f8_decode<WIDE>(p, s_ts, s_off, ntile, t, g);
      tl.n0 += 128 * half;
      // a row without a token is zero whatever the weights are (0 NaN is not); looked at below
      int src = 0;
      if (p.row_src && r < tl.rows) src = __ldcg(p.row_src + tl.row0 + r);
      float acc[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i] = 0.0f;
      float sc[4];
#pragma unroll 1
      for (int kb = 0; kb < nk; ++kb) {
        if ((kb & 3) == 0) {
          ok = tc::mbar_wait_warp(&sfull[slot], sph, abort);
          if (!ok) break;
          const float4 f = sS[(slot * 2 + half) * 128 + r];
          sc[0] = f.x; sc[1] = f.y; sc[2] = f.z; sc[3] = f.w;
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sempty[slot]);
          if (++slot == 2) { slot = 0; sph ^= 1u; }
        }
        const float now = sc[0];
        sc[0] = sc[1]; sc[1] = sc[2]; sc[2] = sc[3];
        ok = tc::mbar_wait_warp(&dfull[b], bph, abort);
        if (!ok) break;
        tc::fence_after_sync();
        const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + b * C::kCols + half * 128;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          tc::tmem_ld32(taddr + 32 * c, v);
          tc::tmem_ld_wait(v);
          if (c == 3) {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&dempty[b]);
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[32 * c + j] = fmaf(__uint_as_float(v[j]), now, acc[32 * c + j]);
        }
        if (++b == C::kBufs) { b = 0; bph ^= 1u; }
      }
      if (!ok) break;
      if ((unsigned)src >= (unsigned)p.n_src) {
#pragma unroll
        for (int i = 0; i < 128; ++i) acc[i] = 0.0f;
      }
      // 32 rows x 128 bytes, two such windows at a time, through the warp's own 8 KB (16-byte
      // chunks swizzled by row as TMA reads them: no bank conflicts), stored by TMA, or where
      // the tile's rows end inside by the warp. (Read back and stored by the warp throughout,
      // in windows of 64 bytes: 246 us.)
      constexpr int kVec = 16 / (int)sizeof(TO), kWin = 8 * kVec;
      const int row = tl.row0 + q * 32, rows = min(32, tl.rows - q * 32);
#pragma unroll
      for (int c = 0; c < 128; c += 2 * kWin) {
        if (lane == 0) tc::bulk_wait_read();
        __syncwarp();
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(buf + w * 4096 + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                pack16(acc + c + w * kWin + j * kVec, (const TO*)nullptr);
        tc::fence_async_shared();
        __syncwarp();
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int col = tl.n0 + c + w * kWin;
          if (col >= p.N) break;
          if (rows == 32) {
            if (lane == 0) tc::tma_store_2d(&tmO, buf + w * 4096, col, row);
          } else {
            const int ch = lane & 7;
            for (int rr = lane >> 3; rr < rows; rr += 4)
              if (col + ch * kVec < p.N)
                *reinterpret_cast<uint4*>(static_cast<TO*>(p.out) + (size_t)(row + rr) * p.N + col + ch * kVec) =
                    *reinterpret_cast<const uint4*>(buf + w * 4096 + rr * 128 + ((ch ^ (rr & 7)) << 4));
          }
        }
        if (lane == 0) tc::bulk_commit();
      }
    }
    if (lane == 0) tc::bulk_wait();  // before the shared memory goes away
    if (!ok && lane == 0) {
      *abort = 1;
      record_error(p.st, kStatusTimeout, kTimeoutGemm, blockIdx.x);
    }
  } else {
    // ---------------------------------------------------------------- epilogue, narrow
    // a thread holds one channel; each warp keeps the block's 64 row scales for itself
    const int q = warp & 3;
    float* s_sc = reinterpret_cast<float*>(sE) + q * 64;
    uint32_t b = 0, bph = 0;
    bool ok = true;
    int g = 0;
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
      const F8Tile tl = f8_decode<WIDE>(p, s_ts, s_off, ntile, t, g);
      const int chan = tl.n0 + q * 32 + lane, used = (tl.rows + 15) & ~15;
      const float* xs[2];
      bool has[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int r = lane + 32 * u;
        int src = -1;
        if (r < tl.rows) src = p.row_src ? __ldcg(p.row_src + tl.row0 + r) : tl.row0 + r;
        has[u] = (unsigned)src < (unsigned)p.n_src;
        xs[u] = p.xs + (has[u] ? (size_t)src * nk : 0);
      }
      const float* ws = p.ws + ((size_t)tl.g * ((p.N + 127) / 128) + tl.n0 / 128) * nk;
      float acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0.0f;
      // scales of the next two blocks
      float w[2], s0[2], s1[2];
      auto load = [&](int kb, int i) {
        const bool in = kb < nk;
        w[i] = in ? __ldcg(ws + kb) : 0.0f;
        s0[i] = in && has[0] ? __ldcg(xs[0] + kb) : 0.0f;
        s1[i] = in && has[1] ? __ldcg(xs[1] + kb) : 0.0f;
      };
      load(0, 0);
      load(1, 1);
      for (int kb = 0; kb < nk; ++kb) {
        __syncwarp();
        s_sc[lane] = s0[0] * w[0];
        s_sc[lane + 32] = s1[0] * w[0];
        __syncwarp();
        w[0] = w[1];
        s0[0] = s0[1];
        s1[0] = s1[1];
        load(kb + 2, 1);
        ok = tc::mbar_wait_warp(&dfull[b], bph, abort);
        if (!ok) break;
        tc::fence_after_sync();
        const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + b * C::kCols;
#pragma unroll
        for (int c = 0; c < 64; c += 16) {
          if (c >= used) break;
          float v[16];
          tc::tmem_ld16(taddr + c, v);
          if (c + 16 >= used) {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&dempty[b]);
          }
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 f = *reinterpret_cast<const float4*>(s_sc + c + i);
            acc[c + i] = fmaf(v[i], f.x, acc[c + i]);
            acc[c + i + 1] = fmaf(v[i + 1], f.y, acc[c + i + 1]);
            acc[c + i + 2] = fmaf(v[i + 2], f.z, acc[c + i + 2]);
            acc[c + i + 3] = fmaf(v[i + 3], f.w, acc[c + i + 3]);
          }
        }
        if (++b == C::kBufs) { b = 0; bph ^= 1u; }
      }
      if (!ok) break;
      // a row without a token is zero whatever the weights are (0 NaN is not)
      const uint32_t some[2] = {__ballot_sync(0xffffffffu, has[0]), __ballot_sync(0xffffffffu, has[1])};
      if (chan < p.N) {
        TO* out = static_cast<TO*>(p.out) + (size_t)tl.row0 * p.N + chan;
#pragma unroll
        for (int i = 0; i < 64; ++i, out += p.N)
          if (i < tl.rows) *out = Elem<TO>::from_f32(some[i >> 5] >> (i & 31) & 1u ? acc[i] : 0.0f);
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
  tc::fence_after_sync();
  if (warp == 2) tc::tmem_dealloc(tmem, 512);
}

// From this many rows an expert on average the wide tiles, where they are enough to go round: a
// weight passes once for 128 rows, not 64, and the epilogue's work is shared by eight warps.
// Measured (us, wide and narrow; rows an expert): 160 experts of 5120 to 1536 channels, 2: 177 and
// 171, 8: 208 and 206, 16: 211 and 213, 32: 216 and 238, 64: 217 and 344; 8 of 4096 to 14336, 2: 74
// and 71, 8: 79 and 82, 16: 80 and 97, 64: 83 and 153; 128 of 2048 to 768, 4: 44 and 40, 8: 45 and
// 47, 32: 48 and 56. One expert of 5120 to 5120 (20 wide tiles for 152 SMs), 16: 27 and 15, 64: 26
// and 23.
constexpr int kWideRows = 12, kWideRowsAnyhow = 96;

template <bool WIDE, typename TO>
cudaError_t run_f8(const F8Args& p, const void* wq, long long tile_bound, cudaStream_t s) {
  alignas(64) CUtensorMap tw, to;
  constexpr bool kF32 = sizeof(TO) == 4;
  if (!encode_tmap_2d(&tw, wq, false, (uint64_t)p.E * p.N, p.KD / 2, 128, 64) ||
      (WIDE && !encode_tmap_2d(&to, p.out, kF32, p.TK, p.N, 32, kF32 ? 32 : 64)))
    return cudaErrorInvalidValue;
  if (!WIDE) to = tw;  // (not used)
  auto kern = f8_gemm_kernel<WIDE, TO>;
  const int smem = (int)f8_smem<WIDE>();
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int grid = (int)std::min<long long>(device_sms(), std::max<long long>(tile_bound, 1));
  SMOE_LAUNCH(kern, grid, F8Cfg<WIDE>::kThreads, smem, s, tw, to, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_expert_matmul_f8(const smoe_desc& d, int n_out, int n_in, const void* xq,
                                    const float* xs, const int32_t* row_src,
                                    const int32_t* expert_off, const void* wq, const float* w_scale,
                                    void* out, void* ws, cudaStream_t s) {
  const int TK = d.T * d.K;
  const F8Args p{static_cast<const uint8_t*>(xq), xs, row_src, expert_off, w_scale, out,
                 static_cast<DeviceStatus*>(ws), d.E, TK, row_src ? d.T : TK, n_out, n_in};
  const long long few = (long long)std::max(d.E, ceil_div(TK, 128)) * ceil_div(n_out, 256);
  const bool wide = (long long)TK >= (long long)(2 * few >= device_sms() ? kWideRows : kWideRowsAnyhow) * d.E;
  // no more tiles than this, whatever the rows' spread over the experts
  const long long bound = ((long long)ceil_div(TK, wide ? 128 : 64) + std::min(TK, d.E)) *
                          ceil_div(n_out, wide ? 256 : 128);
  if (d.dtype == SMOE_F32) return wide ? run_f8<true, float>(p, wq, bound, s) : run_f8<false, float>(p, wq, bound, s);
  return wide ? run_f8<true, __nv_bfloat16>(p, wq, bound, s) : run_f8<false, __nv_bfloat16>(p, wq, bound, s);
}

}  // namespace smoe
