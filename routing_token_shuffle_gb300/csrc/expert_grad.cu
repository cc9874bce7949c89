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
// Measured: 160 experts of 1536 x 5120, 49152 rows, 940 us (5.0 GB of gradients: 5.4 TB/s; a fill of
// that buffer takes 655); 128 of 768 x 2048, 131072 rows, added to earlier gradients, 434 us. Without
// its stores the first took 676 us: loads, MMAs and the epilogue's passage through shared memory
// overlap, and each still slows the others. The sums leaving through TMA instead of the warps'
// stores: 1046 us.
#include <algorithm>
#include <climits>
#include <cuda_fp8.h>

#include "tc_common.cuh"

namespace smoe {
namespace {

// Six stages are two times three planes (five: 903 fp32 rows of 24 experts of 1416 x 1000 53 us, against
// 46; bf16 1 to 2 % slower). They leave 768 bytes for aligning the block's shared memory, which starts
// on a multiple of 256 at least.
constexpr int kDwStages = 6, kDwSlack = 768, kDwWarps = 8, kDwThreads = 128 + 32 * kDwWarps;
constexpr int kDwCols = 1024 / kDwWarps;  // columns of an epilogue warp
// The tensor core cuts its sums off at 24 bits instead of rounding them, addition by addition, so
// long sums drift (1024 rows: 1.2e-6 of the result). So the rows after the first chunk of an
// expert go into the other TMEM accumulator, chunk by chunk, which the epilogue adds, rounded, to
// the first one. For fp32 operands, whose six products add up six times as often, after fewer rows.
// A choice of time against accuracy (131072 rows of 128 experts, accumulated, us and relative error in the
// norm, a plain fp32 sum 2.7e-7: chunks of 256 rows 554 and 2.2e-7, 512: 479 and 4.3e-7, 768: 447 and
// 6.7e-7, 1024: 432 and 8.5e-7, one: 402; 8192 rows of one expert, plain 9.5e-7: 27.9 and 2.4e-7, 25.7 and
// 4.7e-7, 25.1 and 6.7e-7, 24.5 and 9.9e-7; terms of one sign lose up to 5e-6 with 1024): what enters
// the sums has 2^-9 of its own. (With the sums in registers, 128 of them a thread, 530 us.)
template <int PL> constexpr int kDwChunk = PL == 1 ? 1024 : 128;
constexpr int kDwHalf = 128 * 128;  // bytes of an operand's stage in a CTA: 64 rows of 128 channels
constexpr size_t kDwSmem = kDwSlack + kDwStages * 2 * kDwHalf + kDwWarps * 4096 +
                           8 * (3 * kDwStages + 2 * 2 + 1) + 16 + 4 * (kMaxGroups + 2);

struct DwArgs {
  const int32_t* expert_off;
  const float* add;   // nullable
  float* dw;
  DeviceStatus* st;
  int E, TK, M, N;    // M = n_out, N = n_in
  int mt, nt;         // tiles of each
  int slices;         // of an expert's rows: each slice's sums in a matrix of their own
};

struct DwTile {
  int e, m0, n0, row0, rows, slice;
};

__device__ __forceinline__ DwTile dw_decode(const DwArgs& p, const int32_t* off, int t) {
  DwTile r;
  r.slice = t % p.slices;
  t /= p.slices;
  const int per = p.mt * p.nt;
  r.e = t / per;
  const int in = t - r.e * per, m = in / p.nt;
  r.m0 = m * 256;
  r.n0 = (in - m * p.nt) * 256;
  r.row0 = off[r.e];
  r.rows = off[r.e + 1] - r.row0;
  if (p.slices > 1) {
    const int step = ((r.rows + p.slices - 1) / p.slices + 63) & ~63, from = min(r.rows, r.slice * step);
    r.row0 += from;
    r.rows = min(r.rows - from, step);
  }
  return r;
}

// The rows [left, the next multiple of 16) of a stage become zeros, by a warp, which orders them
// before the async proxy afterwards.
__device__ __forceinline__ void dw_clear(uint8_t* a, uint8_t* b, int left, int lane) {
  for (int i = left * 8 + lane; i < ((left + 15) & ~15) * 8; i += 32)  // 16 bytes each
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      *reinterpret_cast<uint4*>(a + j * 8192 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
      *reinterpret_cast<uint4*>(b + j * 8192 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
}

// PL = 3: fp32 operands as three bf16 planes each, [3][TK][channels], whose sum they are: the six
// products of planes that reach 2^-24 of a term are added up, which is a product in fp32. A
// plane of both operands takes a stage; the MMAs of 64 rows wait for three stages.
template <int PL>
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

  if (base - smem_raw > kDwSlack) {  // (never seen; both CTAs alike)
    if (threadIdx.x == 0) record_error(p.st, kStatusTimeout, kTimeoutGemm, -1);
    return;
  }
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
  const int total = *s_bad ? 0 : p.E * p.mt * p.nt * p.slices;
  volatile int* abort = s_abort;
  // A tile's columns: 256, or 128 where the matrix has no more; half of them staged by each CTA.

  // 384 threads of 168 registers at launch, 104 + 2 x 200 = 3 x 168 from here on
  if (warp < 4) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
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
      for (int i = 0; i < PL * ((tl.rows + 63) >> 6); ++i) {
        const int r = i / PL * 64, row = i % PL * p.TK + tl.row0 + r;
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
            tc::tma_load_2d_pair(sA + s * kDwHalf + j * 8192, &tmA, on, m0 + 64 * j, row);
          for (int j = 0; j < nb; ++j)
            tc::tma_load_2d_pair(sB + s * kDwHalf + j * 8192, &tmB, on, n0 + 64 * j, row);
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
    uint32_t s = 0, ph = 0, d = 0, eph = 0x3;  // eph: a phase bit for each accumulator
    bool ok = true, in = false;
    for (int t = first; t < total && ok; t += stride) {
      const DwTile tl = dw_decode(p, s_off, t);
      if (tl.rows == 0) continue;
      const uint32_t idesc = tc::instr_desc(false, 256, tl.n0 + 128 < p.N ? 256 : 128) |
                             tc::kIdescTransA | tc::kIdescTransB;
      for (int r = 0; r < tl.rows; r += 64) {
        const int left = min(64, tl.rows - r), steps = (left + 15) >> 4;
        const uint32_t at = r < kDwChunk<PL> ? d : d ^ 1u, acc = tmem + at * 256;
        const bool start = r % kDwChunk<PL> == 0, end = (r + 64) % kDwChunk<PL> == 0 || r + 64 >= tl.rows;
        if (start) {
          ok = tc::mbar_wait_warp(&dempty[at], eph >> at & 1u, abort);
          if (!ok) break;
          eph ^= 1u << at;
        }
        uint64_t ad[PL], bd[PL];
        uint64_t* e_bar[PL];
#pragma unroll
        for (int i = 0; i < PL; ++i) {
          if (left & 15) {
            // the peer's zeros are acquired with its word
            ok = tc::mbar_wait_warp_shared(&full[s], ph, abort);
            if (!ok) break;
            dw_clear(sA + s * kDwHalf, sB + s * kDwHalf, left, lane);
            if (i == PL - 1) {
              tc::fence_async_shared();
              __syncwarp();
            }
          } else if (i > 0 || !in) {
            ok = tc::mbar_wait_warp(&full[s], ph, abort);
            if (!ok) break;
          }
          ad[i] = tc::sw128_mnmajor_desc(tc::smem_u32(sA + s * kDwHalf));
          bd[i] = tc::sw128_mnmajor_desc(tc::smem_u32(sB + s * kDwHalf));
          e_bar[i] = &empty[s];
          if (++s == kDwStages) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
        tc::fence_after_sync();
        const bool in_next = tc::mbar_test(&full[s], ph);
        if (lead) {
          // the smallest products first: (2, 0), (1, 1), (0, 2), (1, 0), (0, 1), (0, 0)
#pragma unroll
          for (int sum = PL - 1; sum >= 0; --sum)
#pragma unroll
            for (int i = sum; i >= 0; --i)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (k < steps)
                  tc::mma_bf16_pair(acc, ad[i] + 128 * k, bd[sum - i] + 128 * k, idesc,
                                    !start || k > 0 || i != PL - 1);
#pragma unroll
          for (int i = 0; i < PL; ++i) tc::commit_pair(e_bar[i], 0x3);
          if (end) tc::commit_pair(&dfull[at], 0x3);
        }
        in = __all_sync(0xffffffffu, in_next);
      }
      d ^= 1u;
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
      it += PL * ((tl.rows + 63) >> 6);
      if ((tl.rows & 15) == 0) continue;
      for (int i = PL; i > 0; --i) {
        const uint32_t s = (it - i) % kDwStages;
        ok = tc::mbar_wait_warp(&last[s], lph >> s & 1u, abort);
        if (!ok) break;
        lph ^= 1u << s;
        dw_clear(sA + s * kDwHalf, sB + s * kDwHalf, tl.rows & 63, lane);
      }
      if (!ok) break;
      tc::fence_async_shared();
      __syncwarp();
      if (lane == 0)
        for (int i = PL; i > 0; --i)
          tc::mbar_arrive_cluster_shared(tc::cluster_addr(&full[(it - i) % kDwStages], 0));
    }
    if (!ok && lane == 0) {
      *abort = 1;
      record_error(p.st, kStatusTimeout, kTimeoutGemm, blockIdx.x);
    }
    __syncwarp();
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ---------------------------------------------------------------- epilogue
    // Each warp 32 rows of kDwCols columns, in windows of 32 columns through 4 KB of its own
    // (16-byte chunks swizzled by row: no bank conflicts), added to and stored as whole lines. What
    // is added is loaded a window ahead.
    const int q = warp & 3, part = (warp - 4) >> 2;
    constexpr int kWins = kDwCols / 32;
    uint8_t* buf = sE + (warp - 4) * 4096;
    const int ch = lane & 7, sub = lane >> 3;
    uint32_t d = 0, fph = 0;  // fph: a phase bit for each accumulator
    bool ok = true;
    auto wait = [&](uint32_t at) {
      ok = tc::mbar_wait_warp(&dfull[at], fph >> at & 1u, abort);
      fph ^= 1u << at;
      tc::fence_after_sync();
    };
    auto read_out = [&](uint32_t at) {
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_remote(tc::cluster_addr(&dempty[at], 0));
    };
    for (int t = first; t < total && ok; t += stride) {
      const DwTile tl = dw_decode(p, s_off, t);
      const int m0 = tl.m0 + (int)rank * 128 + q * 32, n0 = tl.n0 + part * kDwCols;
      const int mrows = min(32, p.M - m0), ncols = min(kDwCols, p.N - n0);  // may be below 1
      const size_t at = (((size_t)tl.slice * p.E + tl.e) * p.M + m0 + sub) * p.N + n0 + ch * 4;
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
      const uint32_t sums = tmem + ((uint32_t)(q * 32) << 16) + d * 256 + part * kDwCols;
      const uint32_t more = tmem + ((uint32_t)(q * 32) << 16) + (d ^ 1u) * 256 + part * kDwCols;
      if (tl.rows > 0) wait(d);
      for (int r = kDwChunk<PL>; r < tl.rows && ok; r += kDwChunk<PL>) {  // chunks behind the first
        wait(d ^ 1u);
        if (!ok) break;
#pragma unroll 1
        for (int c = 0; c < kDwCols; c += 32) {
          uint32_t v[32], u[32];
          tc::tmem_ld32(sums + c, u);
          tc::tmem_ld32(more + c, v);
          tc::tmem_ld_wait(u);
          tc::tmem_ld_wait(v);
#pragma unroll
          for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) + __uint_as_float(v[i]));
          tc::tmem_st32(sums + c, u);
        }
        tc::tmem_st_wait();
        read_out(d ^ 1u);
      }
      if (!ok) break;
#pragma unroll
      for (int w = 0; w < kWins; ++w) {
        if (w >= nwin) break;
        __syncwarp();  // TMEM loads are a whole warp's
        uint32_t v[32];
        if (tl.rows > 0) {
          tc::tmem_ld32(sums + 32 * w, v);
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
        read_out(d);
        d ^= 1u;
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

// ------------------------------------------------------------------ slices
// A contraction whose output tiles do not fill the GPU is cut into slices, whose sums are added here
// in their order: the result does not depend on timing.
__global__ void __launch_bounds__(256)
sum_slices_kernel(const float4* parts, int slices, long long rows, int row_vecs, bool segments,
                  const int32_t* expert_off, int E, int TK, const float4* add, float4* out) {
  pdl_wait_and_trigger();
  bool bad = false;
  for (int g = threadIdx.x; g <= E; g += 256) {
    const int lo = expert_off[g], hi = g < E ? expert_off[g + 1] : lo;
    bad |= lo < 0 || hi < lo || hi > TK;
  }
  if (__syncthreads_or(bad)) return;  // the products recorded it
  const long long first = segments ? expert_off[0] : 0, last = segments ? expert_off[E] : rows;
  for (long long i = first * row_vecs + (long long)blockIdx.x * 256 + threadIdx.x; i < last * row_vecs;
       i += (long long)gridDim.x * 256) {
    float4 s = add ? add[i] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float4 t = __ldcs(parts + i);
    for (int k = 1; k < slices; ++k) {
      const float4 v = __ldcs(parts + k * rows * row_vecs + i);
      t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
    }
    out[i] = make_float4(s.x + t.x, s.y + t.y, s.z + t.z, s.w + t.w);
  }
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

}  // namespace

cudaError_t launch_sum_slices(const float* parts, int slices, long long rows, int row_len, bool segments,
                              const int32_t* expert_off, int E, int TK, const float* add, float* out,
                              cudaStream_t s) {
  const int grid = std::min(ceil_div(rows * (row_len / 4), 256), 152 * 8);
  SMOE_LAUNCH(sum_slices_kernel, grid, 256, 0, s, reinterpret_cast<const float4*>(parts), slices, rows, row_len / 4,
              segments, expert_off, E, TK, reinterpret_cast<const float4*>(add), reinterpret_cast<float4*>(out));
  return cudaGetLastError();
}

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
  const size_t planes = d.dtype == SMOE_F32 ? (size_t)d.T * d.K * std::max(d.d, d.F) * 6 : 0;
  L->planes_a = take(planes);
  L->planes_b = take(planes);
  const size_t weights = has_weight_planes(d) ? (size_t)d.E * d.d * d.F * 6 : 0;
  L->planes_w = take(weights);
  L->planes_w2 = take(weights);
  L->parts = take(kPartBytes);
  L->total = off;
}

cudaError_t launch_expert_rows(const smoe_desc& d, int n_out, int n_in, const void* a, const void* w,
                               const void* a2, const void* w2, bool transposed,
                               const int32_t* expert_off, void* out, void* ws, cudaStream_t s) {
  if (d.dtype != SMOE_F32)
    return launch_expert_rows_bf16(d, n_out, n_in, a, w, a2, w2, transposed, expert_off, out, ws, s);
  return launch_expert_rows_f32(d, n_out, n_in, static_cast<const float*>(a), static_cast<const float*>(w),
                                static_cast<const float*>(a2), static_cast<const float*>(w2), transposed,
                                expert_off, static_cast<float*>(out), ws, s);
}

namespace {

template <int PL>
cudaError_t run_dw(const void* dy, const void* x, DwArgs p, float* parts, cudaStream_t s) {
  const long long size = (long long)p.E * p.M * p.N;
  p.slices = slices_of((long long)p.E * p.mt * p.nt, device_sms() / 2, p.TK / p.E / (PL == 1 ? 512 : 128), size);
  float* const dw = p.dw;
  const float* const add = p.add;
  if (p.slices > 1) {
    p.dw = parts;
    p.add = nullptr;
  }
  alignas(64) CUtensorMap A, B;
  if (!encode_tmap_2d(&A, dy, false, (uint64_t)PL * p.TK, p.M, 64, 64) ||
      !encode_tmap_2d(&B, x, false, (uint64_t)PL * p.TK, p.N, 64, 64))
    return cudaErrorInvalidValue;
  auto kern = dw_kernel<PL>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kDwSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(2 * (int)std::min<long long>(device_sms() / 2, (long long)p.E * p.mt * p.nt * p.slices));
  cfg.blockDim = dim3(kDwThreads);
  cfg.dynamicSmemBytes = kDwSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  SMOE_COUNT_LAUNCH(1);
  const cudaError_t launched = cudaLaunchKernelEx(&cfg, kern, A, B, p);
  if (launched != cudaSuccess || p.slices == 1) return launched;
  return launch_sum_slices(parts, p.slices, (long long)p.E * p.M, p.N, false, p.expert_off, p.E, p.TK, add, dw, s);
}

// The planes of both operands' rows of the segments, 8 values a thread.
__global__ void __launch_bounds__(256)
split_rows_kernel(const float* a, const float* b, int na, int nb, uint4* pa, uint4* pb,
                  const int32_t* expert_off, int E, int TK) {
  pdl_wait_and_trigger();
  const int va = na >> 3, vb = nb >> 3;
  const long long it = (long long)blockIdx.x * 256 + threadIdx.x;
  const int r = (int)(it / (va + vb)), v = (int)(it - (long long)r * (va + vb));
  if (r < max(expert_off[0], 0) || r >= min(expert_off[E], TK)) return;
  const bool first = v < va;
  const int n = first ? va : vb, c = first ? v : v - va;
  const float4* from = reinterpret_cast<const float4*>(first ? a : b) + ((size_t)r * n + c) * 2;
  const float4 x0 = __ldcg(from), x1 = __ldcg(from + 1);
  float x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
  uint4* to = (first ? pa : pb) + (size_t)r * n + c;
#pragma unroll
  for (int pl = 0; pl < 3; ++pl) {
    float y[8];
    split_planes(x, y);
    to[(size_t)pl * TK * n] = pack16(y, (const __nv_bfloat16*)nullptr);
  }
}

// From this many rows an expert and multiply-adds on an fp32 weight gradient runs on the tensor
// cores. Measured (us, planes and CUDA cores; rows an expert): 24 experts of 1416 x 1000, 8: 43 and
// 38, 16: 44 and 51, 128: 89 and 255; 8 of 512 x 512, 32: 14 and 10, 64: 15 and 18, 128: 20 and 32; 4
// of 256 x 256, 128: 17 and 15.
constexpr int kPlaneRows = 16;
constexpr double kPlaneMacs = 1e8;

}  // namespace

cudaError_t launch_expert_dw(const smoe_desc& d, int n_out, int n_in, const void* dy, const void* x,
                             const int32_t* expert_off, const float* add, float* dw, void* ws,
                             cudaStream_t s) {
  const int TK = d.T * d.K, wide = std::max(d.d, d.F);
  DeviceStatus* st = static_cast<DeviceStatus*>(ws);
  const DwArgs p{expert_off, add, dw, st, d.E, TK, n_out, n_in, ceil_div(n_out, 256), ceil_div(n_in, 256), 1};
  ProductLayout L;
  product_ws_layout(d, &L);
  float* parts = ws_ptr<float>(ws, L.parts);
  if (d.dtype != SMOE_F32) return run_dw<1>(dy, x, p, parts, s);
  const float *fy = static_cast<const float*>(dy), *fx = static_cast<const float*>(x);
  // (the planes' place is the descriptor's)
  if (n_out > wide || n_in > wide || (double)TK * n_out * n_in < kPlaneMacs ||
      (long long)TK < (long long)kPlaneRows * d.E || 3LL * TK > INT_MAX / 2 ||
      (long long)TK * (n_out / 8 + n_in / 8) > INT_MAX)
    return launch_expert_dw_f32(d, n_out, n_in, fy, fx, expert_off, add, dw, ws, s);
  uint4 *pa = ws_ptr<uint4>(ws, L.planes_a), *pb = ws_ptr<uint4>(ws, L.planes_b);
  SMOE_LAUNCH(split_rows_kernel, ceil_div((long long)TK * (n_out / 8 + n_in / 8), 256), 256, 0, s, fy, fx, n_out, n_in, pa, pb,
              expert_off, d.E, TK);
  return run_dw<3>(pa, pb, p, parts, s);
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
