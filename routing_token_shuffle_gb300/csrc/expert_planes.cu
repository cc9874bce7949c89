// fp32 products of many rows on the tensor cores: each operand as three bf16 planes whose sum it
// is, and the six products of planes that reach 2^-24 of a term added up,
//   kind 0  y[r, n] = sum_k x[r, k] w[e, n, k]
//   kind 1  dx[r, k] = sum_n dy[r, n] w[e, n, k]  (+ a second pair)
// (the weight gradients' form is in expert_grad.cu, which this follows: persistent pairs of CTAs,
// 256 x 256 tiles, 128 rows and half of the columns staged by each CTA, a plane of both operands a
// stage, three stages for 64 of the contraction). The weights lie along the contraction in kind 0
// (K-major boxes of 64 x 128) and across it in kind 1 (MN-major, two boxes of 64 x 64). Tensor maps
// end with each matrix, so what lies past a contraction's end reads as zeros. The tensor core cuts
// its sums off: after 128 of the contraction the next ones begin in the other TMEM accumulator,
// which the epilogue adds, rounded, to the first.
// Measured: 8192 rows of 8 experts, 2048 to 1024 channels, 232 us with the planes' making (148 TFLOP/s
// of the product's own; the CUDA cores' tiles 994); smaller ones at kPlaneRows in expert_f32.cu.
#include <algorithm>

#include "tc_common.cuh"

namespace smoe {
namespace {

constexpr int kPlStages = 5, kPlWarps = 8, kPlThreads = 128 + 32 * kPlWarps;
constexpr int kPlHalf = 128 * 128;   // bytes of an operand's stage in a CTA
constexpr int kPlChunk = 2;          // stages of 64 to an accumulator
constexpr size_t kPlSmem = 1024 + kPlStages * 2 * kPlHalf + kPlWarps * 4096 +
                           8 * (2 * kPlStages + 2 * 2 + 1) + 16 + 4 * 2 * (kMaxGroups + 2);

struct PlArgs {
  const int32_t* expert_off;
  float* out;
  DeviceStatus* st;
  int E, TK, N, K;
  int pairs;           // kind 1: operand pairs (1 or 2)
  int slices;          // of the contraction: each slice's sums in a matrix of their own
  long long size;      // floats of such a matrix
};

struct PlTile {
  int e, m0, n0, row0, rows, kb0, nk, slice;  // kb0, nk: of 64, over both pairs
};

__device__ __forceinline__ PlTile pl_decode(const PlArgs& p, const int32_t* ts, const int32_t* off,
                                            int nt, int t, int& g) {
  PlTile r;
  r.slice = t % p.slices;
  t /= p.slices;
  while (ts[g + 1] * nt <= t) ++g;
  const int mt = ts[g + 1] - ts[g], local = t - ts[g] * nt, n = local / mt;
  r.e = g;
  r.m0 = (local - n * mt) * 256;
  r.n0 = n * 256;
  r.row0 = off[g];
  r.rows = off[g + 1] - off[g];
  const int all = p.pairs * ((p.K + 63) >> 6), step = (all + p.slices - 1) / p.slices;
  r.kb0 = min(all, r.slice * step);
  r.nk = min(all - r.kb0, step);
  return r;
}

template <int KIND>
__global__ void __launch_bounds__(kPlThreads, 1)
planes_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
              const __grid_constant__ CUtensorMap tmA2, const __grid_constant__ CUtensorMap tmB2,
              const PlArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sA = base;
  uint8_t* sB = sA + kPlStages * kPlHalf;
  uint8_t* sE = sB + kPlStages * kPlHalf;
  uint64_t* full = reinterpret_cast<uint64_t*>(sE + kPlWarps * 4096);
  uint64_t* empty = full + kPlStages;
  uint64_t* dfull = empty + kPlStages;
  uint64_t* dempty = dfull + 2;
  uint64_t* drain = dempty + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(drain + 1);
  int* s_abort = reinterpret_cast<int*>(s_tmem + 1);
  int32_t* s_ts = reinterpret_cast<int32_t*>(s_abort + 1);
  int32_t* s_off = s_ts + kMaxGroups + 2;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = tc::cluster_rank();
  const int first = blockIdx.x >> 1, stride = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kPlStages; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      tc::mbar_init(&dfull[a], 1);
      tc::mbar_init(&dempty[a], 2 * kPlWarps);
    }
    tc::mbar_init(drain, 1);
    *s_abort = 0;
    tc::mbar_init_fence();
    tc::tma_prefetch_map(&tmA);
    tc::tma_prefetch_map(&tmB);
    tc::tma_prefetch_map(&tmA2);
    tc::tma_prefetch_map(&tmB2);
  }
  pdl_wait_and_trigger();
  __syncwarp();
  tc::cluster_arrive();
  if (warp == 3) {  // row tiles of each expert; a bad expert_off schedules nothing
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
      const int n = !bad && g < p.E ? (s_off[g + 1] - s_off[g] + 255) / 256 : 0;
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
  const int nt = (p.N + 255) / 256;
  const int total = s_ts[p.E] * nt * p.slices;
  const int nk1 = (p.K + 63) >> 6;
  volatile int* abort = s_abort;
  // A tile's columns: 256, or 128 where the matrix has no more; half of them staged by each CTA.

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA
    const bool lead = tc::elect_one();
    uint32_t s = 0, ph = 1, it = 0;
    bool ok = true;
    int g = 0;
    for (int t = first; t < total && ok; t += stride) {
      const PlTile tl = pl_decode(p, s_ts, s_off, nt, t, g);
      const int nb = tl.n0 + 128 < p.N ? 2 : 1, n0 = tl.n0 + (int)rank * 64 * nb;
      const int row = tl.row0 + tl.m0 + (int)rank * 128;
      for (int i = 0; i < 3 * tl.nk; ++i) {
        const int kb = tl.kb0 + i / 3, pl = i % 3;
        ok = tc::mbar_wait_warp(&empty[s], ph, abort);
        if (!ok) break;
        if (lead) {
          const bool second = kb >= nk1;
          const int k0 = (second ? kb - nk1 : kb) * 64, mat = pl * p.E + tl.e;
          const CUtensorMap* a = second ? &tmA2 : &tmA;
          const CUtensorMap* b = second ? &tmB2 : &tmB;
          const uint32_t on = tc::cluster_addr(&full[s], 0);
          if (rank == 0) tc::mbar_expect_tx(&full[s], 2 * (kPlHalf + (KIND == 0 ? 2 : nb) * 8192));
          tc::tma_load_3d_pair(sA + s * kPlHalf, a, on, k0, row, pl);
          if (KIND == 0) {
            tc::tma_load_3d_pair(sB + s * kPlHalf, b, on, k0, n0, mat);
          } else {
            for (int j = 0; j < nb; ++j)
              tc::tma_load_3d_pair(sB + s * kPlHalf + j * 8192, b, on, n0 + 64 * j, k0, mat);
          }
        }
        __syncwarp();
        ++it;
        if (++s == kPlStages) { s = 0; ph ^= 1u; }
      }
    }
    if (lead) {
      if (!ok) {
        *abort = 1;
        record_error(p.st, kStatusTimeout, kTimeoutGemm, blockIdx.x);
      }
      // The copies in flight land before shared memory goes away, whichever role gave up: the
      // leader waits for both CTAs' (a barrier that the peer did not get to never completes: then
      // the limit is waited out once), the peer cannot see its own complete.
      volatile int never = 0;
      if (rank == 0) {
        for (uint32_t j = it > kPlStages ? it - kPlStages : 0; j < it; ++j)
          if (!tc::mbar_wait(&full[j % kPlStages], (j / kPlStages) & 1u, &never)) break;
      } else if (*abort) {
        tc::wait_out();
      }
    }
    __syncwarp();
  } else if (warp == 1 && rank == 0) {
    // ---------------------------------------------------------------- MMA issuer (of the pair)
    // (24 MMAs a wait: by lane 0 8192 rows of 8 experts took 232 us, under elect.sync 240)
    const bool lead = lane == 0;
    constexpr uint32_t kStepB = KIND == 0 ? 2 : 128;
    uint32_t s = 0, ph = 0, d = 0, eph = 0x3;  // eph: a phase bit for each accumulator
    bool ok = true, in = false;
    int g = 0;
    for (int t = first; t < total && ok; t += stride) {
      const PlTile tl = pl_decode(p, s_ts, s_off, nt, t, g);
      if (tl.nk == 0) continue;
      const uint32_t idesc = tc::instr_desc(false, 256, tl.n0 + 128 < p.N ? 256 : 128) |
                             (KIND == 0 ? 0u : tc::kIdescTransB);
      for (int kb = 0; kb < tl.nk; ++kb) {
        const uint32_t at = kb < kPlChunk ? d : d ^ 1u, acc = tmem + at * 256;
        const bool start = kb % kPlChunk == 0, end = (kb + 1) % kPlChunk == 0 || kb + 1 == tl.nk;
        if (start) {
          ok = tc::mbar_wait_warp(&dempty[at], eph >> at & 1u, abort);
          if (!ok) break;
          eph ^= 1u << at;
        }
        uint64_t ad[3], bd[3];
        uint64_t* e_bar[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          if (i > 0 || !in) ok = tc::mbar_wait_warp(&full[s], ph, abort);
          if (!ok) break;
          ad[i] = tc::sw128_kmajor_desc(tc::smem_u32(sA + s * kPlHalf));
          bd[i] = KIND == 0 ? tc::sw128_kmajor_desc(tc::smem_u32(sB + s * kPlHalf))
                            : tc::sw128_mnmajor_desc(tc::smem_u32(sB + s * kPlHalf));
          e_bar[i] = &empty[s];
          if (++s == kPlStages) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
        tc::fence_after_sync();
        const bool in_next = tc::mbar_test(&full[s], ph);
        if (lead) {
          // the smallest products first: (2, 0), (1, 1), (0, 2), (1, 0), (0, 1), (0, 0)
#pragma unroll
          for (int sum = 2; sum >= 0; --sum)
#pragma unroll
            for (int i = sum; i >= 0; --i)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                tc::mma_bf16_pair(acc, ad[i] + 2 * k, bd[sum - i] + kStepB * k, idesc, !start || k > 0 || i != 2);
#pragma unroll
          for (int i = 0; i < 3; ++i) tc::commit_pair(e_bar[i], 0x3);
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
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- epilogue
    // Each warp 32 rows of 128 columns, in windows of 32 columns through 4 KB of its own
    // (16-byte chunks swizzled by row: no bank conflicts), stored as whole lines.
    const int q = warp & 3, half = (warp - 4) >> 2;
    uint8_t* buf = sE + (warp - 4) * 4096;
    const int ch = lane & 7, sub = lane >> 3;
    uint32_t d = 0, fph = 0;  // fph: a phase bit for each accumulator
    bool ok = true;
    int g = 0;
    auto wait = [&](uint32_t at) {
      ok = tc::mbar_wait_warp(&dfull[at], fph >> at & 1u, abort);
      fph ^= 1u << at;
      tc::fence_after_sync();
    };
    auto read_out = [&](uint32_t at) {
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_remote(tc::cluster_addr(&dempty[at], 0));
      __syncwarp();
    };
    for (int t = first; t < total && ok; t += stride) {
      const PlTile tl = pl_decode(p, s_ts, s_off, nt, t, g);
      const int m0 = tl.m0 + (int)rank * 128 + q * 32, n0 = tl.n0 + half * 128;
      const int mrows = min(32, tl.rows - m0), ncols = min(128, p.N - n0);  // may be below 1
      const int nwin = mrows > 0 && ncols > 0 ? (ncols + 31) >> 5 : 0;
      float* out = p.out + tl.slice * p.size + (size_t)(tl.row0 + m0 + sub) * p.N + n0 + ch * 4;
      const uint32_t sums = tmem + ((uint32_t)(q * 32) << 16) + d * 256 + half * 128;
      const uint32_t more = tmem + ((uint32_t)(q * 32) << 16) + (d ^ 1u) * 256 + half * 128;
      if (tl.nk > 0) wait(d);
      for (int kb = kPlChunk; kb < tl.nk && ok; kb += kPlChunk) {  // chunks behind the first
        wait(d ^ 1u);
        if (!ok) break;
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
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
#pragma unroll 1
      for (int w = 0; w < nwin; ++w) {
        __syncwarp();  // TMEM loads are a whole warp's
        uint32_t v[32];
        if (tl.nk > 0) {
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
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rr = i * 4 + sub;
          const float4 o = *reinterpret_cast<const float4*>(buf + rr * 128 + ((ch ^ (rr & 7)) << 4));
          if (rr < mrows && w * 32 + ch * 4 < ncols)
            *reinterpret_cast<float4*>(out + (size_t)(i * 4) * p.N + w * 32) = o;
        }
      }
      if (tl.nk > 0) {
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

// One matrix' planes, 8 values a thread (the rule of split_planes).
__global__ void __launch_bounds__(256)
split_kernel(const float4* x, long long vecs, uint4* planes) {
  pdl_wait_and_trigger();
  for (long long v = (long long)blockIdx.x * 256 + threadIdx.x; v < vecs; v += (long long)gridDim.x * 256) {
    const float4 a = __ldcg(x + 2 * v), b = __ldcg(x + 2 * v + 1);
    float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int pl = 0; pl < 3; ++pl) {
      float y[8];
      split_planes(f, y);
      planes[pl * vecs + v] = pack16(y, (const __nv_bfloat16*)nullptr);
    }
  }
}

cudaError_t split(const float* x, long long n, void* planes, cudaStream_t s) {
  const int grid = std::min(ceil_div(n / 8, 256), 152 * 16);
  SMOE_LAUNCH(split_kernel, grid, 256, 0, s, reinterpret_cast<const float4*>(x), n / 8, static_cast<uint4*>(planes));
  return cudaGetLastError();
}

template <int KIND>
cudaError_t run_planes(const smoe_desc& d, int n_out, int n_in, const float* a, const float* w, const float* a2,
                       const float* w2, const int32_t* expert_off, float* out, void* ws, cudaStream_t s) {
  ProductLayout L;
  product_ws_layout(d, &L);
  const int TK = d.T * d.K, N = KIND == 0 ? n_out : n_in, K = KIND == 0 ? n_in : n_out;
  void *pa = ws_ptr<char>(ws, L.planes_a), *pb = ws_ptr<char>(ws, L.planes_b);
  void *pw = ws_ptr<char>(ws, L.planes_w), *pw2 = ws_ptr<char>(ws, L.planes_w2);
  const long long weights = (long long)d.E * n_out * n_in;
  cudaError_t e = split(a, (long long)TK * K, pa, s);
  if (e == cudaSuccess) e = split(w, weights, pw, s);
  if (e == cudaSuccess && a2) e = split(a2, (long long)TK * K, pb, s);
  if (e == cudaSuccess && a2) e = split(w2, weights, pw2, s);
  if (e != cudaSuccess) return e;
  if (!a2) {
    pb = pa;
    pw2 = pw;
  }
  alignas(64) CUtensorMap A, B, A2, B2;
  const uint32_t box = KIND == 0 ? 128 : 64;
  if (!encode_tmap_3d(&A, pa, false, 3, TK, K, 128, 64) || !encode_tmap_3d(&A2, pb, false, 3, TK, K, 128, 64) ||
      !encode_tmap_3d(&B, pw, false, 3ull * d.E, n_out, n_in, box, 64) ||
      !encode_tmap_3d(&B2, pw2, false, 3ull * d.E, n_out, n_in, box, 64))
    return cudaErrorInvalidValue;
  PlArgs p{expert_off, out, ws_ptr<DeviceStatus>(ws, L.status), d.E, TK, N, K, a2 ? 2 : 1, 1, (long long)TK * N};
  const long long tiles = (long long)std::max(ceil_div(TK, 256), std::min(TK, d.E)) * ceil_div(N, 256);
  const long long most = ((long long)ceil_div(TK, 256) + std::min(TK, d.E)) * ceil_div(N, 256);
  p.slices = slices_of(tiles, device_sms() / 2, (long long)p.pairs * ceil_div(K, 64) / 4, p.size);
  float* parts = ws_ptr<float>(ws, L.parts);
  if (p.slices > 1) p.out = parts;
  auto kern = planes_kernel<KIND>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPlSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(2 * (int)std::min<long long>(device_sms() / 2, most * p.slices));
  cfg.blockDim = dim3(kPlThreads);
  cfg.dynamicSmemBytes = kPlSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  SMOE_COUNT_LAUNCH(1);
  e = cudaLaunchKernelEx(&cfg, kern, A, B, A2, B2, p);
  if (e != cudaSuccess || p.slices == 1) return e;
  return launch_sum_slices(parts, p.slices, TK, N, true, expert_off, d.E, TK, nullptr, out, s);
}

}  // namespace

cudaError_t launch_expert_rows_planes(const smoe_desc& d, int n_out, int n_in, const float* a, const float* w,
                                      const float* a2, const float* w2, bool transposed,
                                      const int32_t* expert_off, float* out, void* ws, cudaStream_t s) {
  return transposed ? run_planes<1>(d, n_out, n_in, a, w, a2, w2, expert_off, out, ws, s)
                    : run_planes<0>(d, n_out, n_in, a, w, a2, w2, expert_off, out, ws, s);
}

}  // namespace smoe
