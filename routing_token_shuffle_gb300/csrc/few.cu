// The whole MoE layer for a few tokens (T <= 64) in one kernel: gate, softmax and grouped
// top-K, the touched experts' SwiGLU FFN (shared experts included) and the weighted sum.
//
// At these batches the layer is the stream of the touched experts' weights from HBM
// (3 F d b bytes each), so the kernel is built around that stream: one persistent CTA per
// SM, launched cooperatively, whose producer warp keeps a ring of TMA loads in flight
// across the phases, and two grid-wide barriers where a phase needs every SM's results:
//   gate      logits = x W_g^T, spread over the SMs          -- barrier 1 --
//   routes    every CTA selects the T tokens' experts from the T x E logits (see kSelectAll)
//   up        H[slot][t] = w_{t,e} silu(W1 x_t) (W3 x_t), 0 where t is not routed to the
//             slot's expert e (slots: the shared experts, then the touched routed ones)
//   down      y_t = sum over slots of W2_e H[slot][t]        -- barrier 2 before it --
// With the routing weight folded into H and zeros for the other tokens, the down product
// over all slots is one contraction of length slots x F, whose accumulator is the layer's
// output: no per-expert outputs, no combine.
// The shared experts' up tiles do not wait for the routes: they stream while the gate and
// the selection run. The W2 tiles at the head of a CTA's down range do not wait for barrier
// 2: they are loaded into the free stages before it.
//
// (Zeros for the tokens of other experts also mean that a weight of W2 that is not finite
// reaches every token of the call.)
//
// Work is split evenly: the 128-row x 128-byte weight blocks of a phase, taken in order,
// are cut into one contiguous range per CTA, whatever the tile borders. A tile whose blocks
// lie in several ranges is finished by the CTA that holds its first block: the others
// write fp32 partial sums and a flag, and the owner adds them in ascending order (the
// result does not depend on timing). A CTA's first segment never waits, so the owner's wait
// (for its successors' first segments) cannot be circular.
//
// An A tile is 128 weight rows (up: 64 rows of W1 and the same 64 of W3), the B tile is all
// T tokens padded to NP rows; fp32 accumulation. Every wait is bounded (see tc_common.cuh).
//
// Measured: bf16, 64 tokens of a 160-expert layer of 5120 x 1536 with two shared experts 1.06
// ms (6.2 TB/s of the touched weights, 0.93 of the measured copy rate), 3 tokens of 8 experts
// of 4096 x 14336 242 us (6 TB/s), one token of 128 experts of 2048 x 768 29 us (75 MB: 11 us
// of stream, 7 us until the routes are known, two barriers and the joining of sums). fp32, 13
// tokens of 24 experts of 1000 x 1416 90 us: 51 us of HBM, 11 until the routes are known, and
// the shared expert's blocks, where FMAs and shared memory take twice the stream's time. The
// same layer with 32 tokens 209 us and with 64 tokens 410 us, against 61 and 64 us of HBM: above
// 16 tokens the routed tokens are not packed (see kPack) and groups of four of them are
// multiplied by every weight of their experts.
#include <algorithm>
#include <cfloat>
#include <climits>

#include "few_ring.cuh"
#include "tc_common.cuh"

namespace smoe {
namespace {

constexpr int kFewThreads = 384;
constexpr uint32_t kFewA = kFewStageA;

struct FewArgs {
  const void* x;
  const void* w_gate;
  void* y;
  float* logits;        // [T, E] in the workspace
  float* logits_out;    // nullable outputs
  int32_t* topk_idx;
  float* topk_w;
  void* h;              // [slots, T, F] fp32, or [slots, 2, T, F] bf16
  float* partial;       // [2][kFewMaxCtas][NP * 128]
  uint32_t* flags;      // [3][kFewMaxCtas]
  int32_t* ridx;        // [T, K] routes in the workspace (T > kSelectAll)
  float* rw;
  uint32_t* ctl;        // barrier 1, barrier 2, selected tokens, exits
  DeviceStatus* st;
  int T, d, E, K, H, F, S, renorm, stages;
};

// The 128-byte weight blocks of a phase, kper to a tile, cut into one range per CTA.
// bf16: the stream from HBM is the time of a block whatever its tokens. Equal ranges, in
// blocks; in whole tiles where the last round of tiles has one for at least 6 of 10 CTAs: an
// SM can stream twice its share of HBM's rate, so that many keep it busy, and no sums have to
// be joined (one token of a 128-expert layer, 96 up tiles: 33 -> 30 us).
// fp32: ranges of equal weight; a block takes longer the more tokens its expert has, and
// equal ranges left the slowest CTA at 1.4 times the mean. Up to 16 tokens kPackBlock + (the
// expert's tokens): 4, 8 and 16 gave 93, 91 and 100 us with 13 tokens, 104, 98 and 105 with 16.
// Above, 2 + (groups of four tokens): 900 clocks with one group and 1700 with four.
constexpr int kPackBlock = 8;
struct Range {
  int kper, unit, quot, rem;
  const int* table;  // fp32: first block of each CTA, in shared memory
  __device__ __forceinline__ Range(int kper_, int tiles, int n) : kper(kper_), table(nullptr) {
    const int last = tiles % n;
    unit = last * 10 >= n * 6 ? kper_ : 1;
    const int units = unit == 1 ? tiles * kper_ : tiles;
    quot = units / n;
    rem = units - quot * n;
  }
  __device__ __forceinline__ Range(int kper_, const int* table_)
      : kper(kper_), unit(1), quot(0), rem(0), table(table_) {}
  __device__ __forceinline__ int first(int cta) const {
    return table ? table[cta] : (cta * quot + min(cta, rem)) * unit;
  }
  __device__ __forceinline__ bool any(int cta) const {
    return table ? table[cta] < table[cta + 1] : quot > 0 || cta < rem;
  }
};

// First block of CTA `cta` of nc when the blocks of `tiles` tiles, each of nshared slots of
// weight wshared and nact slots of the weights in pre (a prefix), per_slot blocks a slot,
// are cut by weight.
__device__ __forceinline__ int weighted_first(int cta, int nc, int tiles, int per_slot, int nshared,
                                              int wshared, const int* pre, int nact) {
  const long long tile_w = (long long)(nshared * wshared + pre[nact]) * per_slot;
  const long long at = tile_w * tiles * cta / nc;
  const int tile = (int)(at / tile_w);
  const int base = tile * (nshared + nact) * per_slot;
  if (tile == tiles) return base;
  long long left = at - tile_w * tile;
  const long long shared_w = (long long)nshared * wshared * per_slot;
  if (left < shared_w) return base + (int)(left / wshared);
  left -= shared_w;
  int lo = 0, hi = nact - 1;
  while (lo < hi) {  // largest slot whose weight prefix is at most what is left
    const int mid = (lo + hi + 1) >> 1;
    if ((long long)pre[mid] * per_slot <= left) lo = mid; else hi = mid - 1;
  }
  const int in = (int)((left - (long long)pre[lo] * per_slot) / (pre[lo + 1] - pre[lo]));
  return base + (nshared + lo) * per_slot + in;
}

__device__ __forceinline__ bool group_and(int id, int threads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void group_sync(int id, int threads) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_release(uint32_t* p, uint32_t v) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ void add_release(uint32_t* p) {
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p) : "memory");
}
// bounded wait for *p >= want (signed: a counter that starts below zero is that much short)
__device__ __forceinline__ bool wait_ge(const uint32_t* p, int want, volatile int* abort) {
  if ((int)ld_acquire(p) >= want) return true;
  const unsigned long long t0 = tc::globaltimer();
  for (uint32_t i = 1;; ++i) {
    if ((int)ld_acquire(p) >= want) return true;
    if ((i & 63u) == 0 && (*abort || tc::globaltimer() - t0 > tc::kWaitTimeoutNs)) return false;
  }
}

// 16 bytes of x and W_g: their contribution to a logit
__device__ __forceinline__ float dot16(const uint4& a, const uint4& b, float s, const float* tag) {
  float u[4], v[4];
  unpack16(a, u, tag);
  unpack16(b, v, tag);
#pragma unroll
  for (int i = 0; i < 4; ++i) s = fmaf(u[i], v[i], s);
  return s;
}
__device__ __forceinline__ float dot16(const uint4& a, const uint4& b, float s,
                                       const __nv_bfloat16* tag) {
  float u[8], v[8];
  unpack16(a, u, tag);
  unpack16(b, v, tag);
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(u[i], v[i], s);
  return s;
}

// Logits of this CTA's units, 4 experts x 8 tokens each, by warps 2-11, which split the
// contraction; red: [10][32] floats. The 32 sums of a warp's lanes are added by halving:
// after 31 shuffles lane l holds sum l.
template <typename TE>
__device__ __forceinline__ void gate_logits(const FewArgs& p, float* red, int gt) {
  constexpr int V = Elem<TE>::kPerVec16;
  const int lane = gt & 31;
  const int nv = p.d / V, groups = (p.T + 7) / 8;
  const uint4* x = static_cast<const uint4*>(p.x);
  const uint4* w = static_cast<const uint4*>(p.w_gate);
  const int units = (p.E + 3) / 4 * groups;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int e0 = u / groups * 4, t0 = (u % groups) * 8, nt = min(8, p.T - t0);
    float acc[32] = {};  // [token][expert]
#pragma unroll 1
    for (int v = gt; v < nv; v += kGateThreads) {
      uint4 wv[4], xv[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) wv[j] = __ldg(w + (size_t)min(e0 + j, p.E - 1) * nv + v);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < nt) xv[i] = __ldcg(x + (size_t)(t0 + i) * nv + v);  // y may be the same buffer
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < nt) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[4 * i + j] = dot16(xv[i], wv[j], acc[4 * i + j], (const TE*)nullptr);
        }
    }
#pragma unroll
    for (int half = 16; half; half >>= 1) {
      const bool up = lane & half;
#pragma unroll
      for (int i = 0; i < half; ++i) {
        const float give = up ? acc[i] : acc[i + half];
        acc[i] = (up ? acc[i + half] : acc[i]) + __shfl_xor_sync(0xffffffffu, give, half);
      }
    }
    group_sync(2, kGateThreads);  // red is free
    red[gt] = acc[0];
    group_sync(2, kGateThreads);
    if (gt < 32 && (lane >> 2) < nt && e0 + (lane & 3) < p.E) {
      float sum = 0.0f;
#pragma unroll
      for (int k = 0; k < kGateThreads / 32; ++k) sum += red[k * 32 + lane];
      p.logits[(size_t)(t0 + (lane >> 2)) * p.E + e0 + (lane & 3)] = sum;
    }
  }
}

// order-preserving image of a logit (-0 and +0 alike); 0 is kept for "taken"
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  const uint32_t k = (u >> 31) ? ~u : (u | 0x80000000u);
  return k ? k : 1u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float((k >> 31) ? (k ^ 0x80000000u) : ~k);
}

// One warp selects token t's experts: group h's K/H largest logits, descending, the lower
// index first on ties; weights are the softmax over all E logits at the picks. Lane j < K
// returns pick j and its weight; lane l holds the logits of experts l, l + 32, ...
// (kPer of them: the fewer, the shorter each pick and the code to fetch, which runs once or
// a few times per launch).
template <int kPer>
__device__ __forceinline__ void select_token(const FewArgs& p, int t, int lane, int* idx, float* w) {
  uint32_t key[kPer], best = 0;
  float v[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    v[i] = lane + 32 * i < p.E ? __ldcg(p.logits + (size_t)t * p.E + lane + 32 * i) : 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    key[i] = lane + 32 * i < p.E ? key_of(v[i]) : 0u;
    best = max(best, key[i]);
  }
  const float mx = value_of(__reduce_max_sync(0xffffffffu, best));
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (key[i]) sum += expf(v[i] - mx);
#pragma unroll
  for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  const int per = p.E / p.H, kh = p.K / p.H;
  int my_idx = 0;
  uint32_t my_key = 0;
#pragma unroll 1
  for (int h = 0, j = 0; h < p.H; ++h) {
    const int lo = h * per - lane, hi = lo + per;  // expert lane + 32 i is in [lo, hi) + lane
#pragma unroll 1
    for (int q = 0; q < kh; ++q, ++j) {
      uint32_t m = 0;
      int at = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (32 * i >= lo && 32 * i < hi && key[i] > m) { m = key[i]; at = 32 * i; }
      const uint32_t top = __reduce_max_sync(0xffffffffu, m);
      const int pick = (int)__reduce_min_sync(0xffffffffu, m == top ? (uint32_t)(lane + at) : ~0u);
      if (lane == j) { my_idx = pick; my_key = top; }
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (lane + 32 * i == pick) key[i] = 0u;
    }
  }
  float my_w = lane < p.K ? expf(value_of(my_key) - mx) / sum : 0.0f;
  if (p.renorm) {
    float s = my_w;
#pragma unroll
    for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    my_w /= s;
  }
  *idx = my_idx;
  *w = my_w;
}

// Up to this many tokens every CTA selects all of them, one per warp: shared memory holds
// the routes without another pass through L2. Above it CTA t selects token t alone and the
// CTAs exchange the routes, one more grid-wide wait: 64 tokens of 160 experts took 22 us
// in rounds of ten tokens per CTA.
constexpr int kSelectAll = kGateThreads / 32;

// NP, ND: rows of the B tile of the up and of the down product. fp32: ND = NP, one row of H a
// token. bf16: two rows a token, H's bf16 rounding and the bf16 rounding of what it left, so
// that the down product sees 16 bits of H: T tokens' rows, then T rows of rests, whose
// accumulator columns the epilogue adds to the first ones. Rounding H to bf16 alone made the
// layer's error 1.4 to 1.6 times that of rounding its output; the second row is free up to 32
// tokens (the stream from HBM is the time) and takes 64 tokens from 1.03 to 1.06 ms.
template <typename TE, int NP, int ND>
__global__ void __launch_bounds__(kFewThreads, 1)
moe_few_kernel(const __grid_constant__ CUtensorMap tmX,   // [T, d], NP-row box
               const __grid_constant__ CUtensorMap tmW1,  // [(E+S) F, d], 64-row box
               const __grid_constant__ CUtensorMap tmW3,
               const __grid_constant__ CUtensorMap tmW2,  // [(E+S) d, F], 128-row box
               const __grid_constant__ CUtensorMap tmH,   // [slots T (bf16: 2 T), F], ND-row box
               const FewArgs p) {
  constexpr int BK = 128 / (int)sizeof(TE);
  constexpr uint32_t kB = ND * 128;                // B stage (the up product's tile may be smaller)
  constexpr bool kTC = sizeof(TE) == 2;            // bf16: tcgen05; fp32: FMAs on the CUDA cores
  // TMEM: two accumulators of ND columns (reads of 16 columns may start at column T)
  constexpr uint32_t kCols = ND == 16 ? 64 : 2 * ND;
  // Consumer threads: 4 warps read the accumulators (bf16), 8 warps multiply (fp32): two
  // groups of four, which take every other block. A warp takes all 128 rows of its block, four
  // to a lane, 16 tokens and a share of the contraction: shared memory returns 128 bytes a
  // clock, broadcast or not, so a token's values have to serve four rows (one row a lane and
  // all tokens: 512 clocks of shared memory for every four tokens of a block, against 712 that
  // its load from HBM takes; now 128).
  constexpr int kCons = kTC ? 128 : 256;
  constexpr int kTokSplit = NP / 16, kKSplit = 8 / kTokSplit;
  // fp32, up to 16 tokens: only the routed tokens of a block are multiplied. In the up product,
  // whose tile is one expert's, they take the first accumulators, so that the unrolled code
  // runs straight on and ends at the last of them: stepping over the other tokens' code, at
  // every block, cost more than the FMAs (106 -> 91 us with 13 tokens of 3 from 24 experts).
  // Rows of H that no routed token owns are then neither written nor read.
  constexpr bool kPack = !kTC && NP == 16;
  constexpr int kXch = few_xch(!kTC);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int S = p.stages;
  uint8_t* sA = base;
  uint8_t* sB = base + (size_t)S * kFewA;
  float* s_xch = reinterpret_cast<float*>(sB + (size_t)S * kB);  // [128][kXch], four of them for fp32
  uint64_t* full = reinterpret_cast<uint64_t*>(s_xch + (kTC ? 1 : 4) * 128 * kXch);
  uint64_t* empty = full + kFewMaxStages;
  uint64_t* tfull = empty + kFewMaxStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint64_t* routed = drain + 1;
  unsigned long long* s_mask = reinterpret_cast<unsigned long long*>(routed + 1);
  int* s_abort = reinterpret_cast<int*>(s_mask + p.E);
  int* s_nact = s_abort + 1;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(s_nact + 1);
  float* s_red = reinterpret_cast<float*>(s_tmem + 2);     // [10][32]
  float* s_wcol = s_red + kGateThreads;                    // [64]
  int* s_use = reinterpret_cast<int*>(s_wcol + 64);        // [64]
  int* s_tok = s_use + 64;                                 // [64] token of each column (kPack)
  int32_t* s_act = s_tok + 64;                             // [E]
  int32_t* s_idx = s_act + p.E;                            // [T K]
  float* s_w = reinterpret_cast<float*>(s_idx + p.T * p.K);
  int32_t* s_first = reinterpret_cast<int32_t*>(s_w + p.T * p.K);  // fp32: [2][kFewMaxCtas + 1]
  int32_t* s_pre = s_first + 2 * (kFewMaxCtas + 1);                // fp32: [E + 1]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x, nc = gridDim.x;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], kTC ? 1 : kCons / 64);
    }
    for (int a = 0; a < 2; ++a) {
      tc::mbar_init(&tfull[a], 1);
      tc::mbar_init(&tempty[a], 128);
    }
    tc::mbar_init(drain, 1);
    tc::mbar_init(routed, 1);
    *s_abort = 0;
    *s_nact = 0;
    tc::mbar_init_fence();
    tc::tma_prefetch_map(&tmX);
    tc::tma_prefetch_map(&tmW1);
    tc::tma_prefetch_map(&tmW3);
    tc::tma_prefetch_map(&tmW2);
    tc::tma_prefetch_map(&tmH);
  }
  for (int i = threadIdx.x; i < p.E; i += kFewThreads) s_mask[i] = 0;
  if (kTC && warp == 2) {
    tc::tmem_alloc(s_tmem, kCols);
    tc::tmem_relinquish();
  }
  if (kTC) tc::fence_before_sync();
  __syncthreads();
  if (kTC) tc::fence_after_sync();
  const uint32_t tmem = kTC ? *s_tmem : 0u;
  volatile int* abort = s_abort;
  const int FB = (p.F + 63) / 64, nkd = (p.d + BK - 1) / BK, nkf = (p.F + BK - 1) / BK;
  // parts: 0 up of the shared experts (fp32: none, all of them are in part 1, where the
  // tiles cut at its borders would cost more than the early start gains), 1 up of the routed
  // ones, 2 down. Slots: the shared experts, then the touched ones.
  const int slot1 = kTC ? p.S : 0;  // first slot of part 1
  auto expert_of = [&](int slot) { return slot < p.S ? p.E + slot : s_act[slot - p.S]; };
  auto part_range = [&](int part) {
    if (part == 0) return Range(nkd, kTC ? p.S * FB : 0, nc);
    const int down = (p.d + 127) / 128;
    if (!kTC && part == 1) return Range(nkd, s_first);
    if (!kTC) return Range((p.S + *s_nact) * nkf, s_first + kFewMaxCtas + 1);
    if (part == 1) return Range(nkd, *s_nact * FB, nc);
    const int kper = (p.S + *s_nact) * nkf;
    return Range(kper, down, nc);
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    const bool lead = tc::elect_one();
    uint32_t it = 0;
    bool ok = true;
    // The place of the next block, stepped without divisions: this thread's instructions
    // between two stages are the stream's rate (decoding every block from its index with
    // divisions held the stream at 5.3 TB/s).
    struct Place {
      int tile, kb, fb, slot, row;  // fb, slot: down only; row: of the A tile
    };
    auto row_of = [&](int part, int tile, int slot) {
      if (part == 2) return expert_of(slot) * p.d + tile * 128;
      const int li = tile / FB;
      return expert_of((part == 0 ? 0 : slot1) + li) * p.F + (tile - li * FB) * 64;
    };
    auto place = [&](int part, const Range& r, int i) {
      Place at;
      at.tile = i / r.kper;
      at.kb = i - at.tile * r.kper;
      at.slot = part == 2 ? at.kb / nkf : 0;
      at.fb = at.kb - at.slot * nkf;
      at.row = row_of(part, at.tile, at.slot);
      return at;
    };
    auto step = [&](int part, const Range& r, Place& at) {
      ++at.fb;
      if (++at.kb == r.kper) {
        ++at.tile;
        at.kb = at.slot = at.fb = 0;
      } else if (part == 2 && at.fb == nkf) {
        ++at.slot;
        at.fb = 0;
      } else {
        return;
      }
      at.row = row_of(part, at.tile, at.slot);
    };
    auto load_a = [&](uint32_t s, int part, const Place& at) {
      if (!lead) return;
      tc::mbar_expect_tx(&full[s], kFewA + (part < 2 ? NP : ND) * 128);
      if (part < 2) {
        tc::tma_load_2d(sA + s * kFewA, &tmW1, &full[s], at.kb * BK, at.row);
        tc::tma_load_2d(sA + s * kFewA + kFewA / 2, &tmW3, &full[s], at.kb * BK, at.row);
      } else {
        tc::tma_load_2d(sA + s * kFewA, &tmW2, &full[s], at.fb * BK, at.row);
      }
    };
    auto load_b = [&](uint32_t s, int part, const Place& at) {
      if (!lead) return;
      if (part < 2) tc::tma_load_2d(sB + s * kB, &tmX, &full[s], at.kb * BK, 0);
      else tc::tma_load_2d(sB + s * kB, &tmH, &full[s], at.fb * BK, at.slot * p.T * (kTC ? 2 : 1));
    };
    uint32_t s = 0, ph = 1;  // stage and the parity its release is awaited with
    auto next_stage = [&] {
      ++it;
      if (++s == (uint32_t)S) { s = 0; ph ^= 1u; }
    };
    for (int part = 0; part < 3 && ok; ++part) {
      if (part == 1 && !tc::mbar_wait_warp(routed, 0, abort)) { ok = false; break; }
      const Range r = part_range(part);
      int i = r.first(cta);
      const int end = r.first(cta + 1);
      if (i == end) continue;
      Place at = place(part, r, i);
      if (part == 2) {
        // weights ahead of barrier 2: the A halves of the first stages
        const uint32_t s0 = s, it0 = it;
        Place ahead = at;
        for (int j = min(end - i, S); j > 0; --j) {
          if (!tc::mbar_wait_warp(&empty[s], ph, abort)) { ok = false; break; }
          load_a(s, part, ahead);
          step(part, r, ahead);
          next_stage();
        }
        if (ok) ok = __all_sync(0xffffffffu, !lead || wait_ge(p.ctl + 1, nc, abort));
        // H was written by other SMs through the generic proxy
        asm volatile("fence.proxy.async.global;" ::: "memory");
        // (also after a wait that gave up: the stages' byte counts must complete)
        uint32_t sb = s0;
        for (uint32_t q = it0; q < it; ++q) {
          load_b(sb, part, at);
          step(part, r, at);
          if (++sb == (uint32_t)S) sb = 0;
        }
        i += (int)(it - it0);
        if (!ok) break;
      }
      for (; i < end; ++i) {
        if (!tc::mbar_wait_warp(&empty[s], ph, abort)) { ok = false; break; }
        load_a(s, part, at);
        load_b(s, part, at);
        step(part, r, at);
        next_stage();
      }
    }
    if (lead) {
      if (!ok) {
        *abort = 1;
        record_error(p.st, kStatusTimeout, kTimeoutFew, cta);
      }
      // the copies in flight land before the CTA's shared memory goes away, also where it was
      // another role that gave up
      volatile int never = 0;
      const uint32_t firstj = it > (uint32_t)S ? it - S : 0;
      for (uint32_t j = firstj; j < it; ++j) tc::mbar_wait(&full[j % S], (j / S) & 1u, &never);
    }
  } else if (kTC && warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    const bool lead = tc::elect_one();
    uint32_t s = 0, ph = 0, tcount = 0;
    bool ok = true, in = false;
    for (int part = 0; part < 3 && ok; ++part) {
      if (part == 1 && !tc::mbar_wait_warp(routed, 0, abort)) { ok = false; break; }
      const Range r = part_range(part);
      const int end = r.first(cta + 1);
      const uint32_t idesc = tc::instr_desc(false, 128, part < 2 ? NP : ND);
      for (int i = r.first(cta); i < end && ok; ++tcount) {
        const int n = min(r.kper - i % r.kper, end - i);
        const uint32_t a = tcount & 1u, aph = (tcount >> 1) & 1u;
        if (!tc::mbar_wait_warp(&tempty[a], aph ^ 1u, abort)) { ok = false; break; }
        tc::fence_after_sync();
        for (int j = 0; j < n; ++j) {
          if (!in && !tc::mbar_wait_warp(&full[s], ph, abort)) { ok = false; break; }
          tc::fence_after_sync();
          const uint64_t adesc = tc::sw128_kmajor_desc(tc::smem_u32(sA + s * kFewA));
          const uint64_t bdesc = tc::sw128_kmajor_desc(tc::smem_u32(sB + s * kB));
          uint64_t* used = &empty[s];
          if (++s == (uint32_t)S) { s = 0; ph ^= 1u; }
          // asking for the next stage takes ~100 clocks: while this one's MMAs are issued
          // (one token of the 128-expert layer 29.8 -> 29.0 us, 64 tokens level)
          const bool next = tc::mbar_test(&full[s], ph);
          if (lead) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc::mma_bf16(tmem + a * ND, adesc + 2 * k, bdesc + 2 * k, idesc, (j > 0 || k > 0) ? 1u : 0u);
            tc::commit(used);
          }
          in = __all_sync(0xffffffffu, next);
        }
        i += n;
        if (ok && lead) tc::commit(&tfull[a]);
        __syncwarp();
      }
    }
    if (lead) {
      if (!ok) {
        *abort = 1;
        record_error(p.st, kStatusTimeout, kTimeoutFew, cta);
      }
      // wait for every MMA this thread issued before TMEM is released
      volatile int never = 0;
      tc::commit(drain);
      tc::mbar_wait(drain, 0, &never);
    }
    __syncwarp();
  } else if (warp >= 2) {
    // ---------------------------------------------------------------- gate and routes
    const int gt = threadIdx.x - 64;
    gate_logits<TE>(p, s_red, gt);
    group_sync(2, kGateThreads);
    bool ok = true;
    if (gt == 0) {
      for (int q = 0; q < 3; ++q) p.flags[q * kFewMaxCtas + cta] = 0;
      add_release(p.ctl);  // after every write of this CTA that the barrier ordered before it
      ok = wait_ge(p.ctl, nc, abort);
    }
    ok = group_and(2, kGateThreads, ok);
    if (ok) {
      const int step = p.T <= kSelectAll ? p.T : nc;
      for (int t = p.T <= kSelectAll ? gt >> 5 : gt < 32 ? cta : p.T; t < p.T; t += step) {
        int idx;
        float w;
        if (p.E <= 128) select_token<4>(p, t, lane, &idx, &w);
        else if (p.E <= 256) select_token<8>(p, t, lane, &idx, &w);
        else select_token<16>(p, t, lane, &idx, &w);
        if (lane < p.K) {
          const int at = t * p.K + lane;
          if (p.T > kSelectAll) {
            p.ridx[at] = idx;
            p.rw[at] = w;
          } else {
            s_idx[at] = idx;
            s_w[at] = w;
            atomicOr(s_mask + idx, 1ull << t);
          }
          if (p.topk_idx && (cta == 0 || p.T > kSelectAll)) p.topk_idx[at] = idx;
          if (p.topk_w && (cta == 0 || p.T > kSelectAll)) p.topk_w[at] = w;
        }
        __syncwarp();
        if (p.T > kSelectAll && lane == 0) add_release(p.ctl + 2);
      }
      if (p.T > kSelectAll) {
        if (gt == 0) ok = wait_ge(p.ctl + 2, p.T, abort);
        ok = group_and(2, kGateThreads, ok);
        for (int i = gt; ok && i < p.T * p.K; i += kGateThreads) {
          s_idx[i] = __ldcg(p.ridx + i);
          s_w[i] = __ldcg(p.rw + i);
          atomicOr(s_mask + s_idx[i], 1ull << (i / p.K));
        }
      }
    }
    if (!ok && gt == 0) {
      *abort = 1;
      record_error(p.st, kStatusTimeout, kTimeoutFew, cta);
    }
    if (ok) {
      if (p.logits_out && cta == 0)
        for (int i = gt; i < p.T * p.E; i += kGateThreads) p.logits_out[i] = __ldcg(p.logits + i);
      group_sync(2, kGateThreads);
      if (gt < 32) {  // touched experts, ascending
        int n = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
          const bool on = e0 + lane < p.E && s_mask[e0 + lane] != 0;
          const uint32_t b = __ballot_sync(0xffffffffu, on);
          if (on) s_act[n + __popc(b & ((1u << lane) - 1u))] = e0 + lane;
          n += __popc(b);
        }
        if (lane == 0) *s_nact = n;
        if (!kTC) {  // the slots' weights (see Range), as a prefix
          __syncwarp();
          int carry = 0;
          for (int i0 = 0; i0 < n; i0 += 32) {
            int w = 0;
            if (i0 + lane < n) {
              const unsigned long long m = s_mask[s_act[i0 + lane]];
              int most = 0;
#pragma unroll 1
              for (int q16 = 0; q16 < kTokSplit; ++q16) {
                uint32_t g = (uint32_t)(m >> (16 * q16)) & 0xffffu;
                if (!kPack) {
                  g |= g >> 2;
                  g |= g >> 1;
                  g &= 0x1111u;
                }
                most = max(most, __popc(g));
              }
              w = kPack ? kPackBlock + most : 2 + kTokSplit * most;
            }
            int incl = w;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
              const int y = __shfl_up_sync(0xffffffffu, incl, off);
              if (lane >= off) incl += y;
            }
            if (i0 + lane < n) s_pre[i0 + lane] = carry + incl - w;
            carry += __shfl_sync(0xffffffffu, incl, 31);
          }
          if (lane == 0) s_pre[n] = carry;
        }
      }
      group_sync(2, kGateThreads);
      if (!kTC) {
        const int every = kPack ? kPackBlock + p.T : 2 + kTokSplit * ((min(p.T, 16) + 3) / 4);
        for (int i = gt; i < 2 * (nc + 1); i += kGateThreads) {
          if (i <= nc) s_first[i] = weighted_first(i, nc, 1, FB * nkd, p.S, every, s_pre, *s_nact);
          else s_first[kFewMaxCtas + i - nc] =
                   weighted_first(i - nc - 1, nc, (p.d + 127) / 128, nkf, p.S, every, s_pre, *s_nact);
        }
        group_sync(2, kGateThreads);
      }
      if (gt == 0) tc::mbar_arrive(routed);
    }
    if (ok && warp >= 4 && warp < 4 + kCons / 32) {
      // -------------------------------------------------------------- products, epilogue
      const int q = warp & 3, row = q * 32 + lane, half = (warp - 4) >> 2, ct = row + 128 * half;
      const int ks = (warp - 4) % kKSplit, tq = (warp - 4) / kKSplit;  // fp32: this warp's share
      (void)ks;
      (void)tq;
      uint32_t s = 0, ph = 0, tcount = 0;
      for (int part = 0; part < 3 && ok; ++part) {
        const Range r = part_range(part);
        const int end = r.first(cta + 1);
        float* partial = p.partial + (size_t)(part & 1) * kFewMaxCtas * NP * 128;
        uint32_t* flags = p.flags + part * kFewMaxCtas;
        for (int i = r.first(cta); i < end && ok;) {
          const int tile = i / r.kper, k0 = i - tile * r.kper;
          const int k1 = min(r.kper, k0 + end - i);
          float acc[kTC ? 1 : 4][kTC ? 1 : 16] = {};  // [rows lane + 32 r][columns 16 tq + t]
          const uint32_t ta = tcount & 1u, taph = (tcount >> 1) & 1u;
          ++tcount;
          if (kTC) {
            ok = tc::mbar_wait_warp(&tfull[ta], taph, abort);
          } else {
            // only the tokens of a block's expert (above 16 tokens only their groups of four): the
            // others are not kept (up) or zero (down)
            const unsigned long long every = ~0ull >> (64 - p.T);
            int slot = part == 2 ? k0 / nkf : slot1 + tile / FB;
            int left = part == 2 ? (slot + 1) * nkf - k0 : r.kper;
            unsigned long long on = slot < p.S ? every : s_mask[s_act[slot - p.S]];
            for (int kb = k0; kb < k1 && ok; ++kb) {
              if (left-- == 0) {
                ++slot;
                left = nkf - 1;
                on = slot < p.S ? every : s_mask[s_act[slot - p.S]];
              }
              if (few_group(kb - k0) != ks / (kKSplit / 2)) {  // the other group's block
                if (++s == (uint32_t)S) { s = 0; ph ^= 1u; }
                continue;
              }
              ok = tc::mbar_wait_warp(&full[s], ph, abort);
              if (!ok) break;
              const uint8_t* a = sA + s * kFewA + lane * 128;
              const uint8_t* b = sB + s * kB + tq * 16 * 128;
              const uint32_t on16 = (uint32_t)(on >> (16 * tq)) & 0xffffu;
#pragma unroll
              for (int c0 = 0; c0 < (kTC || on16 == 0 ? 0 : 16 / kKSplit); c0 += 2) {
                const int c = ks % (kKSplit / 2) * (16 / kKSplit) + c0;
                float4 av[2][4];
#pragma unroll
                for (int cc = 0; cc < 2; ++cc)
#pragma unroll
                  for (int r4 = 0; r4 < 4; ++r4)
                    av[cc][r4] = *reinterpret_cast<const float4*>(a + r4 * 4096 + (((c + cc) ^ (lane & 7)) << 4));
                auto token = [&](int j, int t) {  // accumulator j += A times row t of B
#pragma unroll
                  for (int cc = 0; cc < 2; ++cc) {
                    const float4 bv = *reinterpret_cast<const float4*>(b + t * 128 + (((c + cc) ^ (t & 7)) << 4));
#pragma unroll
                    for (int r4 = 0; r4 < 4; ++r4) {
                      float& s4 = acc[kTC ? 0 : r4][kTC ? 0 : j];
                      s4 = fmaf(av[cc][r4].x, bv.x, s4);
                      s4 = fmaf(av[cc][r4].y, bv.y, s4);
                      s4 = fmaf(av[cc][r4].z, bv.z, s4);
                      s4 = fmaf(av[cc][r4].w, bv.w, s4);
                    }
                  }
                };
                if (kPack && part < 2) {
                  uint32_t m = on16;
#pragma unroll
                  for (int j = 0; j < 16; j += 2) {
                    if (m == 0) break;
                    const int t0 = __ffs(m) - 1;
                    m &= m - 1;
                    const int t1 = m ? __ffs(m) - 1 : t0;
                    m &= m - 1;
                    token(j, t0);
                    token(j + 1, t1);
                  }
                } else {
#pragma unroll
                  for (int t = 0; t < 16; t += 4) {
                    if (((on16 >> t) & 15) == 0) continue;
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                      if (kPack && ((on16 >> (t + u)) & 1) == 0) continue;
                      token(t + u, t + u);
                    }
                  }
                }
              }
              __syncwarp();
              if (lane == 0) tc::mbar_arrive(&empty[s]);
              if (++s == (uint32_t)S) { s = 0; ph ^= 1u; }
            }
          }
          // whether other CTAs hold later blocks of a tile that starts here
          int c1 = cta + 1;
          if (k0 == 0 && k1 != r.kper) {
            while (r.first(c1) < (tile + 1) * r.kper) ++c1;  // cta + 1 .. c1 - 1 hold the rest
            for (int c = cta + 1 + ct; c < c1; c += kCons)
              if (r.any(c)) ok = ok && wait_ge(flags + c, 1, abort);
          }
          // one outcome for the consumer warps, which go on to barriers together
          ok = group_and(1, kCons, ok);
          if (!ok) break;
          i += k1 - k0;
          if (kTC) tc::fence_after_sync();
          const int li = tile / FB, fb = tile - li * FB, slot = (part == 0 ? 0 : slot1) + li;
          if (part < 2 && k0 == 0 && ct < 64) {  // the tokens of this expert and their weights
            float w = 1.0f;
            int use = row < p.T, at = row;
            if (slot >= p.S) {
              const int e = s_act[slot - p.S];
              const unsigned long long m = s_mask[e], before = (1ull << row) - 1;
              use = (int)((m >> row) & 1);
#pragma unroll 1
              for (int k = 0; k < p.K && use; ++k)
                if (s_idx[row * p.K + k] == e) w = s_w[row * p.K + k];
              if (kPack) at = use ? __popcll(m & before) : __popcll(m) + __popcll(~m & before);
            }
            s_wcol[at] = w;
            s_use[at] = use;
            if (kPack) s_tok[at] = row;
          }
          float* mine = s_xch + row * kXch;
          const int cols = kPack && part < 2 && slot >= p.S ? __popcll(s_mask[s_act[slot - p.S]]) : p.T;
#pragma unroll
          for (int c0 = 0; c0 < NP; c0 += 16) {
            if (c0 >= cols) break;
            const int nt = min(16, cols - c0);
            if (kTC) {
              const uint32_t col = tmem + ((uint32_t)(q * 32) << 16) + ta * ND + c0;
              float v[16];
              __syncwarp();  // a whole warp's loads: lanes that split in waits and stores join
              tc::tmem_ld16(col, v);
              if (part == 2) {  // and the rests' products
                float w[16];
                tc::tmem_ld16(col + p.T, w);
#pragma unroll
                for (int t = 0; t < 16; ++t) v[t] += w[t];
              }
#pragma unroll
              for (int t = 0; t < 16; ++t) mine[t] = v[t];
            } else {
              if (c0) group_sync(1, kCons);  // the last 16 tokens' sums have been used
              // the contraction's shares: into min(kKSplit, 4) buffers, four more added to
              // them, and the buffers' sum into the first. By 16 bytes: this code runs once a
              // tile, and fetching it costs as much as running it (4200 -> 1900 clocks)
              constexpr int kBuf = kKSplit < 4 ? kKSplit : 4;
              float* buf = s_xch + ((ks & 3) * 128 + lane) * kXch;
#pragma unroll 1
              for (int k = 0; k < kKSplit; k += 4) {
                if (tq == c0 / 16 && (ks & ~3) == k) {
#pragma unroll
                  for (int t = 0; t < (kTC ? 0 : 16); t += 4) {
                    if (kPack && t >= nt) break;
#pragma unroll
                    for (int r4 = 0; r4 < 4; ++r4) {
                      float4* x = reinterpret_cast<float4*>(buf + 32 * r4 * kXch + t);
                      float4 v = k == 0 ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : *x;
                      v.x += acc[kTC ? 0 : r4][kTC ? 0 : t];
                      v.y += acc[kTC ? 0 : r4][kTC ? 0 : t + 1];
                      v.z += acc[kTC ? 0 : r4][kTC ? 0 : t + 2];
                      v.w += acc[kTC ? 0 : r4][kTC ? 0 : t + 3];
                      *x = v;
                    }
                  }
                }
                group_sync(1, kCons);
              }
#pragma unroll
              for (int t = 8 * half; t < 8 * half + 8; t += 4) {
                if (kPack && t >= nt) break;
                float4 sum = *reinterpret_cast<const float4*>(mine + t);
#pragma unroll
                for (int k = 1; k < kBuf; ++k) {
                  const float4 v = *reinterpret_cast<const float4*>(mine + k * 128 * kXch + t);
                  sum.x += v.x;
                  sum.y += v.y;
                  sum.z += v.z;
                  sum.w += v.w;
                }
                *reinterpret_cast<float4*>(mine + t) = sum;
              }
              group_sync(1, kCons);
            }
            if (k0 != 0) {  // the tile belongs to an earlier CTA
              float* out = partial + ((size_t)cta * NP + c0) * 128 + row;
#pragma unroll 4
              for (int t = half; t < nt; t += kCons / 128) __stcg(out + t * 128, mine[t]);
              continue;
            }
            // add the following CTAs' sums in order, 16 loads in flight
            if (nt == 1) {
#pragma unroll 1
              for (int cb = cta + 1; cb < c1 && half == 0; cb += 16) {
                float in[16];
#pragma unroll
                for (int c = 0; c < 16; ++c)
                  in[c] = cb + c < c1 && r.any(cb + c)
                              ? __ldcg(partial + ((size_t)(cb + c) * NP + c0) * 128 + row) : 0.0f;
                float v = mine[0];
#pragma unroll
                for (int c = 0; c < 16; ++c) v += in[c];
                mine[0] = v;
              }
            } else {
              constexpr int kT = kTC ? 16 : 8, kC = kPack ? 4 : 2;  // tokens of a thread, CTAs at a time
              const int t0 = kT * half;
#pragma unroll 1
              for (int c = cta + 1; c < c1; c += kC) {
                const float* src = partial + ((size_t)c * NP + c0 + t0) * 128 + row;
                float in[kC][kT];
#pragma unroll
                for (int k = 0; k < kC; ++k) {
                  const bool on = c + k < c1 && r.any(c + k);
#pragma unroll
                  for (int t = 0; t < kT; ++t)
                    in[k][t] = on && t0 + t < nt ? __ldcg(src + ((size_t)k * NP + t) * 128) : 0.0f;
                }
                float v[kT];
#pragma unroll
                for (int t = 0; t < kT; ++t) v[t] = mine[t0 + t];
#pragma unroll
                for (int k = 0; k < kC; ++k)
#pragma unroll
                  for (int t = 0; t < kT; ++t) v[t] += in[k][t];
#pragma unroll
                for (int t = 0; t < kT; ++t) mine[t0 + t] = v[t];
              }
            }
            if (!kTC) group_sync(1, kCons);
            if (part < 2) {
              if (kTC) group_sync(1, kCons);
#pragma unroll 1
              for (int j = ct; j < 64 * nt; j += kCons) {
                const int fr = j & 63, t = j >> 6, f = fb * 64 + fr;
                const float g = s_xch[fr * kXch + t];
                const float hv = g / (1.0f + expf(-g)) * s_xch[(64 + fr) * kXch + t] * s_wcol[c0 + t];
                if (f < p.F) {
                  const float use = s_use[c0 + t] ? hv : 0.0f;
                  const TE hi = Elem<TE>::from_f32(use);
                  const int tok = kPack ? s_tok[t] : c0 + t;
                  TE* out = static_cast<TE*>(p.h) + ((size_t)slot * (kTC ? 2 : 1) * p.T + tok) * p.F + f;
                  *out = hi;
                  if (kTC) {
                    const float back = Elem<TE>::to_f32(hi);
                    out[(size_t)p.T * p.F] = Elem<TE>::from_f32(fabsf(back) <= FLT_MAX ? use - back : 0.0f);
                  }
                }
              }
              if (kTC) group_sync(1, kCons);
            } else {
              const int n = tile * 128 + row;
              if (n < p.d) {
#pragma unroll 1
                for (int t = half; t < nt; t += kCons / 128)
                  static_cast<TE*>(p.y)[(size_t)(c0 + t) * p.d + n] = Elem<TE>::from_f32(mine[t]);
              }
            }
          }
          if (kTC) {  // the accumulator is read out: the MMAs of another tile may start
            tc::fence_before_sync();
            tc::mbar_arrive(&tempty[ta]);
          }
          if (k0 != 0 || !kTC) group_sync(1, kCons);
          if (k0 != 0 && ct == 0) st_release(flags + cta, 1u);
        }
        if (part == 1 && ok) {  // this CTA's part of H is written: barrier 2
          group_sync(1, kCons);
          if (ct == 0) add_release(p.ctl + 1);
        }
      }
      if (!ok && lane == 0) {
        *abort = 1;
        record_error(p.st, kStatusTimeout, kTimeoutFew, cta);
      }
    }
  }
  __syncwarp();
  if (kTC) tc::fence_before_sync();
  __syncthreads();
  if (kTC) {
    tc::fence_after_sync();
    if (warp == 2) tc::tmem_dealloc(tmem, kCols);
  }
  if (threadIdx.x == 0) {
    // the last CTA leaves the counters at zero for the next call on this workspace
    __threadfence();
    if (atomicAdd(p.ctl + 3, 1u) == (uint32_t)nc - 1u) {
      p.ctl[0] = 0;
      p.ctl[1] = 0;
      p.ctl[2] = 0;
      p.ctl[3] = 0;
    }
  }
}

template <typename TE, int NP, int ND>
cudaError_t run_few(const smoe_desc& d, const void* x, const void* w_gate, const void* w1,
                    const void* w3, const void* w2, void* y, float* logits, int32_t* topk_idx,
                    float* topk_w, void* ws, cudaStream_t s) {
  constexpr bool kF32 = sizeof(TE) == 4;
  constexpr uint32_t BK = 128 / sizeof(TE);
  FewLayout L;
  few_ws_layout(d, &L);
  const uint64_t G = (uint64_t)d.E + d.n_shared;
  alignas(64) CUtensorMap tX, tW1, tW3, tW2, tH;
  void* h = ws_ptr<char>(ws, L.h);
  if (!encode_tmap_2d(&tX, x, kF32, d.T, d.d, NP, BK) ||
      !encode_tmap_2d(&tW1, w1, kF32, G * d.F, d.d, 64, BK) ||
      !encode_tmap_2d(&tW3, w3, kF32, G * d.F, d.d, 64, BK) ||
      !encode_tmap_2d(&tW2, w2, kF32, G * d.d, d.F, 128, BK) ||
      !encode_tmap_2d(&tH, h, kF32, L.slots * d.T * (kF32 ? 1 : 2), d.F, ND, BK))
    return cudaErrorInvalidValue;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  FewArgs p{x, w_gate, y, ws_ptr<float>(ws, L.logits), logits, topk_idx, topk_w, h,
            ws_ptr<float>(ws, L.partial), ws_ptr<uint32_t>(ws, L.flags),
            ws_ptr<int32_t>(ws, L.ridx), ws_ptr<float>(ws, L.rw),
            ws_ptr<uint32_t>(ws, kFewCtl), ws_ptr<DeviceStatus>(ws, L.status),
            d.T, d.d, d.E, d.K, d.H, d.F, d.n_shared, d.renorm, 0};
  p.stages = few_stages(kF32, d.E, (size_t)d.T * d.K, ND);
  auto kern = moe_few_kernel<TE, NP, ND>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // every CTA resident: they wait on one another
  attr[0].val.cooperative = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(std::min(sms, kFewMaxCtas));
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = kFewSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  SMOE_COUNT_LAUNCH(1);
  return cudaLaunchKernelEx(&cfg, kern, tX, tW1, tW3, tW2, tH, p);
}

template <typename TE>
cudaError_t run_few_t(const smoe_desc& d, const void* x, const void* w_gate, const void* w1,
                      const void* w3, const void* w2, void* y, float* logits, int32_t* topk_idx,
                      float* topk_w, void* ws, cudaStream_t s) {
  constexpr int W = sizeof(TE) == 2 ? 2 : 1;  // B rows of a token in the down product
  if (W == 2 && d.T <= 8)
    return run_few<TE, 16, 16>(d, x, w_gate, w1, w3, w2, y, logits, topk_idx, topk_w, ws, s);
  if (d.T <= 16)
    return run_few<TE, 16, 16 * W>(d, x, w_gate, w1, w3, w2, y, logits, topk_idx, topk_w, ws, s);
  if (d.T <= 32)
    return run_few<TE, 32, 32 * W>(d, x, w_gate, w1, w3, w2, y, logits, topk_idx, topk_w, ws, s);
  return run_few<TE, 64, 64 * W>(d, x, w_gate, w1, w3, w2, y, logits, topk_idx, topk_w, ws, s);
}

}  // namespace

void few_ws_layout(const smoe_desc& d, FewLayout* L) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) / 256 * 256;
    return o;
  };
  L->slots = std::min<size_t>(d.E, (size_t)d.T * d.K) + d.n_shared;
  const size_t np = d.T <= 16 ? 16 : d.T <= 32 ? 32 : 64;
  L->status = take(256);
  L->flags = take(4 * 3 * kFewMaxCtas);
  L->logits = take(4 * (size_t)d.T * d.E);
  L->ridx = take(4 * (size_t)d.T * d.K);
  L->rw = take(4 * (size_t)d.T * d.K);
  L->partial = take(4 * 2 * kFewMaxCtas * np * 128);
  L->h = take(L->slots * d.T * d.F * 4);  // fp32, or two bf16 a value
  L->total = off;
}

cudaError_t launch_moe_few(const smoe_desc& d, const void* x, const void* w_gate, const void* w1,
                           const void* w3, const void* w2, void* y, float* logits,
                           int32_t* topk_idx, float* topk_w, void* ws, cudaStream_t s) {
  if (d.dtype == SMOE_F32)
    return run_few_t<float>(d, x, w_gate, w1, w3, w2, y, logits, topk_idx, topk_w, ws, s);
  return run_few_t<__nv_bfloat16>(d, x, w_gate, w1, w3, w2, y, logits, topk_idx, topk_w, ws, s);
}

}  // namespace smoe
