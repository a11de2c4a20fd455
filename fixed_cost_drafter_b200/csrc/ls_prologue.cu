// The drafter's projections ahead of its attention: boundary keys/values from the boundary
// hidden vectors, block queries from the drafter's block inputs (LongSpark paper page,
// Figure 2 caption (c): the drafter uses the views; its projections are not described,
// the reading is a plain linear map per tapped layer). Both are dense contractions over
// the hidden size, so they run on the 5th-generation tensor cores:
//   Y[rows][n] = sum_k W[l][n][k] X[rows][l][k]   (bf16 in, fp32 accumulate, bf16 out)
// with the weights as the MMA's A operand (M = 128 weight rows per unit, K-major) and the
// activations as its B operand (N = up to 256 activation rows, K-major): the weights
// stream through once, the few activation rows come from L2.
//
// Persistent kernel, 7 warps: warp 0 TMA producer of the weights (a ring of 6 stages of 64
// hidden entries of the unit's 128 weight rows, from HBM), warp 6 TMA producer of the
// activations (3 stages of up to 256 rows, mostly from L2), both 128-byte swizzled; warp 1
// TMEM allocator and MMA issuer (double-buffered accumulator, 2 x 256 columns). Every wait,
// MMA issue and commit of the one MMA-issuing thread takes tens of nanoseconds, so a k-step
// costs it one wait and one commit: both producers' copies of k-step k complete on the
// weight ring's barrier of k (two arrivals), and the release of that barrier's stage also
// frees the activation stage of k (the activation ring, 3 deep, is refilled for k-step k
// once k - 3 is released, which the weight ring's barrier of k - 3 tells). Warps 2-5
// epilogue (one TMEM subpartition each: a thread owns one weight row, its outputs go
// through a shared-memory tile so that whole 256-byte output rows leave as 16-byte
// stores). Units: (problem, layer, 128-row weight tile, activation tile), queries first.
// The activation tiles of a weight tile follow one another: the CTAs that run together read it
// from HBM once (64 requests of 16 rows, 4 tiles: 158 -> 125 us).
// CTA c runs units c, c + grid, ... whole as long as every CTA has one; the k-steps of the
// units left over (boundary tiles, whose outputs are few) are spread evenly over all CTAs,
// so that every SM streams the same weight bytes, and run first. A piece of such a split
// tile leaves its fp32 partial sums in the state's scratch; the last piece of a tile to
// arrive adds them up in piece order (the same sum whatever the arrival order) and stores
// the tile.
// Launched as the programmatic dependent of the kernel before it on the stream: the weights
// (the drafter's parameters, nearly all of the bytes) stream from the start; the
// activations (the block inputs and the boundary view, which that kernel may write: a
// commit writes the boundary view) are read only after the grid dependency wait. Every
// thread triggers this grid's dependents once it has passed that wait.
// Every wait is bounded.
#include <type_traits>

#include "ls_tc.cuh"

namespace ls {

namespace {

constexpr int kPThreads = 224;                       // 7 warps
constexpr int kPKStep = kProKStep;                   // hidden entries per stage
constexpr int kPTileN = kProTileN;                   // weight rows per unit (MMA M)
constexpr int kPMaxAct = kProMaxAct;                 // activation rows per unit (MMA N)
constexpr int kPAStages = 6;                         // weight ring (read from HBM: deeper)
constexpr int kPBStages = 3;                         // activation ring (read from L2)
constexpr int kPABytes = kPTileN * kPKStep * 2;      // 16 KB
constexpr int kPBBytes = kPMaxAct * kPKStep * 2;     // 32 KB
constexpr int kPOutRows = 128;                       // activation rows per epilogue pass
constexpr int kPOutBytes = kPOutRows * kPTileN * 2;  // 32 KB: [128 rows][128 weight rows] bf16
constexpr int kPSmemBytes = kPAStages * kPABytes + kPBStages * kPBBytes + kPOutBytes + 1024;
constexpr uint32_t kPTmemCols = 512;

struct PProblem {
  int32_t n_out;         // weight rows (output columns) per layer, a multiple of 128
  int32_t rows_per_seq;  // activation rows per sequence and layer: 1 (boundary) or B (block)
  int32_t pitch;         // tile rows per sequence: rows_per_seq, with adapters rounded up to 16 (see PLora)
  int32_t seq_per_unit;  // sequences per activation tile
  int32_t load_rows;     // activation rows of a tile's box: seq_per_unit * pitch
  int32_t act_rows;      // the MMA's N: load_rows rounded up to 16 (the rows past load_rows
                         // are stale shared memory feeding accumulator columns never stored)
  int32_t m_tiles;       // activation tiles: ceil(b / seq_per_unit)
  int32_t n_units;       // L * (n_out / 128) * m_tiles
  int32_t is_4d;         // X tensor map is 4-D (block rows) or 3-D (boundary)
  __nv_bfloat16* y;      // [b][L][rows_per_seq][n_out]
};

struct PArgs {
  PProblem pr[2];
  int32_t b, L, k_steps;
  int32_t n_units;
  int32_t n_full;     // units [0, n_full) run whole, round robin over the CTAs
  int32_t rem_steps;  // k-steps of the split units [n_full, n_units) (all boundary tiles), 0 if none
  float* part;        // [slot][128][pr[1].act_rows] partial sums of the split tiles' pieces
  int32_t* count;     // [unit - n_full] arrivals of a split tile's pieces (zero between calls)
  int32_t* err;
};

// Low-rank adapters (ls_draft_prologue_lora): scale * (A x) of problem p, by lora_low_kernel.
// Block queries take them as further k-steps of their unit: weight rows B_a of the sequence's
// adapter against split[], low as two bf16 parts (high + low: 16 bits of the fp32 sum, as both operands
// of the product have one type; what is left out, 2^-17 of an inner sum, is of the size of the fp32
// sums' own rounding over 4096 entries, and outputs have 8 bits: 16 requests' queries at rank 16 are
// 1.6621e-3 off the 64-bit ones, as those of a plain form with fp32 inner sums are), into the
// sequence's accumulator columns only. For that a sequence's block starts at a multiple of 16
// columns, the MMA's step in N (the rows between are outside the tensor map's block dimension and
// read as zeros): no adapter's infinities reach another sequence. Boundary rows, whose sequences
// share 16 columns, are added by the epilogue in fp32; one row is cheap, and lora_low_kernel has
// multiplied them by B already.
struct PLora {
  ls_lora bank;
  __nv_bfloat16* split;  // [b][L][2][pitch][rank]
  float* add;            // [b][L][2 Hkv D]: scale * B (A boundary)
};

struct PBars {
  uint64_t afull[kPAStages], aempty[kPAStages];  // per k-step k: stage k mod kPAStages of
                                                 // both rings full (2 arrivals) / released
  uint64_t acc_full[2], acc_empty[2];
  uint64_t out_full, out_free;  // epilogue pass: staged by all 128 threads / copied out
  uint64_t drain;               // after an abort: the MMAs issued so far have completed
  uint64_t epi;                 // the 128 epilogue threads meet (split tiles' arrivals)
  uint32_t tmem_base;
  uint32_t abort;
  uint32_t last;                // the epilogue's piece was its tile's last to arrive
  int32_t issued[2];            // k-steps each producer arrived for (weights, activations)
};

struct PUnit {
  int p, l, nt, mt;
};

__device__ inline PUnit unit_of(const PArgs& a, int u) {
  PUnit r;
  r.p = u < a.pr[0].n_units ? 0 : 1;
  if (r.p) u -= a.pr[0].n_units;
  const int mts = a.pr[r.p].m_tiles, nts = a.pr[r.p].n_out / kPTileN;
  r.mt = u % mts;
  u /= mts;
  r.nt = u % nts;
  r.l = u / nts;
  return r;
}

// This CTA's work: pieces of the split units first (a contiguous range of their flattened
// k-steps, [g0, g1) = [c T / grid, (c + 1) T / grid)), then its whole units. With the
// pieces first, the sum of a split tile (by its last piece to arrive) runs in the epilogue
// warps while the CTA's whole units stream, instead of after them.
struct PWork {
  int n_pieces, n_items;
  int64_t g0, g1;
};

struct PItem {
  int u;       // unit
  int k0, k1;  // its k-steps [k0, k1)
  int slot;    // -1: the whole unit; else the piece's partial-sum slot
  int r;       // split unit index (u - n_full)
};

__device__ inline int64_t range_begin(int c, int64_t T, int grid) { return int64_t(c) * T / grid; }

// the CTA whose range holds split k-step g: the largest c with c T / grid <= g (rounded down)
__device__ inline int range_cta(int64_t g, int64_t T, int grid) { return int(((g + 1) * grid + T - 1) / T) - 1; }

__device__ inline PWork work_of(const PArgs& a) {
  PWork w;
  const int c = int(blockIdx.x), G = int(gridDim.x);
  const int n_whole = c < a.n_full ? (a.n_full - 1 - c) / G + 1 : 0;
  w.g0 = range_begin(c, a.rem_steps, G);
  w.g1 = range_begin(c + 1, a.rem_steps, G);
  w.n_pieces = w.g1 > w.g0 ? int((w.g1 - 1) / a.k_steps - w.g0 / a.k_steps + 1) : 0;
  w.n_items = w.n_pieces + n_whole;
  return w;
}

__device__ inline PItem item_of(const PArgs& a, const PWork& w, int i) {
  PItem it;
  if (i >= w.n_pieces) {
    it.u = int(blockIdx.x) + (i - w.n_pieces) * int(gridDim.x);
    it.k0 = 0;
    it.k1 = a.k_steps;
    it.slot = -1;
    it.r = -1;
    return it;
  }
  it.r = int(w.g0 / a.k_steps) + i;
  const int64_t lo = int64_t(it.r) * a.k_steps;
  it.u = a.n_full + it.r;
  it.k0 = int((w.g0 > lo ? w.g0 : lo) - lo);
  it.k1 = int((w.g1 < lo + a.k_steps ? w.g1 : lo + a.k_steps) - lo);
  // (CTA, split unit) pairs are ordered the same way in both: c + r is unique per piece
  it.slot = int(blockIdx.x) + it.r;
  return it;
}

// uses of stage st among the first n k-steps of a ring of nst stages
__device__ inline int stage_uses(int n, int st, int nst) { return n > st ? (n - 1 - st) / nst + 1 : 0; }

__device__ inline bool pwait(PBars& s, uint64_t* bar, uint32_t parity, int32_t* err) {
#pragma unroll 1
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 1023) == 1023 && *reinterpret_cast<volatile uint32_t*>(&s.abort)) return false;
  }
  set_err(err, LS_DEVERR_WAIT_TIMEOUT);
  *reinterpret_cast<volatile uint32_t*>(&s.abort) = 1;
  return false;
}

// The same by a whole warp.
__device__ inline bool pwait_warp(PBars& s, uint64_t* bar, uint32_t parity, int32_t* err) {
  return __all_sync(0xffffffffu, pwait(s, bar, parity, err));
}

template <bool kLora>
__global__ void __launch_bounds__(kPThreads, 1)
prologue_kernel(const __grid_constant__ PArgs a, const __grid_constant__ PLora lora, const __grid_constant__ CUtensorMap w0, const __grid_constant__ CUtensorMap x0,
                const __grid_constant__ CUtensorMap w1, const __grid_constant__ CUtensorMap x1,
                const __grid_constant__ CUtensorMap wl, const __grid_constant__ CUtensorMap xl) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  __shared__ PBars s;
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* a_ring = smem;                              // [kPAStages][16 KB]
  unsigned char* b_ring = a_ring + kPAStages * kPABytes;     // [kPBStages][32 KB]
  unsigned char* out_st = b_ring + kPBStages * kPBBytes;     // [128][128] bf16
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PWork w = work_of(a);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kPAStages; ++i) { mbar_init(&s.afull[i], 2); mbar_init(&s.aempty[i], 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(&s.acc_full[i], 1); mbar_init(&s.acc_empty[i], 128); }
    mbar_init(&s.out_full, 128);
    mbar_init(&s.out_free, 128);
    mbar_init(&s.drain, 1);
    mbar_init(&s.epi, 128);
    s.abort = 0;
    s.issued[0] = s.issued[1] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s.tmem_base)),
                 "r"(kPTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  // With adapters the kernel before is lora_low_kernel, which lets this one start once everything
  // before it has completed: only what it writes itself is waited for, by the epilogue (at its
  // start) and by the producers before their first adapter step.
  // (The producers wait for themselves: that of the weights once its first ring is on its way.)
  if (kLora ? warp >= 2 && warp <= 5 : warp != 0) {
    grid_dependency_wait();
    allow_dependent_launch();
  }

  // The sequences of a unit that take further k-steps for their adapters (whole warp): calls
  // step(sequence of the tile, adapter, rank chunk of 64) in order until it returns false.
  auto adapter_steps = [&](const PItem& it, const PUnit& u, auto&& step) -> bool {
    if constexpr (kLora) {
      if (u.p != 0 || it.k1 != a.k_steps) return true;
      const PProblem& P = a.pr[0];
      const int seq0 = u.mt * P.seq_per_unit, n = min(P.seq_per_unit, a.b - seq0);  // at most 16
      const int mine = lane < n ? lora.bank.adapter_of[seq0 + lane] : -1;
      for (unsigned todo = __ballot_sync(0xffffffffu, mine >= 0 && mine < lora.bank.n_adapters); todo; todo &= todo - 1) {
        const int i = __ffs(int(todo)) - 1, ad = __shfl_sync(0xffffffffu, mine, i);
        for (int rc = 0; rc < lora.bank.rank; rc += kPKStep)
          if (!step(i, ad, rc)) return false;
      }
    }
    return true;
  };

  // (The producers and the MMA issuer walk their loops as whole warps, one elected lane issuing:
  // what the loops work out is then the same in every lane, as the issued instructions want it.)
  auto produce = [&](auto weights) {
    constexpr bool is_a = decltype(weights)::value;
    constexpr int nst = is_a ? kPAStages : kPBStages;
    unsigned char* const ring = is_a ? a_ring : b_ring;
    constexpr int kBytes = is_a ? kPABytes : kPBBytes;
    // the weights are read once: they must not push the activations (read again by
    // every weight tile of the layer) out of L2
    const uint64_t pol = is_a ? l2_evict_first() : l2_evict_last();
    bool waited = !kLora && !is_a, ok = true;
    auto wait_grid = [&]() {
      if (waited) return;
      grid_dependency_wait();
      allow_dependent_launch();
      waited = true;
    };
    int k = 0, st = 0, bar = 0;      // k-step; its stage of this ring; its barrier
    int back = 0, back_parity = 0;   // k - nst's barrier and its phase
    // k-step k's stage is free for its next copy (false: gave up): the MMAs of the k-step that
    // used it before (k - nst) have completed. The MMAs of a k-step complete in order, and the
    // one wait before for the same barrier covered its previous phase, so the parity names this
    // phase.
    auto begin_step = [&]() -> bool {
      if (k < nst) return true;
      if (!kLora) wait_grid();  // (the first ring's weights are in flight)
      if (!pwait_warp(s, &s.aempty[back], uint32_t(back_parity), a.err)) return false;
      if (++back == kPAStages) { back = 0; back_parity ^= 1; }
      return true;
    };
    auto end_step = [&]() {
      __syncwarp();
      ++k;
      if (++st == nst) st = 0;
      if (++bar == kPAStages) bar = 0;
    };
    for (int i = 0; i < w.n_items && ok; ++i) {
      const PItem it = item_of(a, w, i);
      const PUnit u = unit_of(a, it.u);
      const PProblem& P = a.pr[u.p];
      const CUtensorMap* m = is_a ? (u.p ? &w1 : &w0) : (u.p ? &x1 : &x0);
      const uint32_t bytes = is_a ? uint32_t(kPABytes) : uint32_t(P.load_rows * kPKStep * 2);
      const int row = is_a ? u.l * P.n_out + u.nt * kPTileN : u.mt * P.seq_per_unit;
      const bool is_4d = P.is_4d;
      for (int ks = it.k0; ks < it.k1; ++ks) {
        if (!begin_step()) { ok = false; break; }
        if (elect_one()) {
          uint64_t* full = &s.afull[bar];
          mbar_arrive_expect_tx(full, bytes);
          if constexpr (is_a) tma_load_2d_hint(ring + st * kBytes, m, ks * kPKStep, row, full, pol);
          else if (is_4d) tma_load_4d_hint(ring + st * kBytes, m, ks * kPKStep, 0, u.l, row, full, pol);
          else tma_load_3d_hint(ring + st * kBytes, m, ks * kPKStep, u.l, row, full, pol);
        }
        end_step();
      }
      if (!ok) break;
      ok = adapter_steps(it, u, [&](int i, int ad, int rc) -> bool {
        wait_grid();
        if (!begin_step()) return false;
        if (elect_one()) {
          uint64_t* full = &s.afull[bar];
          mbar_arrive_expect_tx(full, is_a ? uint32_t(kPABytes) : uint32_t(2 * P.pitch * kPKStep * 2));
          if constexpr (is_a)
            tma_load_2d(ring + st * kBytes, &wl, rc, (ad * a.L + u.l) * P.n_out + u.nt * kPTileN, full);
          else
            tma_load_2d(ring + st * kBytes, &xl, rc, ((row + i) * a.L + u.l) * 2 * P.pitch, full);
        }
        end_step();
        return true;
      });
    }
    if (lane == 0) s.issued[is_a ? 0 : 1] = k;
    wait_grid();  // (every thread of the CTA passes the wait before it triggers)
  };

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producers
    // warp 0: the weights (A) of every k-step; warp 6: the activations (B)
    if (lane == 0) { prefetch_map(&w0); prefetch_map(&w1); }
    produce(std::true_type{});
  } else if (warp == 6) {
    if (lane == 0) { prefetch_map(&x0); prefetch_map(&x1); }
    produce(std::false_type{});
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    bool ok = true;
    int sa = 0, sb = 0;       // the k-step's stages
    uint32_t parity = 0;      // of its barrier
    const uint64_t da0 = sdesc(smem_u32(a_ring), 16, 1024), db0 = sdesc(smem_u32(b_ring), 16, 1024);
    bool ready = false;       // the k-step's copies were seen complete during the one before
    auto begin_step = [&]() -> bool {
      if (!__all_sync(0xffffffffu, ready) && !pwait_warp(s, &s.afull[sa], parity, a.err)) return false;
      tc_fence_after();
      // asked now, needed after the MMAs' issue (an answer takes about 200 cycles)
      const bool wrap = sa + 1 == kPAStages;
      ready = mbar_test(&s.afull[wrap ? 0 : sa + 1], parity ^ uint32_t(wrap));
      return true;
    };
    auto end_step = [&]() {
      __syncwarp();
      if (++sa == kPAStages) { sa = 0; parity ^= 1; }
      if (++sb == kPBStages) sb = 0;
    };
    for (int i = 0; i < w.n_items && ok; ++i) {
      const PItem it = item_of(a, w, i);
      const PUnit u = unit_of(a, it.u);
      const PProblem& P = a.pr[u.p];
      const int ab = i & 1;
      if (!pwait_warp(s, &s.acc_empty[ab], ((i >> 1) & 1) ^ 1, a.err)) break;
      tc_fence_after();
      const uint32_t id = idesc_bf16(P.act_rows, false, kPTileN);
      const uint32_t d = tmem + uint32_t(ab * kPMaxAct);
      for (int ks = it.k0; ks < it.k1; ++ks) {
        if (!begin_step()) { ok = false; break; }
        const uint64_t da = da0 + uint32_t(sa * (kPABytes >> 4)), db = db0 + uint32_t(sb * (kPBBytes >> 4));
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kPKStep / 16; ++kk)  // K = 16 per MMA: 32 bytes along the row
            mma_bf16(d, da + uint32_t(kk * 2), db + uint32_t(kk * 2), id, (ks > it.k0 || kk > 0) ? 1u : 0u);
          mma_commit(&s.aempty[sa]);  // frees both stages of the k-step
        }
        end_step();
      }
      if (ok)
        ok = adapter_steps(it, u, [&](int i, int, int rc) -> bool {
          if (!begin_step()) return false;
          const uint64_t da = da0 + uint32_t(sa * (kPABytes >> 4)), db = db0 + uint32_t(sb * (kPBBytes >> 4));
          const uint32_t ids = idesc_bf16(P.pitch, false, kPTileN), ds = d + uint32_t(i * P.pitch);
          const uint32_t low_part = uint32_t(P.pitch * kPKStep * 2 >> 4);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kPKStep / 16; ++kk) {
              if (rc + 16 * kk >= lora.bank.rank) break;
#pragma unroll
              for (int part = 0; part < 2; ++part)  // the high and the low part of the inner products
                mma_bf16(ds, da + uint32_t(kk * 2), db + part * low_part + uint32_t(kk * 2), ids, 1u);
            }
            mma_commit(&s.aempty[sa]);
          }
          end_step();
          return true;
        });
      if (ok && elect_one()) mma_commit(&s.acc_full[ab]);
      __syncwarp();
    }
    if (kLora) {  // (every thread passes the wait before it triggers)
      grid_dependency_wait();
      allow_dependent_launch();
    }
  } else {
    // ------------------------------------------------------------ epilogue (warps 2-5)
    // Per 128 activation rows: each thread writes its weight row's outputs (a column of the
    // staging tile [row][128 weight rows]), then all 128 threads copy the tile's valid rows
    // out as 16-byte pieces of 256-byte output rows. fetch(col, v) gives the thread's 32
    // accumulator values of activation rows col .. col + 31 (TMEM, or summed partials).
    const int sub = warp & 3;
    const int ecol = 32 * sub + lane;  // this thread's weight row within the unit
    const int etid = threadIdx.x - 64;  // 0..127
    const uint32_t trow = tmem + (uint32_t(32 * sub) << 16);
    __nv_bfloat16* stage = reinterpret_cast<__nv_bfloat16*>(out_st);
    int pass = 0;  // epilogue passes so far (phases of out_full / out_free)
    int meets = 0;  // phases of `epi` so far
    bool ok = true;
    // all 128 epilogue threads meet here (bounded: a thread that gave up makes the rest give up)
    auto epi_meet = [&]() -> bool {
      mbar_arrive(&s.epi);
      return __all_sync(0xffffffffu, pwait(s, &s.epi, uint32_t(meets++) & 1, a.err));
    };
    // the adapters' part of boundary rows col .. col + n - 1, for this thread's weight row
    auto add_boundary = [&](const PUnit& u, const PProblem& P, int col, int n, float (&v)[32]) {
      const int sq = u.mt * P.seq_per_unit + col;
      const float* add = lora.add + (int64_t(sq) * a.L + u.l) * P.n_out + u.nt * kPTileN + ecol;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        if (j >= n) break;
        const int ad = lora.bank.adapter_of[sq + j];
        if (ad >= 0 && ad < lora.bank.n_adapters) v[j] += __ldcg(add + int64_t(j) * a.L * P.n_out);
      }
    };
    auto store_tile = [&](const PUnit& u, const PProblem& P, auto&& fetch) -> bool {
      const int seq0 = u.mt * P.seq_per_unit;
      const int rows = min(P.seq_per_unit, a.b - seq0) * P.pitch;  // activation rows of the tile
      for (int r0 = 0; r0 < rows; r0 += kPOutRows, ++pass) {
        // the staging tile is free once every thread has copied the previous pass out
        if (pass > 0 && !__all_sync(0xffffffffu, pwait(s, &s.out_free, (pass - 1) & 1, a.err))) return false;
        const int nr = min(kPOutRows, P.act_rows - r0);
        for (int c0 = 0; c0 < nr; c0 += 32) {
          float v[32];
          fetch(r0 + c0, v);
          if constexpr (kLora) {
            if (u.p && r0 + c0 < rows) add_boundary(u, P, r0 + c0, min(32, rows - r0 - c0), v);
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) stage[(c0 + j) * kPTileN + ecol] = __float2bfloat16_rn(v[j]);
        }
        mbar_arrive(&s.out_full);
        if (!__all_sync(0xffffffffu, pwait(s, &s.out_full, pass & 1, a.err))) return false;
        const int vr = min(kPOutRows, rows - r0);
        for (int c = etid; c < vr * 16; c += 128) {  // 16 pieces of 16 bytes per row
          const int m = r0 + (c >> 4);
          const int sq = seq0 + m / P.pitch, r = m % P.pitch;
          if (r >= P.rows_per_seq) continue;
          uint4* dst = reinterpret_cast<uint4*>(P.y + ((int64_t(sq) * a.L + u.l) * P.rows_per_seq + r) * P.n_out +
                                                u.nt * kPTileN) + (c & 15);
          *dst = reinterpret_cast<const uint4*>(stage + (c >> 4) * kPTileN)[c & 15];
        }
        mbar_arrive(&s.out_free);
      }
      return true;
    };
    for (int i = 0; i < w.n_items && ok; ++i) {
      const PItem it = item_of(a, w, i);
      const PUnit u = unit_of(a, it.u);
      const PProblem& P = a.pr[u.p];
      const int ab = i & 1;
      if (!__all_sync(0xffffffffu, pwait(s, &s.acc_full[ab], (i >> 1) & 1, a.err))) break;
      tc_fence_after();
      if (it.slot < 0) {
        ok = store_tile(u, P, [&](int col, float (&v)[32]) { tmem_ld32(trow + uint32_t(ab * kPMaxAct + col), v); });
        tc_fence_before();
        mbar_arrive(&s.acc_empty[ab]);
        continue;
      }
      // a piece of a split tile: its partial sums (this thread's weight row, all activation
      // rows) go to its slot, and the accumulator is released at once
      const int na = P.act_rows;  // a multiple of 16
      float* mine = a.part + (int64_t(it.slot) * kPTileN + ecol) * na;
      for (int c0 = 0; c0 < na; c0 += 32) {
        float v[32];
        tmem_ld32(trow + uint32_t(ab * kPMaxAct + c0), v);
#pragma unroll
        for (int j = 0; j < 32; j += 4)
          if (c0 + j < na) *reinterpret_cast<float4*>(mine + c0 + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
      }
      tc_fence_before();
      mbar_arrive(&s.acc_empty[ab]);
      __threadfence();  // this thread's partials are visible before the arrival below
      if (!epi_meet()) { ok = false; break; }
      const int64_t T = a.rem_steps;
      const int G = int(gridDim.x);
      const int c_first = range_cta(int64_t(it.r) * a.k_steps, T, G);
      const int c_last = range_cta(int64_t(it.r + 1) * a.k_steps - 1, T, G);
      if (etid == 0) s.last = atomicAdd(a.count + it.r, 1) == c_last - c_first ? 1u : 0u;
      if (!epi_meet()) { ok = false; break; }
      if (!s.last) continue;
      __threadfence();  // every piece's partials are visible from here on
      ok = store_tile(u, P, [&](int col, float (&v)[32]) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0.f;
        for (int c = c_first; c <= c_last; ++c) {  // slot order: the same sum for every arrival order
          const float* src = a.part + (int64_t(c + it.r) * kPTileN + ecol) * na + col;
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            if (col + j < na) {
              const float4 x = __ldcg(reinterpret_cast<const float4*>(src + j));
              v[j] += x.x; v[j + 1] += x.y; v[j + 2] += x.z; v[j + 3] += x.w;
            }
          }
        }
      });
      if (etid == 0) a.count[it.r] = 0;  // ready for the next call
    }
  }

  __syncthreads();
  if (warp == 0 && lane == 0 && s.abort) {
    // let the copies still in flight land before the shared memory is released: a k-step
    // barrier that only one producer arrived for (the other gave up first; the producers
    // are at most a ring apart, so by one use of a barrier) gets the other's arrival, then
    // each barrier's last phase completes once its copies have landed
    for (int st = 0; st < kPAStages; ++st) {
      const int na = stage_uses(s.issued[0], st, kPAStages), nb = stage_uses(s.issued[1], st, kPAStages);
      if (na != nb) mbar_arrive(&s.afull[st]);
      const int n = na > nb ? na : nb;
      if (n > 0) mbar_wait_bounded(&s.afull[st], uint32_t(n - 1) & 1, kWaitLimit);
    }
  }
  if (warp == 1 && s.abort && elect_one()) {
    // and the MMAs issued so far, before TMEM is released
    mma_commit(&s.drain);  // tracks every MMA this thread (the same one each time) issued
    mbar_wait_bounded(&s.drain, 0, kWaitLimit);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kPTmemCols) : "memory");
  }
}

// low = scale (A x), a CTA per (sequence, layer) and 8 NT of the rank, and one for its boundary row
// (the whole rank, and its outputs).
// Its bytes (x and A once each) are few beside the weights'; what counts is the latency, as the
// projections' kernel follows: the warps spread over the hidden size, 64 entries at a time. A
// thread's 32-byte load of sixteen entries of a row is its part of four m16n8k16 products'
// operands (their k order is free), and a row's four threads read a whole 128-byte line: with
// 16-byte loads, half lines, the L1 cache was the bound (64 requests at rank 64: 57 us instead of
// 47, 16 at rank 16: 13 instead of 9). Where x or A is not 32-byte aligned, two 16-byte loads take
// its place. The warps' sums are added in warp order. Boundary rows grouped by adapter, so that A
// and B are read once for several of them, made their CTAs' chains longer: 60 us. (Run beside the
// projections instead, a warp per 8 of the rank and no shared memory, it took longer than their
// first units: 160 us instead of 82 for 16 requests at rank 16.)
// (two CTAs per SM with 8 warps where the loads in flight need the registers)
__host__ __device__ constexpr int low_warps(int nt) { return nt <= 2 ? 16 : 8; }
constexpr int kLoraMaxRank = 128;

__device__ inline void mma_bf16_warp(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// This warp's part of acc = x A^T: 64 of every 64 W hidden entries. xr: the rows g and g + 8 of
// MT 16-row tiles (or, with one row, that row); wr: row g of NT 8-row tiles of A; both from this
// thread's entry on.
template <int MT, int NT, int W, bool kWide, int NX>
__device__ inline void low_products(float (&acc)[MT][NT][4], const __nv_bfloat16* const (&xr)[NX],
                                    const __nv_bfloat16* const (&wr)[NT], int hidden, int warp) {
  auto load = [](const __nv_bfloat16* p, uint4 (&v)[2]) {
    if constexpr (kWide) {
      ld_nc_v8(p, v[0], v[1]);
    } else {
      v[0] = ld_nc_v4(p);
      v[1] = ld_nc_v4(p + 8);
    }
  };
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.f;
  constexpr int kAhead = NX + NT <= 4 ? 2 : 1;  // steps whose loads are in flight together
#pragma unroll 1
  for (int k0 = warp * 64; k0 < hidden; k0 += 64 * W * kAhead) {
    uint4 av[kAhead][NX][2], bv[kAhead][NT][2];
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
      const int k = min(k0 + 64 * W * s, hidden - 64);
#pragma unroll
      for (int m = 0; m < NX; ++m) load(xr[m] + k, av[s][m]);
#pragma unroll
      for (int n = 0; n < NT; ++n) load(wr[n] + k, bv[s][n]);
    }
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
      if (k0 + 64 * W * s >= hidden) break;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const uint4 &lo = av[s][NX == 1 ? 0 : 2 * m][h], &hi = av[s][NX == 1 ? 0 : 2 * m + 1][h], &w = bv[s][n][h];
            mma_bf16_warp(acc[m][n], lo.x, hi.x, lo.y, hi.y, w.x, w.y);
            mma_bf16_warp(acc[m][n], lo.z, hi.z, lo.w, hi.w, w.z, w.w);
          }
    }
  }
}

// MT: 16-row tiles of activation rows (block rows up to 32). NT: 8-entry tiles of the rank. (Rows
// and rank entries past the last are read as the last one again and not stored: with a branch
// per tile the loads would wait for one another.)
template <int MT, int NT, bool kWide>
__global__ void __launch_bounds__(low_warps(NT) * 32, NT == 4 ? 2 : 1) lora_low_kernel(const __grid_constant__ PLora lora, const __nv_bfloat16* x,
                                                                  const __nv_bfloat16* boundary, int L, int B,
                                                                  int hidden, int n_kv, int32_t* err) {
  constexpr int kLowWarps = low_warps(NT);
  __shared__ __align__(16) float red[kLowWarps][16][8 * NT + 2];
  __shared__ float low_s[kLoraMaxRank];
  const int R = lora.bank.rank;
  const int b = int(blockIdx.x) / L, l = int(blockIdx.x) - b * L;
  // the first CTAs, which have most to do: a (sequence, layer)'s boundary row, the whole rank
  const bool p = blockIdx.y == 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  grid_dependency_wait();
  allow_dependent_launch();
  const int ad = lora.bank.adapter_of[b];
  if (ad < 0 || ad >= lora.bank.n_adapters) {  // none: its place is read by the epilogue and left out
    if (ad != -1 && threadIdx.x == 0) set_err(err, LS_DEVERR_ADAPTER);
    return;
  }
  const __nv_bfloat16* bank = static_cast<const __nv_bfloat16*>(p ? lora.bank.a_kv : lora.bank.a_q) +
                              (int64_t(ad) * L + l) * R * hidden + t * 16;
  const float scale = lora.bank.scale[ad];
  if (!p) {
    const int r0 = int(blockIdx.y - 1) * 8 * NT, nr = min(8 * NT, R - r0);
    const __nv_bfloat16 *xr[2 * MT], *wr[NT];
#pragma unroll
    for (int m = 0; m < 2 * MT; ++m)
      xr[m] = x + ((int64_t(b) * L + l) * B + min(m * 8 + g, B - 1)) * hidden + t * 16;
#pragma unroll
    for (int n = 0; n < NT; ++n) wr[n] = bank + int64_t(r0 + min(8 * n + g, nr - 1)) * hidden;
    float acc[MT][NT][4];
    low_products<MT, NT, kLowWarps, kWide>(acc, xr, wr, hidden, warp);
    const int pitch = (B + 15) & ~15;  // (rows past the block feed columns that are not stored)
    __nv_bfloat16* split = lora.split + (int64_t(b) * L + l) * 2 * pitch * R;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        *reinterpret_cast<float2*>(&red[warp][g][8 * n + 2 * t]) = make_float2(acc[m][n][0], acc[m][n][1]);
        *reinterpret_cast<float2*>(&red[warp][g + 8][8 * n + 2 * t]) = make_float2(acc[m][n][2], acc[m][n][3]);
      }
      __syncthreads();
      for (int i = threadIdx.x; i < 16 * nr; i += kLowWarps * 32) {
        const int row = 16 * m + i / nr, r = i % nr;
        if (row >= B) break;
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < kLowWarps; ++v) sum += red[v][i / nr][r];
        sum *= scale;
        const __nv_bfloat16 hi = __float2bfloat16_rn(sum);
        const float rest = sum - __bfloat162float(hi);
        split[row * R + r0 + r] = hi;
        split[(pitch + row) * R + r0 + r] = __float2bfloat16_rn(fabsf(rest) < INFINITY ? rest : 0.f);  // (an infinite sum stays infinite)
      }
      __syncthreads();
    }
    return;
  }
  const __nv_bfloat16* const xr[1] = {boundary + (int64_t(b) * L + l) * hidden + t * 16};
  float* const part = &red[0][0][0];  // [warps][8 NT]
  for (int r0 = 0; r0 < R; r0 += 8 * NT) {
    const int nr = min(8 * NT, R - r0);
    const __nv_bfloat16* wr[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) wr[n] = bank + int64_t(r0 + min(8 * n + g, nr - 1)) * hidden;
    float acc[1][NT][4];
    low_products<1, NT, kLowWarps, kWide>(acc, xr, wr, hidden, warp);
    if (g == 0) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
        *reinterpret_cast<float2*>(part + (warp * NT + n) * 8 + 2 * t) = make_float2(acc[0][n][0], acc[0][n][1]);
    }
    __syncthreads();
    if (int(threadIdx.x) < nr) {
      float sum = 0.f;
#pragma unroll
      for (int v = 0; v < kLowWarps; ++v) sum += part[v * NT * 8 + threadIdx.x];
      low_s[r0 + threadIdx.x] = sum * scale;
    }
    __syncthreads();
  }
  // the boundary row's outputs: kOut weight rows per thread at a time, their loads together
  constexpr int kOut = 4, kThreads = kLowWarps * 32;
  const __nv_bfloat16* wb = static_cast<const __nv_bfloat16*>(lora.bank.b_kv) + (int64_t(ad) * L + l) * n_kv * R;
  float* add = lora.add + (int64_t(b) * L + l) * n_kv;
  for (int n0 = threadIdx.x; n0 < n_kv; n0 += kOut * kThreads) {
    float y[kOut] = {};
#pragma unroll 2
    for (int e = 0; e < R; e += 8) {
      uint4 w[kOut];
#pragma unroll
      for (int u = 0; u < kOut; ++u) w[u] = ld_nc_v4(wb + int64_t(min(n0 + u * kThreads, n_kv - 1)) * R + e);
#pragma unroll
      for (int u = 0; u < kOut; ++u) {
        float f[8];
        Elem<__nv_bfloat16>::to_f32(w[u], f);
#pragma unroll
        for (int q = 0; q < 8; ++q) y[u] = fmaf(f[q], low_s[e + q], y[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kOut; ++u)
      if (n0 + u * kThreads < n_kv) add[n0 + u * kThreads] = y[u];
  }
}

bool encode_bf16(void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
                 CUtensorMap* out) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, cuuint32_t(rank), base, dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool prologue_supported(const Dev& p) { return prologue_shapes_ok(p.dtype, p.hidden, p.Hq, p.Hkv, p.D, p.B); }

size_t lora_workspace_bytes(const ls_config& c, int rank) {
  // the block rows' inner products, then the boundary rows' finished sums
  const int64_t bl = int64_t(c.batch) * c.n_layers;
  return size_t(align256(bl * ((c.block + 15) & ~15) * rank * 4) + align256(bl * 2 * c.n_kv_heads * c.head_dim * 4));
}

cudaError_t launch_prologue(const Dev& p, const void* w_kv, const void* w_q, const void* x, const ls_lora* lora,
                            void* low, void* bkv, void* q, int sms, cudaStream_t stream) {
  const auto kernel = lora ? prologue_kernel<true> : prologue_kernel<false>;
  // per launch: the attribute belongs to the current device's copy of the kernel
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPSmemBytes);
  if (e != cudaSuccess) return e;
  PArgs a{};
  a.b = p.b;
  a.L = p.L;
  a.k_steps = p.hidden / kPKStep;
  a.err = p.err;
  const cuuint64_t hb = cuuint64_t(p.hidden) * 2;
  // problem 0: block queries, X = x [b][L][B][hidden]
  PProblem& Q = a.pr[0];
  Q.n_out = p.Hq * p.D;
  Q.rows_per_seq = p.B;
  Q.pitch = lora ? (p.B + 15) & ~15 : p.B;
  Q.seq_per_unit = kPMaxAct / Q.pitch < p.b ? kPMaxAct / Q.pitch : p.b;
  Q.load_rows = Q.seq_per_unit * Q.pitch;
  Q.act_rows = (Q.load_rows + 15) & ~15;
  Q.m_tiles = (p.b + Q.seq_per_unit - 1) / Q.seq_per_unit;
  Q.n_units = p.L * (Q.n_out / kPTileN) * Q.m_tiles;
  Q.is_4d = 1;
  Q.y = static_cast<__nv_bfloat16*>(q);
  // problem 1: boundary keys/values, X = the state's boundary view [b][L][hidden]
  PProblem& K = a.pr[1];
  K.n_out = 2 * p.Hkv * p.D;
  K.rows_per_seq = K.pitch = 1;
  K.seq_per_unit = p.b < kPMaxAct ? p.b : kPMaxAct;
  K.load_rows = K.seq_per_unit;
  K.act_rows = (K.load_rows + 15) & ~15;
  K.m_tiles = (p.b + K.seq_per_unit - 1) / K.seq_per_unit;
  K.n_units = p.L * (K.n_out / kPTileN) * K.m_tiles;
  K.is_4d = 0;
  K.y = static_cast<__nv_bfloat16*>(bkv);
  a.n_units = Q.n_units + K.n_units;

  CUtensorMap mw0, mx0, mw1, mx1;
  {
    const cuuint64_t dims[2] = {cuuint64_t(p.hidden), cuuint64_t(p.L) * Q.n_out};
    const cuuint64_t str[1] = {hb};
    const cuuint32_t box[2] = {kPKStep, kPTileN};
    if (!encode_bf16(const_cast<void*>(w_q), 2, dims, str, box, &mw0)) return cudaErrorInvalidValue;
  }
  {
    const cuuint64_t dims[4] = {cuuint64_t(p.hidden), cuuint64_t(p.B), cuuint64_t(p.L), cuuint64_t(p.b)};
    const cuuint64_t str[3] = {hb, hb * p.B, hb * p.B * p.L};
    const cuuint32_t box[4] = {kPKStep, cuuint32_t(Q.pitch), 1, cuuint32_t(Q.seq_per_unit)};
    if (!encode_bf16(const_cast<void*>(x), 4, dims, str, box, &mx0)) return cudaErrorInvalidValue;
  }
  {
    const cuuint64_t dims[2] = {cuuint64_t(p.hidden), cuuint64_t(p.L) * K.n_out};
    const cuuint64_t str[1] = {hb};
    const cuuint32_t box[2] = {kPKStep, kPTileN};
    if (!encode_bf16(const_cast<void*>(w_kv), 2, dims, str, box, &mw1)) return cudaErrorInvalidValue;
  }
  {
    // (rows past the batch in a last, partial tile read as zeros: out of the tensor's bounds)
    const cuuint64_t dims[3] = {cuuint64_t(p.hidden), cuuint64_t(p.L), cuuint64_t(p.b)};
    const cuuint64_t str[2] = {hb, hb * p.L};
    const cuuint32_t box[3] = {kPKStep, 1, cuuint32_t(K.load_rows)};
    if (!encode_bf16(p.boundary, 3, dims, str, box, &mx1)) return cudaErrorInvalidValue;
  }
  PLora pl{};
  CUtensorMap mwl = mw0, mxl = mx0;  // (unused without adapters)
  if (lora) {
    pl.bank = *lora;
    pl.split = static_cast<__nv_bfloat16*>(low);
    pl.add = reinterpret_cast<float*>(static_cast<char*>(low) + align256(int64_t(p.b) * p.L * Q.pitch * lora->rank * 4));
    // the tiles' inner extent is 64 of the rank; what lies past it reads as zeros
    const cuuint64_t rb = cuuint64_t(lora->rank) * 2;
    const int64_t w_rows = int64_t(lora->n_adapters) * p.L * Q.n_out, x_rows = int64_t(p.b) * p.L * 2 * Q.pitch;
    if (w_rows > INT32_MAX || x_rows > INT32_MAX) return cudaErrorNotSupported;
    const cuuint64_t wd[2] = {cuuint64_t(lora->rank), cuuint64_t(w_rows)}, xd[2] = {cuuint64_t(lora->rank), cuuint64_t(x_rows)};
    const cuuint64_t str[1] = {rb};
    const cuuint32_t wbox[2] = {kPKStep, kPTileN}, xbox[2] = {kPKStep, cuuint32_t(2 * Q.pitch)};
    if (!encode_bf16(const_cast<void*>(lora->b_q), 2, wd, str, wbox, &mwl)) return cudaErrorInvalidValue;
    if (!encode_bf16(low, 2, xd, str, xbox, &mxl)) return cudaErrorInvalidValue;
    const int tiles = lora->rank <= 8 ? 1 : (lora->rank <= 16 ? 2 : 4);  // (x is read again for each 32 of the rank)
    const bool two = p.B > 16;
    const bool wide = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(lora->a_q) |
                        reinterpret_cast<uintptr_t>(lora->a_kv)) & 31) == 0;  // (rows are whole 128 bytes, the boundary view is aligned)
    auto pick = [&](auto w) {
      constexpr bool kWide = decltype(w)::value;
      return tiles == 1   ? (two ? lora_low_kernel<2, 1, kWide> : lora_low_kernel<1, 1, kWide>)
             : tiles == 2 ? (two ? lora_low_kernel<2, 2, kWide> : lora_low_kernel<1, 2, kWide>)
                          : (two ? lora_low_kernel<2, 4, kWide> : lora_low_kernel<1, 4, kWide>);
    };
    const auto low_kernel = wide ? pick(std::true_type{}) : pick(std::false_type{});
    e = launch_overlapped(low_kernel, dim3(p.b * p.L, (lora->rank + 8 * tiles - 1) / (8 * tiles) + 1), low_warps(tiles) * 32, 0, stream,
                          pl, static_cast<const __nv_bfloat16*>(x), reinterpret_cast<const __nv_bfloat16*>(p.boundary), p.L, p.B,
                          p.hidden, K.n_out, p.err);
    if (e != cudaSuccess) return e;
  }
  int grid = sms < kProMaxGrid ? sms : kProMaxGrid;
  if (a.n_units < grid) grid = a.n_units;
  // units left over after whole waves: split their k-steps over every CTA when they are all
  // boundary tiles (their partial sums fit the state's scratch: 128 x K.act_rows fp32 each)
  // and there are at least as many k-steps as CTAs (then every CTA's range is non-empty, so
  // a tile's pieces are those of the CTAs from the one holding its first k-step to the one
  // holding its last; with fewer, the CTAs between could hold none and the tile's arrival
  // count would never be reached)
  const int rem = a.n_units % grid;
  const bool split = rem > 0 && rem <= K.n_units && K.act_rows == prologue_boundary_rows(p.b) &&
                     int64_t(rem) * a.k_steps >= grid;
  a.n_full = split ? a.n_units - rem : a.n_units;
  a.rem_steps = split ? rem * a.k_steps : 0;
  a.part = p.pro_part;
  a.count = p.pro_count;
  return launch_overlapped(kernel, dim3(grid), kPThreads, kPSmemBytes, stream, a, pl, mw0, mx0, mw1, mx1, mwl, mxl);
}

}  // namespace ls
