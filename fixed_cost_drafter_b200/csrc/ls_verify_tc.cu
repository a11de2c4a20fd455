// ls_verify_attend_kv4 for many query rows per KV head (a verification pass's B + 1 rows of a
// GQA group) of bf16 states, on the 5th-generation tensor cores.
//
// Measured: 16 requests x 17 rows (68 rows per KV head) at 32K-64K tokens, 906 MB of cache: 520 to
// 550 us over runs (1.7 TB/s), 13.9 ms on CUDA cores. What bounds it: instructions and the
// latencies between roles. The two products of a 128-key chunk (128 rows x 128 keys x D each)
// need 1024 cycles, its bytes about 760 at the copy rate, its weights' exponentials 1024 (68 rows
// fill the lanes of three SM sub-partitions); a chunk takes about 2500, for some 4500 warp
// instructions at 0.45 a cycle and sub-partition. A wait for a barrier costs about 200 cycles
// even when its phase is complete, so each role takes large steps. Tried without gain: a third
// softmax group with its own S buffer, four groups of half-chunks, 28 and 32 warps (fewer
// registers, more instructions), codes fetched by the converting threads themselves (into
// registers or with cp.async: every later fence or load waits for them).
//
// One CTA per SM, 20 warps; the roles meet at mbarriers:
//   warp 10     producer: a chunk's pages into a ring of 3 stages (ls_verify.cuh)
//   warps 11-19 conversion, with the softmax warps that have no rows (68 rows leave two idle, in
//               the SM sub-partition that then has no softmax at all): tasks of 32 rows of a
//               chunk's K or V, round robin, a thread 16 codes (one scale group) at a time; tiles
//               in the 128-byte swizzle, two buffers each. A group's two 16-byte pieces go to
//               different 64-column halves (D = 128), so that eight threads fill a whole 128-byte
//               row; Q and the output columns follow the same order.
//   warp 8      S = Q K^T of a chunk into one of two 128-column buffers
//   warps 0-7   softmax, a thread per query row, 64 keys at a time: weights 2^(x - r) in fp16. The
//               reference r only moves when 64 weights sum to more than 2^15 (fp16 holds up to
//               65504); it is then the maximum less 8, as in ls_verify_mma.cu, and the row of O is
//               scaled in TMEM. The sum is needed anyway: the check costs no maximum. Warps 0-3
//               take the even chunks, 4-7 the odd ones; one O needs one reference, so a group
//               passes it on with each chunk (a counter in shared memory) and takes the other's
//               up before it hands its weights over.
//   warp 9      O += P V, 64 keys at a time, P the MMA's A operand in TMEM. (P over S instead held
//               each S buffer until its P V was done: 513 us.)
// TMEM columns: S 0-255, O 256-383, P 384-511.
// Rounding, exactness of the held values and NaN groups: as in ls_verify_mma.cu.
#include "ls_verify.cuh"
#include "ls_tc.cuh"

namespace ls {

namespace {

constexpr int kTThreads = 640;
constexpr int kTQkWarp = 8, kTPvWarp = 9, kTLoadWarp = 10, kTConvWarp = 11;
constexpr int kTRing = 3;          // stages of raw chunks
constexpr int kTUnit = 32;         // rows of a conversion task
constexpr int kTUnits = kVerChunk / kTUnit;  // of a chunk's keys, and as many of its values
constexpr int kTSub = 64;          // keys the softmax takes at a time
constexpr uint32_t kTCols = 512, kTO = 256, kTP = 384;
constexpr float kTRoom = 8.f;
constexpr float kTMostSum = 32768.f;
constexpr int kNanSlots = 4;       // pieces whose NaN positions are kept (conversion runs at most 2 ahead)

struct TBars {
  uint64_t raw_full[kTRing], raw_empty[kTRing];
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2];
  uint64_t s_full[2], s_free[2], p_full[4], p_free[2];  // p_full: [buffer][half]
  uint64_t h_done;  // the first half's P V
  uint64_t joined[4];      // both warps' sums of a piece
  uint64_t q_full, o_full, o_free, drain[2];
  uint32_t tmem_base, abort;
  uint32_t turn[4];  // chunks whose reference is decided, per 32 rows
  int nan_at[kNanSlots][8];
  float ref[kTcRows];
  float2 state[2][2][kTcRows];  // [piece parity][warp group]: sum and reference of a row
};

// kind::f16 with fp16 A/B, fp32 D
constexpr uint32_t idesc_f16(int n, bool b_mn_major) {
  return (1u << 4) | (uint32_t(b_mn_major) << 16) | (uint32_t(n >> 3) << 17) | (uint32_t(128 >> 4) << 24);
}

__device__ inline void tmem_st16u(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ inline void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The counter of decided chunks: passed on by a release store, polled with a bound.
__device__ inline void turn_set(uint32_t* p, uint32_t v) {
  asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(smem_u32(p)), "r"(v) : "memory");
}
__device__ inline bool turn_wait(TBars& s, uint32_t* p, uint32_t v, int32_t* err) {
  uint32_t x = 0;
#pragma unroll 1
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(x) : "r"(smem_u32(p)) : "memory");
    if (x == v || ((i & 1023) == 1023 && *reinterpret_cast<volatile uint32_t*>(&s.abort))) break;
  }
  if (x != v) {
    if (!*reinterpret_cast<volatile uint32_t*>(&s.abort)) set_err(err, LS_DEVERR_WAIT_TIMEOUT);
    *reinterpret_cast<volatile uint32_t*>(&s.abort) = 1;
  }
  return __all_sync(0xffffffffu, x == v);
}

__device__ inline void fma2(float& x, float& y, float a, float b) {  // x, y = x * a + b, y * a + b
  asm("{\n\t.reg .b64 u, v, w;\n\t"
      "mov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %2};\n\tmov.b64 w, {%3, %3};\n\t"
      "fma.rn.f32x2 u, u, v, w;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
__device__ inline void add2(float& x, float& y, float a, float b) {
  asm("{\n\t.reg .b64 u, v;\n\t"
      "mov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\t"
      "add.rn.f32x2 u, u, v;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
// Column position n of the K / V tiles holds dim dim_of(n): see the conversion.
template <int D>
__device__ constexpr int dim_of(int n) {
  return D == 128 ? 16 * ((n & 63) >> 3) + 8 * (n >> 6) + (n & 7) : n;
}

template <int D>
__global__ void __launch_bounds__(kTThreads, 1) verify_tc_kernel(const VerArgs a) {
  constexpr int kTile = kVerChunk * D * 2;     // one K or V buffer
  constexpr int kRaw = kVerChunk * (D + D / 8);  // a raw chunk
  constexpr int kHalf = kVerChunk * 128;       // 64 columns of it
  constexpr int kGroups = D / kKv4Group;       // threads per row in the conversion
  constexpr int kRowStep = 32 / kGroups, kIter = kTUnit / kRowStep;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  __shared__ TBars s;
  unsigned char* kbuf = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* vbuf = kbuf + 2 * kTile;
  unsigned char* qbuf = vbuf + 2 * kTile;       // [D / 64 halves][128 rows][128 B], as a K tile
  unsigned char* ring = qbuf + kTile;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int act = (a.M + 31) / 32;             // softmax warps with rows
  if (threadIdx.x == 0) {
    for (int i = 0; i < kTRing; ++i) {
      mbar_init(&s.raw_full[i], 1);
      mbar_init(&s.raw_empty[i], 2 * kTUnits);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.kfull[i], kTUnits);
      mbar_init(&s.kempty[i], 1);
      mbar_init(&s.vfull[i], kTUnits);
      mbar_init(&s.vempty[i], 1);
      mbar_init(&s.drain[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.s_free[i], act);
      mbar_init(&s.p_full[2 * i], act);
      mbar_init(&s.p_full[2 * i + 1], act);
      mbar_init(&s.p_free[i], 1);
    }
    mbar_init(&s.q_full, act);
    mbar_init(&s.o_full, 1);
    mbar_init(&s.h_done, 1);
    mbar_init(&s.o_free, 2 * act);
    for (int i = 0; i < 4; ++i) {
      s.turn[i] = 0;
      mbar_init(&s.joined[i], 2);
    }
    s.abort = 0;
    for (int i = 0; i < kNanSlots * 8; ++i) s.nan_at[i >> 3][i & 7] = kVerNone;
    fence_mbar_init();
  }
  if (warp == kTQkWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s.tmem_base)),
                 "r"(kTCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  grid_dependency_wait();
  allow_dependent_launch();

  const bool idle = warp < kTQkWarp && (warp & 3) >= act;  // a softmax warp without rows
  if (warp >= kTConvWarp || idle) {
    // ---------------------------------------------------------------- conversion
    // Every second of them takes keys, the others values. The values' buffers wait for the
    // weights' use of them, which must not hold up the next scores' keys; and a barrier's parity
    // names a phase only while the one before is known to be complete and the one behind cannot
    // be: a warp's tasks of one kind lie at most two chunks apart (at most 2 kTUnits warps), and
    // the products of a chunk wait for its tasks.
    const int spare = kTThreads / 32 - kTConvWarp;
    const int index = idle ? spare + ((warp & 3) - act) * 2 + (warp >> 2) : warp - kTConvWarp;
    const int v = index & 1, me = index >> 1;
    const int n_conv = min((spare + 2 * (4 - act) + 1 - v) / 2, 2 * kTUnits);
    uint64_t* const empty = v ? s.vempty : s.kempty;
    uint64_t* const full = v ? s.vfull : s.kfull;
    unsigned char* const buf = v ? vbuf : kbuf;
    const int r = lane / kGroups, g = lane % kGroups;  // this thread's row (of kRowStep) and group
    const int ps = min(a.page_size, kVerChunk), pshift = min(a.page_shift, 7);  // rows per block of a stage
    VerCursor cur = ver_begin(a, blockIdx.x);
    VerPiece p;
    // next task: unit `task` of the chunk; chunks of the piece from that one on; its first position
    // in the piece; its sequence's rows from there on
    int task = me, chunk = 0, left = 0, piece = -1, rel = 0;
    int64_t held = 0;
    // the thread's 16 codes of a row as two 16-byte pieces of the tile
    auto put = [&](unsigned char* line0, const uint2& w, uint32_t scale) {
      const uint32_t s2 = e4m3x2_to_half2(uint16_t(scale * 0x101u));
      uint32_t h[8];
      e2m1x8_to_half2(w.x, h);
      e2m1x8_to_half2(w.y, h + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = hmul2(h[j], s2);
      *reinterpret_cast<uint4*>(line0) = make_uint4(h[0], h[1], h[2], h[3]);
      // (D = 64: pieces 2 g and 2 g + 1 of the row, whose places differ in the lowest bit)
      unsigned char* second = D == 128 ? line0 + kHalf
                                       : reinterpret_cast<unsigned char*>(reinterpret_cast<uintptr_t>(line0) ^ 16);
      *reinterpret_cast<uint4*>(second) = make_uint4(h[4], h[5], h[6], h[7]);
    };
    // the first piece's place in row r of a task; 8 rows on the swizzle repeats
    constexpr int kPlaces = kRowStep < 8 ? 8 / kRowStep : 1;
    int place[kPlaces];
#pragma unroll
    for (int i = 0; i < kPlaces; ++i) {
      const int row = r + i * kRowStep;
      place[i] = row * 128 + (((D == 128 ? g : 2 * g) ^ (row & 7)) << 4);
    }
    while (me < n_conv) {
      if (left == 0) {
        if (!ver_next(a, cur, p)) break;
        left = int(p.c1 - p.c0);
        held = p.len - p.c0 * kVerChunk;
        rel = 0;
        ++piece;
      }
      if (task >= kTUnits) {
        task -= kTUnits;
        ++chunk;
        --left;
        held -= kVerChunk;
        rel += kVerChunk;
        continue;
      }
      const int row0 = task * kTUnit, st = chunk & 1, rs = chunk % kTRing;
      // codes and scales of the rows' two blocks of 16
      const unsigned char *codes[2], *scales[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int row = row0 + 16 * x;
        const unsigned char* blk = ring + rs * kRaw + (row >> pshift) * kv4_block_bytes(ps, D);
        const int off = (row & (ps - 1)) + v * ps + r;
        codes[x] = blk + off * (D / 2) + g * 8;
        scales[x] = blk + ps * D + off * kGroups + g;
      }
      // (the tile first: the products two chunks back are done, so the stage's phase before this
      // one, three chunks back, is complete, and the parity names this one)
      if (chunk >= 2 && !ver_wait_warp(s, &empty[st], uint32_t((chunk >> 1) - 1) & 1, a.err)) break;
      if (!ver_wait_warp(s, &s.raw_full[rs], uint32_t(chunk / kTRing) & 1, a.err)) break;
      uint2 w[kIter];
      uint32_t sc[kIter];
#pragma unroll
      for (int i = 0; i < kIter; ++i) {
        w[i] = *reinterpret_cast<const uint2*>(codes[i / (kIter / 2)] + (i % (kIter / 2)) * kRowStep * (D / 2));
        sc[i] = scales[i / (kIter / 2)][(i % (kIter / 2)) * kRowStep * kGroups];
      }
      if (v) {
        bool nan = false;
#pragma unroll
        for (int i = 0; i < kIter; ++i) nan |= nan_scale(sc[i]);
        // such a group takes part as zeros (ls_verify.cuh). Its slot is free: P V two chunks back
        // is done, so the output of the piece three chunks back is out
        if (nan) {
#pragma unroll
          for (int i = 0; i < kIter; ++i) {
            if (!nan_scale(sc[i])) continue;
            const int row = row0 + r + i * kRowStep;
            if (row < held) atomicMin(&s.nan_at[piece & (kNanSlots - 1)][g], rel + row);
            sc[i] = 0u;
          }
        }
      }
      unsigned char* tile = buf + st * kTile + row0 * 128;
#pragma unroll
      for (int i = 0; i < kIter; ++i) put(tile + place[i & (kPlaces - 1)] + (i / kPlaces) * (kPlaces * kRowStep * 128), w[i], sc[i]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&full[st]);
        mbar_arrive(&s.raw_empty[rs]);  // the task's codes are read
      }
      task += n_conv;
    }
  } else if (warp == kTLoadWarp) {
    // ---------------------------------------------------------------- producer
    ver_produce<D, kTRing>(a, s, s.raw_full, s.raw_empty, ring);
  } else if (warp == kTQkWarp || warp == kTPvWarp) {
    // ---------------------------------------------------------------- MMA issuers
    // the whole warp walks the chunks; one elected lane issues
    const bool qk = warp == kTQkWarp;
    VerCursor cur = ver_begin(a, blockIdx.x);
    VerPiece p;
    const uint64_t descq = sdesc(smem_u32(qbuf), 16, 1024);
    const uint64_t desc0 = qk ? sdesc(smem_u32(kbuf), 16, 1024) : sdesc(smem_u32(vbuf), kHalf, 1024);
    bool ok = true;
    int k = 0;
    for (int piece = 0; ok && ver_next(a, cur, p); ++piece) {
      const int n = int(p.c1 - p.c0);
      if (qk) {
        ok = ver_wait_warp(s, &s.q_full, uint32_t(piece) & 1, a.err);
      } else if (piece > 0) {
        ok = ver_wait_warp(s, &s.o_free, uint32_t(piece - 1) & 1, a.err);
        // the output of the piece before is out: its NaN positions make room for another's
        if (lane < 8) s.nan_at[(piece - 1) & (kNanSlots - 1)][lane] = kVerNone;
        __syncwarp();
      }
      for (int c = 0; c < n && ok; ++c, ++k) {
        const int st = k & 1;
        const uint32_t phase = uint32_t(k >> 1) & 1;
        const uint32_t sp = tmem + kVerChunk * st;
        const uint64_t desc = desc0 + uint32_t(st * kTile >> 4);
        if (!ver_wait_warp(s, qk ? &s.kfull[st] : &s.vfull[st], phase, a.err)) { ok = false; break; }
        if (qk) {
          if (k >= 2 && !ver_wait_warp(s, &s.s_free[st], phase ^ 1, a.err)) { ok = false; break; }
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t step = uint32_t(((kk >> 2) * kHalf + (kk & 3) * 32) >> 4);
              mma_bf16(sp, descq + step, desc + step, idesc_f16(kVerChunk, false), kk > 0);
            }
            mma_commit(&s.s_full[st]);
            mma_commit(&s.kempty[st]);
          }
          __syncwarp();
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!ver_wait_warp(s, &s.p_full[2 * st + h], phase, a.err)) { ok = false; break; }
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < kTSub / 16; ++kk)
                mma_bf16_ta(tmem + kTO, tmem + kTP + 64 * st + 32 * h + 8 * kk, desc + uint32_t((h * kTSub + kk * 16) * 128 >> 4),
                            idesc_f16(D, true), h == 1 || kk > 0 || c > 0);
              if (h == 0) {
                mma_commit(&s.h_done);
              } else {
                mma_commit(&s.p_free[st]);
                mma_commit(&s.vempty[st]);
                if (c == n - 1) mma_commit(&s.o_full);
              }
            }
            __syncwarp();
          }
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax and output
    const int grp = warp >> 2, wp = warp & 3;  // warp group: even or odd chunks; its 32 rows
    VerCursor cur = ver_begin(a, blockIdx.x);
    VerPiece p;
    const int m = wp * 32 + lane, i = m / a.grp, j = m - i * a.grp;
    const uint32_t trow = tmem + (uint32_t(32 * wp) << 16);
    int k = 0;
    bool ok = true;
    for (int piece = 0; ok && ver_next(a, cur, p); ++piece) {
      // the row's queries, scaled by a power of two, in the tiles' column order
      const bool real = m < a.M && i < p.rows;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) + (int64_t(p.b) * a.n_rows + i) * a.q_stride +
                                 (p.hm * a.grp + j) * D;
      float top = 0.f;
      if (real) {
#pragma unroll 4
        for (int e = 0; e < D; e += 8) {
          float x[8];
          Elem<__nv_bfloat16>::to_f32(ld_nc_v4(src + e), x);
#pragma unroll
          for (int u = 0; u < 8; ++u) top = fmaxf(top, fabsf(x[u]));
        }
      }
      int ex = int(__float_as_uint(top) >> 23) - 127;
      if (top == 0.f || ex > 127) ex = 0;
      if (ex < -126) ex = -126;
      const float f = ldexpf(a.scale_log2, ex);
      if (grp == 0) {
        const float down = ex == 127 ? 0x1p-127f : __uint_as_float(uint32_t(127 - ex) << 23);
#pragma unroll 2
        for (int c8 = 0; c8 < D / 8; ++c8) {
          float x[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) x[u] = 0.f;
          if (real) Elem<__nv_bfloat16>::to_f32(ld_nc_v4(src + dim_of<D>(8 * c8)), x);
          *reinterpret_cast<uint4*>(qbuf + (c8 >> 3) * kHalf + m * 128 + (((c8 & 7) ^ (m & 7)) << 4)) =
              make_uint4(ver_half2(x[0] * down, x[1] * down), ver_half2(x[2] * down, x[3] * down),
                         ver_half2(x[4] * down, x[5] * down), ver_half2(x[6] * down, x[7] * down));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.q_full);
      }

      float ref = -INFINITY, sum = 0.f;
      const int n = int(p.c1 - p.c0);
      // keys this row sees from the piece's first on
      const int64_t span = min(p.len, ver_limit(p, i)) - p.c0 * kVerChunk;
      const int limit = span > (int64_t(1) << 30) ? 1 << 30 : (span < 0 ? 0 : int(span));
      for (int c = 0; c < n && ok; ++c, ++k) {
        if ((k & 1) != grp) continue;
        const uint32_t phase = uint32_t(k >> 1) & 1;
        // the P columns' last use, and the scores
        ok = (k < 2 || ver_wait_warp(s, &s.p_free[grp], phase ^ 1, a.err)) && ver_wait_warp(s, &s.s_full[grp], phase, a.err);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const uint32_t sp = trow + kVerChunk * grp + kTSub * h;
          const int seen = limit - (c * kVerChunk + h * kTSub);
          const bool edge = __any_sync(0xffffffffu, seen < kTSub);
          const uint32_t pp = trow + kTP + 64 * grp + 32 * h;
          float part;
          auto weigh = [&]() {  // P: the 64 weights against ref; part: their sum
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              float x[32];
              uint32_t w[16];
              tmem_ld32(sp + 32 * b, x);
#pragma unroll
              for (int e = 0; e < 32; e += 2) fma2(x[e], x[e + 1], f, -ref);
              if (edge) {
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = 32 * b + e < seen ? x[e] : -INFINITY;
              }
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                x[e] = ver_exp2(x[e]);
                x[e + 1] = ver_exp2(x[e + 1]);
                add2(acc[e & 2], acc[(e & 2) + 1], x[e], x[e + 1]);
                w[e / 2] = ver_half2(x[e], x[e + 1]);
              }
              tmem_st16u(pp + 16 * b, w);
            }
            part = (acc[0] + acc[1]) + (acc[2] + acc[3]);
          };
          weigh();
          float now = ref;  // the row's reference so far
          if (h == 0 && c > 0) {
            if (!turn_wait(s, &s.turn[wp], uint32_t(k), a.err)) { ok = false; break; }
            now = s.ref[m];
          }
          const bool move = !(part <= kTMostSum) || now != ref;
          if (__any_sync(0xffffffffu, move)) {
            float mx = -INFINITY;
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
              float x[32];
              tmem_ld32(sp + 32 * b, x);
#pragma unroll
              for (int e = 0; e < 32; ++e) mx = fmaxf(mx, 32 * b + e < seen ? x[e] * f : -INFINITY);
            }
            const float next = move && mx > now + kTRoom ? mx - kTRoom : now;
            if (next != ref) sum *= ver_exp2(ref - next);
            ref = next;
            if ((c > 0 || h > 0) && __any_sync(0xffffffffu, next != now)) {
              // O holds the keys before these, once their P V has landed
              // (the chunk's before first: a parity names a phase only if the one before is complete)
              ok = k == 0 || ver_wait_warp(s, &s.p_free[grp ^ 1], uint32_t((k - 1) >> 1) & 1, a.err);
              if (ok && h == 1) ok = ver_wait_warp(s, &s.h_done, uint32_t(k) & 1, a.err);
              if (!ok) break;
              tc_fence_after();
              const float al = next == now ? 1.f : ver_exp2(now - next);
#pragma unroll 1
              for (int h2 = 0; h2 < D / 32; ++h2) {
                float ov[32];
                tmem_ld32(trow + kTO + 32 * h2, ov);
#pragma unroll
                for (int e = 0; e < 32; ++e) ov[e] *= al;
                tmem_st32(trow + kTO + 32 * h2, ov);
              }
            }
            // The first weights' stores are asynchronous too: they have to land before others go to
            // the same columns (a load's wait does not cover them).
            tmem_wait_st();
            weigh();
          }
          sum += part;
          if (h == 1) s.ref[m] = ref;
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&s.p_full[2 * grp + h]);
            if (h == 1) {
              turn_set(&s.turn[wp], uint32_t(k) + 1);
              mbar_arrive(&s.s_free[grp]);
            }
          }
        }
      }
      if (!ok) break;
      // both warps' sums of the row; the larger reference is O's
      s.state[piece & 1][grp][m] = make_float2(sum, ref);
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.joined[wp]);
      if (!ver_wait_warp(s, &s.joined[wp], uint32_t(piece) & 1, a.err)) break;
      const float2 other = s.state[piece & 1][grp ^ 1][m];
      const float last = fmaxf(ref, other.y);
      sum = (ref == last ? sum : sum * ver_exp2(ref - last)) + (other.y == last ? other.x : other.x * ver_exp2(other.y - last));
      if (!ver_wait_warp(s, &s.o_full, uint32_t(piece) & 1, a.err)) break;
      tc_fence_after();
      const bool whole = p.c0 == 0 && p.c1 == p.n;
      const int64_t slot = ver_slot(blockIdx.x, p);
      const float inv = !whole ? 1.f : (sum != 0.f ? 1.f / sum : 0.f);
      const int64_t seen_keys = ver_limit(p, i) - p.c0 * kVerChunk;
#pragma unroll 1
      for (int h = grp * (D / 64); h < (grp + 1) * (D / 64); ++h) {  // half of the columns each
        float o[32];
        tmem_ld32(trow + kTO + 32 * h, o);
        if (real) {
#pragma unroll
          for (int c8 = 0; c8 < 4; ++c8) {
            const int d = dim_of<D>(32 * h + 8 * c8);
            const bool bad = s.nan_at[piece & (kNanSlots - 1)][d / kKv4Group] < seen_keys;
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = bad ? NAN : o[8 * c8 + u] * inv;
            if (!whole) {
              float4* dst = reinterpret_cast<float4*>(a.part_o + (slot * a.MR + m) * D + d);
              dst[0] = make_float4(v[0], v[1], v[2], v[3]);
              dst[1] = make_float4(v[4], v[5], v[6], v[7]);
            } else {
              const int64_t at = ver_out_at(a, p.b, i, p.hm * a.grp + j) + d;
              if (a.out_f32) {
                float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at);
                dst[0] = make_float4(v[0], v[1], v[2], v[3]);
                dst[1] = make_float4(v[4], v[5], v[6], v[7]);
              } else {
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at) = Elem<__nv_bfloat16>::from_f32(v);
              }
            }
          }
        }
      }
      if (!whole && real && grp == 0) {
        a.part_ml[(slot * a.MR + m) * 2] = last;
        a.part_ml[(slot * a.MR + m) * 2 + 1] = sum;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.o_free);
    }
  }

  __syncthreads();
  if ((warp == kTQkWarp || warp == kTPvWarp) && s.abort) {  // the MMAs issued so far, before TMEM is freed
    if (elect_one()) {
      mma_commit(&s.drain[warp - kTQkWarp]);
      mbar_wait_bounded(&s.drain[warp - kTQkWarp], 0, kWaitLimit);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kTQkWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTCols) : "memory");
  }
}

template <int D>
cudaError_t launch_tc(const VerArgs& a, cudaStream_t stream) {
  constexpr int smem = 5 * kVerChunk * D * 2 + kTRing * kVerChunk * (D + D / 8) + 1024;
  const cudaError_t e = cudaFuncSetAttribute(verify_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_overlapped(verify_tc_kernel<D>, a.G, kTThreads, smem, stream, a);
}

}  // namespace

cudaError_t launch_verify_tc(const VerArgs& a, cudaStream_t stream) {
  return a.D == 128 ? launch_tc<128>(a, stream) : launch_tc<64>(a, stream);
}

}  // namespace ls
