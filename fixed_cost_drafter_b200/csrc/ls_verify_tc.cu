// ls_verify_attend_kv4 for many query rows per KV head (a verification pass's B + 1 rows of a
// GQA group) of bf16 states, on the 5th-generation tensor cores.
//
// What bounds it: at 68 rows the two products (128 rows x 128 keys x D each, tcgen05 f16) take
// about as long as the bytes of the cache take to arrive, and the operands have to be made
// first: shared memory carries every fp16 operand twice (written by the conversion, read by
// the MMA). So nothing else goes through shared memory: codes come from global memory straight
// into the converting threads' registers, two chunks ahead, and Q and the weights P are the
// MMAs' A operands in TMEM.
//
// One CTA per SM, 14 warps; the roles meet at mbarriers:
//   warps 4-11  conversion: warp w takes 16 rows of each 128-key chunk, a thread 16 codes (one
//               scale group) at a time; K and V tiles in the 128-byte swizzle, two buffers
//               each. A group's two 16-byte pieces go to different 64-column halves (D = 128),
//               so that eight threads fill a whole 128-byte row; Q and the output columns
//               follow the same order.
//   warp 12     S = Q K^T of a chunk into one of two 128-column buffers (8 MMAs of N = 128: an
//               MMA costs its issuing thread about 80 cycles whatever its N)
//   warps 0-3   softmax, a thread per query row, 64 keys at a time: weights 2^(x - r) in fp16,
//               written over S. The reference r only moves when 64 weights sum to more than
//               2^15 (fp16 holds up to 65504); it is then the maximum less 8, as in
//               ls_verify_mma.cu, and the row of O is scaled in TMEM. The sum is needed anyway:
//               the check costs no maximum.
//   warp 13     O += P V, 64 keys at a time
// TMEM columns: S / P 0-255, O 256-383, Q 384-447.
// Rounding, exactness of the held values and NaN groups: as in ls_verify_mma.cu.
#include "ls_verify.cuh"
#include "ls_tc.cuh"

namespace ls {

namespace {

constexpr int kTThreads = 448;
constexpr int kTConv = 8;          // conversion warps
constexpr int kTSub = 64;          // keys the softmax takes at a time
constexpr uint32_t kTCols = 512, kTO = 256, kTQ = 384;
constexpr float kTRoom = 8.f;
constexpr float kTMostSum = 32768.f;
constexpr int kNanSlots = 4;       // pieces whose NaN positions are kept (conversion runs at most 2 ahead)

struct TBars {
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2];
  uint64_t s_full[2], p_full[4], p_free[2];  // p_full: [buffer][half]
  uint64_t h_done;  // the first half's P V
  uint64_t q_full, o_full, o_free, drain[2];
  uint32_t tmem_base, abort;
  int nan_at[kNanSlots][8];
};

__device__ inline bool twait(TBars& s, uint64_t* bar, uint32_t parity, int32_t* err) {
#pragma unroll 1
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 1023) == 1023 && *reinterpret_cast<volatile uint32_t*>(&s.abort)) return false;
  }
  set_err(err, LS_DEVERR_WAIT_TIMEOUT);
  *reinterpret_cast<volatile uint32_t*>(&s.abort) = 1;
  return false;
}
__device__ inline bool twait_warp(TBars& s, uint64_t* bar, uint32_t parity, int32_t* err) {
  return __all_sync(0xffffffffu, twait(s, bar, parity, err));
}

// kind::f16 with fp16 A/B, fp32 D
constexpr uint32_t idesc_f16(int n, bool b_mn_major) {
  return (1u << 4) | (uint32_t(b_mn_major) << 16) | (uint32_t(n >> 3) << 17) | (uint32_t(128 >> 4) << 24);
}

__device__ inline bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

__device__ inline void tmem_ld64(uint32_t taddr, float (&v)[64]) {
  uint32_t r[64];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[32 * h + 0]), "=r"(r[32 * h + 1]), "=r"(r[32 * h + 2]), "=r"(r[32 * h + 3]), "=r"(r[32 * h + 4]),
          "=r"(r[32 * h + 5]), "=r"(r[32 * h + 6]), "=r"(r[32 * h + 7]), "=r"(r[32 * h + 8]), "=r"(r[32 * h + 9]),
          "=r"(r[32 * h + 10]), "=r"(r[32 * h + 11]), "=r"(r[32 * h + 12]), "=r"(r[32 * h + 13]), "=r"(r[32 * h + 14]),
          "=r"(r[32 * h + 15]), "=r"(r[32 * h + 16]), "=r"(r[32 * h + 17]), "=r"(r[32 * h + 18]), "=r"(r[32 * h + 19]),
          "=r"(r[32 * h + 20]), "=r"(r[32 * h + 21]), "=r"(r[32 * h + 22]), "=r"(r[32 * h + 23]), "=r"(r[32 * h + 24]),
          "=r"(r[32 * h + 25]), "=r"(r[32 * h + 26]), "=r"(r[32 * h + 27]), "=r"(r[32 * h + 28]), "=r"(r[32 * h + 29]),
          "=r"(r[32 * h + 30]), "=r"(r[32 * h + 31])
        : "r"(taddr + 32 * h));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ inline void tmem_st32u(uint32_t taddr, const uint32_t* v) {
  tmem_st32(taddr, reinterpret_cast<const float*>(v));
}

__device__ inline float ex2a(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
__device__ inline uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Column position n of the K / V tiles holds dim dim_of(n): see the conversion.
template <int D>
__device__ constexpr int dim_of(int n) {
  return D == 128 ? 16 * ((n & 63) >> 3) + 8 * (n >> 6) + (n & 7) : n;
}

template <int D>
__global__ void __launch_bounds__(kTThreads, 1) verify_tc_kernel(const VerArgs a) {
  constexpr int kTile = kVerChunk * D * 2;     // one K or V buffer
  constexpr int kHalf = kVerChunk * 128;       // 64 columns of it
  constexpr int kGroups = D / kKv4Group;       // threads per row in the conversion
  constexpr int kRowStep = 32 / kGroups, kIter = 16 / kRowStep;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  __shared__ TBars s;
  unsigned char* kbuf = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* vbuf = kbuf + 2 * kTile;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int act = (a.M + 31) / 32;             // softmax warps with rows
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.kfull[i], kTConv);
      mbar_init(&s.kempty[i], 1);
      mbar_init(&s.vfull[i], kTConv);
      mbar_init(&s.vempty[i], 1);
      mbar_init(&s.drain[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.p_full[2 * i], 32 * act);
      mbar_init(&s.p_full[2 * i + 1], 32 * act);
      mbar_init(&s.p_free[i], 1);
    }
    mbar_init(&s.q_full, 32 * act);
    mbar_init(&s.o_full, 1);
    mbar_init(&s.h_done, 1);
    mbar_init(&s.o_free, 32 * act);
    s.abort = 0;
    for (int i = 0; i < kNanSlots * 8; ++i) s.nan_at[i >> 3][i & 7] = kVerNone;
    fence_mbar_init();
  }
  if (warp == 12) {
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

  if (warp >= 4 && warp < 12) {
    // ---------------------------------------------------------------- conversion
    const int cw = warp - 4, row0 = cw * 16;
    const int r = lane / kGroups, g = lane % kGroups;  // this thread's row (of kRowStep) and group
    const int ps = a.page_size;
    VerCursor cur = ver_begin(a, blockIdx.x);
    const int total = int(cur.left);  // chunks of this CTA
    // The lookup walks ahead of the conversion: the page of a chunk is looked up three chunks
    // ahead, its codes are loaded two ahead.
    VerPiece p;
    int64_t pos = 0;   // of this warp's 16 rows in the chunk looked up next
    int left = 0, piece = -1, rel = 0;
    int32_t entry = 0;
    auto look_up = [&]() {
      if (left == 0) {
        if (!ver_next(a, cur, p)) return;
        left = int(p.c1 - p.c0);
        pos = p.c0 * kVerChunk + row0;
        rel = row0;
        ++piece;
      }
      entry = pos < p.len ? __ldg(a.table + int64_t(p.b) * a.max_blocks + (pos >> a.page_shift)) : 0;
    };
    struct Rows {  // a chunk's 16 rows of this warp: codes and scales in flight
      uint2 w[2][kIter];
      uint32_t sc[2][kIter];
      int held, rel, piece;  // rows below the sequence's length, position in the piece, piece
    };
    Rows rows[2];
    const unsigned char* src = nullptr;  // the chunk whose rows are loaded next: its keys' codes
    int to_scales = 0;
    const int code_at = r * (D / 2) + g * 8, scale_at = r * kGroups + g;
    // the chunk looked up becomes the next to load, and the one behind it is looked up
    auto resolve = [&](Rows& q) {
      src = nullptr;
      q.held = 0;
      if (left > 0) {
        if (pos < p.len) {
          int64_t page = entry;
          if (page < 0 || page >= a.num_pages) {
            set_err(a.err, LS_DEVERR_PAGE);
            page = 0;
          }
          const int off = int(pos) & (ps - 1);
          src = a.base + page * a.page_stride + int64_t(p.hm) * kv4_block_bytes(ps, D) + off * (D / 2);
          to_scales = ps * D + off * (D / kKv4Group) - off * (D / 2);
          q.held = p.len - pos < 16 ? int(p.len - pos) : 16;
        }
        q.rel = rel;
        q.piece = piece & (kNanSlots - 1);
        pos += kVerChunk;
        rel += kVerChunk;
        --left;
      }
      look_up();
    };
    auto load = [&](Rows& q, int v) {
      const unsigned char* c = src + v * ps * (D / 2) + code_at;
      const unsigned char* sp = src + to_scales + v * ps * (D / kKv4Group) + scale_at;
#pragma unroll
      for (int i = 0; i < kIter; ++i) {
        q.w[v][i] = make_uint2(0u, 0u);
        q.sc[v][i] = 0u;
        if (src) {
          asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                       : "=r"(q.w[v][i].x), "=r"(q.w[v][i].y)
                       : "l"(c + i * kRowStep * (D / 2)));
          asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(q.sc[v][i]) : "l"(sp + i * kRowStep * kGroups));
        }
      }
    };
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
    // the first piece's place in the thread's rows: row0 + r + i kRowStep; 8 rows apart the
    // swizzle repeats
    int place[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int row = row0 + r + i * kRowStep;
      place[i] = row * 128 + (((D == 128 ? g : 2 * g) ^ (row & 7)) << 4);
    }
    look_up();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      resolve(rows[i]);
      load(rows[i], 0);
      load(rows[i], 1);
    }
    bool ok = true;
    for (int k0 = 0; k0 < total && ok; k0 += 2) {
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        const int k = k0 + st;
        if (k >= total) break;
        Rows& q = rows[st];
        const int held = q.held, at = q.rel, slot = q.piece;
        resolve(q);  // chunk k + 2
        if (k >= 2 && !twait_warp(s, &s.kempty[st], uint32_t((k >> 1) - 1) & 1, a.err)) { ok = false; break; }
#pragma unroll
        for (int i = 0; i < kIter; ++i) put(kbuf + st * kTile + place[i], q.w[0][i], q.sc[0][i]);
        load(q, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.kfull[st]);
        bool nan = false;
#pragma unroll
        for (int i = 0; i < kIter; ++i) nan |= nan_scale(q.sc[1][i]);
        if (nan) {  // such a group takes part as zeros (ls_verify.cuh)
#pragma unroll
          for (int i = 0; i < kIter; ++i) {
            if (!nan_scale(q.sc[1][i])) continue;
            if (r + i * kRowStep < held) atomicMin(&s.nan_at[slot][g], at + r + i * kRowStep);
            q.sc[1][i] = 0u;
          }
        }
        if (k >= 2 && !twait_warp(s, &s.vempty[st], uint32_t((k >> 1) - 1) & 1, a.err)) { ok = false; break; }
#pragma unroll
        for (int i = 0; i < kIter; ++i) put(vbuf + st * kTile + place[i], q.w[1][i], q.sc[1][i]);
        load(q, 1);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.vfull[st]);
      }
    }
  } else if (warp == 12 || warp == 13) {
    // ---------------------------------------------------------------- MMA issuers
    // the whole warp walks the chunks; one elected lane issues
    const bool qk = warp == 12;
    VerCursor cur = ver_begin(a, blockIdx.x);
    VerPiece p;
    const uint64_t desc0 = qk ? sdesc(smem_u32(kbuf), 16, 1024) : sdesc(smem_u32(vbuf), kHalf, 1024);
    bool ok = true;
    int k = 0;
    for (int piece = 0; ok && ver_next(a, cur, p); ++piece) {
      const int n = int(p.c1 - p.c0);
      if (qk) {
        ok = twait_warp(s, &s.q_full, uint32_t(piece) & 1, a.err);
      } else if (piece > 0) {
        ok = twait_warp(s, &s.o_free, uint32_t(piece - 1) & 1, a.err);
        // the output of the piece before is out: its NaN positions make room for another's
        if (lane < 8) s.nan_at[(piece - 1) & (kNanSlots - 1)][lane] = kVerNone;
        __syncwarp();
      }
      for (int c = 0; c < n && ok; ++c, ++k) {
        const int st = k & 1;
        const uint32_t phase = uint32_t(k >> 1) & 1;
        const uint32_t sp = tmem + kVerChunk * st;
        const uint64_t desc = desc0 + uint32_t(st * kTile >> 4);
        if (!twait_warp(s, qk ? &s.kfull[st] : &s.vfull[st], phase, a.err)) { ok = false; break; }
        if (qk) {
          if (k >= 2 && !twait_warp(s, &s.p_free[st], phase ^ 1, a.err)) { ok = false; break; }
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_bf16_ta(sp, tmem + kTQ + 8 * kk, desc + uint32_t(((kk >> 2) * kHalf + (kk & 3) * 32) >> 4),
                          idesc_f16(kVerChunk, false), kk > 0);
            mma_commit(&s.s_full[st]);
            mma_commit(&s.kempty[st]);
          }
          __syncwarp();
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!twait_warp(s, &s.p_full[2 * st + h], phase, a.err)) { ok = false; break; }
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < kTSub / 16; ++kk)
                mma_bf16_ta(tmem + kTO, sp + 32 * h + 8 * kk, desc + uint32_t((h * kTSub + kk * 16) * 128 >> 4),
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
  } else if (warp < act) {
    // ---------------------------------------------------------------- softmax and output
    VerCursor cur = ver_begin(a, blockIdx.x);
    VerPiece p;
    const int m = warp * 32 + lane, i = m / a.grp, j = m - i * a.grp;
    const uint32_t trow = tmem + (uint32_t(32 * warp) << 16);
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
      const float down = ex == 127 ? 0x1p-127f : __uint_as_float(uint32_t(127 - ex) << 23);
      const float f = ldexpf(a.scale_log2, ex);
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        uint32_t w[32];
#pragma unroll
        for (int c8 = 0; c8 < 8; ++c8) {
          float x[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) x[u] = 0.f;
          if (real) Elem<__nv_bfloat16>::to_f32(ld_nc_v4(src + dim_of<D>(64 * h + 8 * c8)), x);
#pragma unroll
          for (int u = 0; u < 4; ++u) w[4 * c8 + u] = pack_half2(x[2 * u] * down, x[2 * u + 1] * down);
        }
        tmem_st32u(trow + kTQ + 32 * h, w);
      }
      tc_fence_before();
      mbar_arrive(&s.q_full);

      float ref = -INFINITY, sum = 0.f;
      const int n = int(p.c1 - p.c0);
      // keys this row sees from the piece's first on
      const int64_t span = min(p.len, ver_limit(p, i)) - p.c0 * kVerChunk;
      const int limit = span > (int64_t(1) << 30) ? 1 << 30 : (span < 0 ? 0 : int(span));
      for (int c = 0; c < n && ok; ++c, ++k) {
        const int st = k & 1;
        const uint32_t phase = uint32_t(k >> 1) & 1;
        if (!twait_warp(s, &s.s_full[st], phase, a.err)) { ok = false; break; }
        tc_fence_after();
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const uint32_t sp = trow + kVerChunk * st + kTSub * h;
          const int seen = limit - (c * kVerChunk + h * kTSub);
          const bool edge = __any_sync(0xffffffffu, seen < kTSub);
          float x[64], part;
          auto weigh = [&]() {  // x: weights against ref; part: their sum
            const float mu = -ref;
            float acc[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = 0.f;
#pragma unroll
            for (int e = 0; e < 64; e += 2) fma2(x[e], x[e + 1], f, mu);
            if (edge) {
#pragma unroll
              for (int e = 0; e < 64; ++e) x[e] = e < seen ? x[e] : -INFINITY;
            }
#pragma unroll
            for (int e = 0; e < 64; e += 2) {
              x[e] = ex2a(x[e]);
              x[e + 1] = ex2a(x[e + 1]);
              add2(acc[e & 6], acc[(e & 6) + 1], x[e], x[e + 1]);
            }
            part = ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
          };
          tmem_ld64(sp, x);
          weigh();
          if (__any_sync(0xffffffffu, part > kTMostSum)) {
            tmem_ld64(sp, x);
            float mx = -INFINITY;
#pragma unroll
            for (int e = 0; e < 64; ++e) mx = fmaxf(mx, e < seen ? x[e] * f : -INFINITY);
            const float nref = part > kTMostSum ? fmaxf(ref, mx - kTRoom) : ref;
            const float al = nref == ref ? 1.f : ex2a(ref - nref);
            ref = nref;
            sum *= al;
            if (c > 0 || h > 0) {  // O holds the keys before these, once their P V has landed
              if (h == 0) {
                ok = twait_warp(s, &s.p_free[st ^ 1], uint32_t((k - 1) >> 1) & 1, a.err);
              } else {
                ok = twait_warp(s, &s.h_done, uint32_t(k) & 1, a.err);
              }
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
              for (int h2 = 0; h2 < D / 32; ++h2) {
                float ov[32];
                tmem_ld32(trow + kTO + 32 * h2, ov);
#pragma unroll
                for (int e = 0; e < 32; ++e) ov[e] *= al;
                tmem_st32(trow + kTO + 32 * h2, ov);
              }
            }
            weigh();
          }
          sum += part;
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) w[e] = pack_half2(x[2 * e], x[2 * e + 1]);
          tmem_st32u(trow + kVerChunk * st + 32 * h, w);
          tc_fence_before();
          mbar_arrive(&s.p_full[2 * st + h]);
        }
      }
      if (!ok || !twait_warp(s, &s.o_full, uint32_t(piece) & 1, a.err)) break;
      tc_fence_after();
      const bool whole = p.c0 == 0 && p.c1 == p.n;
      const int64_t slot = ver_slot(blockIdx.x, p);
      const float inv = !whole ? 1.f : (sum != 0.f ? 1.f / sum : 0.f);
      const int64_t seen_keys = ver_limit(p, i) - p.c0 * kVerChunk;
#pragma unroll 1
      for (int h = 0; h < D / 32; ++h) {
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
      if (!whole && real) {
        a.part_ml[(slot * a.MR + m) * 2] = ref;
        a.part_ml[(slot * a.MR + m) * 2 + 1] = sum;
      }
      tc_fence_before();
      mbar_arrive(&s.o_free);
    }
  }

  __syncthreads();
  if ((warp == 12 || warp == 13) && s.abort) {  // the MMAs issued so far, before TMEM is freed
    if (elect_one()) {
      mma_commit(&s.drain[warp - 12]);
      mbar_wait_bounded(&s.drain[warp - 12], 0, kWaitLimit);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTCols) : "memory");
  }
}

template <int D>
cudaError_t launch_tc(const VerArgs& a, cudaStream_t stream) {
  constexpr int smem = 4 * kVerChunk * D * 2 + 1024;
  const cudaError_t e = cudaFuncSetAttribute(verify_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return ver_launch(verify_tc_kernel<D>, a.G, kTThreads, smem, stream, a);
}

}  // namespace

cudaError_t launch_verify_tc(const VerArgs& a, cudaStream_t stream) {
  return a.D == 128 ? launch_tc<128>(a, stream) : launch_tc<64>(a, stream);
}

}  // namespace ls
