// ls_verify_attend_kv4 for few query rows per KV head (decoding, short blocks) of bf16 states.
//
// Measured: decoding 16 requests at 48K-64K tokens, 1.06 GB of cache: 230 to 238 us, 4.5 TB/s (69 % of
// the copy rate). The work is to turn 4-bit codes into fp16 MMA operands as fast as the bytes
// arrive: about 2200 warp instructions per 128 keys, half of them conversions and scalings, issued
// in 57 % of the cycles. No unit is full (ALU 52 %, DRAM 70 %); what holds a step is latency with few
// warps to cover it: 3.4 warps per sub-partition, and of the 6.0 cycles that a warp spends per
// instruction 1.5 wait for the result before it, 0.8 for other warps' turns, 0.7 for memory, 0.6 for a
// busy pipe. (Four CTAs per SM with two stages each, 96 registers: the same; five: 295 us.)
// The operands are made in registers, from shared
// memory that bulk copies fill (a page's block of one KV head is one contiguous copy), and
// never go back to shared memory: warp-level m16n8k16 products, whose M = 16 side is the
// cache (16 keys, then 16 output dimensions) and whose N = 8 side the query rows.
//   S^T[key][row] = K Q^T: A = 16 keys x 16 dims. The order of the dims within the product is
//     free, so thread t of a row's four takes D/4 consecutive dims: one wide load of codes.
//   O^T[dim][row] = V^T P^T: A = 16 dims x 16 keys. A register pairs two keys of one dim: the
//     codes of two rows are interleaved nibble by nibble before they are converted (two
//     logic operations for four pairs), and a row of the product is any dim: thread group g
//     takes dims g D/8 .. of its keys. P^T comes from S^T by 8x8 transposes in registers.
// A code times its scale is exact in fp16 (ls_kv4.cuh). Queries are scaled per row by a power
// of two to a largest element in [1, 2) and rounded to fp16 (exact for bf16 elements down to
// 2^-14 of the largest). Weights are rounded to fp16 against a reference r that only moves
// when a weight would pass 2^15: w = 2^(x - r), r = (maximum when it moved) - 8, so weights
// down to 2^-22 of the largest keep 11 bits.
// Warps take 32 keys of each 128-key chunk with a softmax state of their own, joined through
// shared memory at the end of a piece (ls_verify.cuh).
#include "ls_verify.cuh"
#include "ls_tc.cuh"

namespace ls {

namespace {

constexpr int kMWarps = 4;                      // consumer warps
constexpr int kMThreads = (kMWarps + 1) * 32;   // and a producer warp
constexpr int kMStages = 3;
constexpr float kMRoom = 8.f;    // log2 of the largest weight when the reference moves
constexpr float kMMost = 15.f;   // and the log2 at which it has to

__host__ __device__ constexpr int stage_bytes(int D) { return kVerChunk * (D + D / 8); }

template <int NT, int D>
struct MShared {
  uint64_t full[kMStages], empty[kMStages];
  uint32_t abort;
  int nan_at[D / kKv4Group];
  float ref[kMWarps][8 * NT], sum[kMWarps][8 * NT];
  alignas(16) float o[8 * NT][D + 4];  // written as float2
};


__device__ inline void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ inline uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ inline void consumers_meet() { asm volatile("bar.sync 1, %0;" ::"n"(kMWarps * 32) : "memory"); }

template <int NT, int D>
__global__ void __launch_bounds__(kMThreads) verify_mma_kernel(const VerArgs a) {
  constexpr int kSteps = D / 16;        // k16 steps of Q K^T; also registers pairs of Q per n-tile
  constexpr int kTiles = D / 16;        // 16-dim tiles of O
  constexpr int kWords = D / 32;        // 8-code words per thread and key of K
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ MShared<NT, D> s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ps = min(a.page_size, kVerChunk);  // rows per block in a stage
  const int pshift = min(a.page_shift, 7);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMStages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], kMWarps);
    }
    s.abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  grid_dependency_wait();
  allow_dependent_launch();
  if (warp == kMWarps) {
    ver_produce<D, kMStages>(a, s, s.full, s.empty, ring);
    return;
  }

  // ------------------------------------------------------------------ consumers
  VerCursor cur = ver_begin(a, blockIdx.x);
  VerPiece p;
  int k = 0;  // chunks so far: stage and phase
  const int g = lane >> 2, t = lane & 3;
  bool ok = true;
  while (ver_next(a, cur, p)) {
    // Q of the piece: rows n = 8 nt + g, dims t D/4 ..
    uint32_t q[NT][kSteps][2];
    float f[NT][2];  // logits (log2 units) per product, of rows 8 nt + 2 t, + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int m = nt * 8 + g, i = m / a.grp, j = m - i * a.grp;
      float x[D / 4];
      float top = 0.f;
      const bool real = m < a.M && i < p.rows;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) + (int64_t(p.b) * a.n_rows + i) * a.q_stride +
                                 (p.hm * a.grp + j) * D + t * (D / 4);
#pragma unroll
      for (int e = 0; e < D / 4; e += 8) {
        if (real) {
          Elem<__nv_bfloat16>::to_f32(ld_nc_v4(src + e), x + e);
        } else {
#pragma unroll
          for (int u = 0; u < 8; ++u) x[e + u] = 0.f;
        }
      }
#pragma unroll
      for (int e = 0; e < D / 4; ++e) top = fmaxf(top, fabsf(x[e]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // the power of two of the row's largest element
      int ex = int(__float_as_uint(top) >> 23) - 127;
      if (top == 0.f || ex > 127) ex = 0;
      if (ex < -126) ex = -126;
      const float down = ex == 127 ? 0x1p-127f : __uint_as_float(uint32_t(127 - ex) << 23);
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        q[nt][st][0] = ver_half2(x[4 * st] * down, x[4 * st + 1] * down);
        q[nt][st][1] = ver_half2(x[4 * st + 2] * down, x[4 * st + 3] * down);
      }
      const float up = ldexpf(a.scale_log2, ex);
      f[nt][0] = __shfl_sync(0xffffffffu, up, (2 * t) * 4);
      f[nt][1] = __shfl_sync(0xffffffffu, up, (2 * t + 1) * 4);
    }
    if (threadIdx.x < D / kKv4Group) s.nan_at[threadIdx.x] = kVerNone;
    consumers_meet();
    float o[NT][kTiles][4], ref[NT][2], sum[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      ref[nt][0] = ref[nt][1] = -INFINITY;
      sum[nt][0] = sum[nt][1] = 0.f;
#pragma unroll
      for (int j = 0; j < kTiles; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][j][e] = 0.f;
    }
    const int64_t full_seen = ver_limit(p, 0);  // keys every row sees

    for (int64_t c = p.c0; c < p.c1; ++c, ++k) {
      const int st = k % kMStages;
      if (ok && !ver_wait_warp(s, &s.full[st], uint32_t(k / kMStages) & 1, a.err)) ok = false;
      if (!ok) continue;
      const unsigned char* base = ring + st * stage_bytes(D);
      const bool edge = (c + 1) * kVerChunk > full_seen;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int key0 = warp * 32 + half * 16;
        const unsigned char* blk = base + (key0 >> pshift) * kv4_block_bytes(ps, D);
        const int off = key0 & (ps - 1);
        // ---- S^T of 16 keys
        float x[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.f;
        {
          const unsigned char* kc = blk + (off + g) * (D / 2) + t * (D / 8);
          const unsigned char* ks = blk + ps * D + (off + g) * (D / kKv4Group) + t * (D / 64);
          uint32_t w[2][kWords], sc[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {  // keys g and g + 8
            if constexpr (D == 128) {
              const uint4 v = *reinterpret_cast<const uint4*>(kc + r * 8 * (D / 2));
              w[r][0] = v.x; w[r][1] = v.y; w[r][2] = v.z; w[r][3] = v.w;
              sc[r] = e4m3x2_to_half2(*reinterpret_cast<const uint16_t*>(ks + r * 8 * (D / kKv4Group)));
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(kc + r * 8 * (D / 2));
              w[r][0] = v.x; w[r][1] = v.y;
              sc[r] = e4m3x2_to_half2(uint16_t(ks[r * 8 * (D / kKv4Group)]));
            }
          }
#pragma unroll
          for (int wi = 0; wi < kWords; ++wi) {  // 8 dims: two k-steps
            uint32_t h[2][4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint32_t s2 = __byte_perm(sc[r], 0, wi >= 2 ? 0x3232 : 0x1010);
              e2m1x8_to_half2(w[r][wi], h[r]);
#pragma unroll
              for (int e = 0; e < 4; ++e) h[r][e] = hmul2(h[r][e], s2);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint32_t av[4] = {h[0][2 * u], h[1][2 * u], h[0][2 * u + 1], h[1][2 * u + 1]};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_f16(x[nt], av, q[nt][2 * wi + u][0], q[nt][2 * wi + u][1]);
            }
          }
        }
        // ---- weights
        uint32_t pt[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          // x[e]: key g (e < 2) or g + 8, row 2 t + (e & 1)
          bool seen[4] = {true, true, true, true};
          if (edge) {
            const int64_t pos = c * kVerChunk + key0 + g;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              seen[e] = pos + (e >> 1) * 8 < min(p.len, ver_limit(p, (nt * 8 + 2 * t + (e & 1)) / a.grp));
          }
          float y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = seen[e] ? fmaf(x[nt][e], f[nt][e & 1], -ref[nt][e & 1]) : -INFINITY;
          const float top = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
          if (__any_sync(0xffffffffu, top > kMMost)) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float mx = fmaxf(seen[e] ? x[nt][e] * f[nt][e] : -INFINITY, seen[e + 2] ? x[nt][e + 2] * f[nt][e] : -INFINITY);
#pragma unroll
              for (int w = 4; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
              const float nref = fmaxf(ref[nt][e], mx - kMRoom);
              const float al = ref[nt][e] == nref ? 1.f : ver_exp2(ref[nt][e] - nref);
              ref[nt][e] = nref;
              sum[nt][e] *= al;
#pragma unroll
              for (int j = 0; j < kTiles; ++j) {
                o[nt][j][e] *= al;
                o[nt][j][e + 2] *= al;
              }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = seen[e] ? fmaf(x[nt][e], f[nt][e & 1], -ref[nt][e & 1]) : -INFINITY;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = ver_exp2(y[e]);
          sum[nt][0] += y[0] + y[2];
          sum[nt][1] += y[1] + y[3];
          pt[nt][0] = transpose8(ver_half2(y[0], y[1]));  // row g, keys 2 t, 2 t + 1
          pt[nt][1] = transpose8(ver_half2(y[2], y[3]));  // keys 2 t + 8, 2 t + 9
        }
        // ---- O^T += V^T P^T
        {
          const unsigned char* vc = blk + (ps + off + 2 * t) * (D / 2) + g * (D / 16);
          const unsigned char* vs = blk + ps * D + (ps + off + 2 * t) * (D / kKv4Group) + g * (D / 8) / kKv4Group;
          uint32_t w[4][kWords / 2], s2[2], bytes = 0;  // keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = (r >> 1) * 8 + (r & 1);
            if constexpr (D == 128) {
              const uint2 v = *reinterpret_cast<const uint2*>(vc + row * (D / 2));
              w[r][0] = v.x; w[r][1] = v.y;
            } else {
              w[r][0] = *reinterpret_cast<const uint32_t*>(vc + row * (D / 2));
            }
            bytes |= uint32_t(vs[row * (D / kKv4Group)]) << (8 * r);
          }
          const uint32_t nan = __vcmpeq4(bytes & 0x7f7f7f7fu, 0x7f7f7f7fu);
          if (nan) {  // such a group takes part as zeros (ls_verify.cuh)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int64_t pos = c * kVerChunk + key0 + 2 * t + (r >> 1) * 8 + (r & 1);
              if (((nan >> (8 * r)) & 1) && pos < p.len)
                atomicMin(&s.nan_at[g * (D / 8) / kKv4Group], int(pos - p.c0 * kVerChunk));
            }
            bytes &= ~nan;
          }
          s2[0] = e4m3x2_to_half2(uint16_t(bytes));
          s2[1] = e4m3x2_to_half2(uint16_t(bytes >> 16));
#pragma unroll
          for (int wi = 0; wi < kWords / 2; ++wi) {
            uint32_t ev[2][4], od[2][4];  // [key pair][dim pair]: dims 2 j and 2 j + 1 of two keys
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint32_t w0 = w[2 * r][wi], w1 = w[2 * r + 1][wi];
              e2m1x8_to_half2((w0 & 0x0f0f0f0fu) | ((w1 << 4) & 0xf0f0f0f0u), ev[r]);
              e2m1x8_to_half2(((w0 >> 4) & 0x0f0f0f0fu) | (w1 & 0xf0f0f0f0u), od[r]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t av[4] = {hmul2(ev[0][j], s2[0]), hmul2(od[0][j], s2[0]), hmul2(ev[1][j], s2[1]),
                                      hmul2(od[1][j], s2[1])};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_f16(o[nt][wi * 4 + j], av, pt[nt][0], pt[nt][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.empty[st]);
    }

    // ---- the warps' states joined, in warp order
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = sum[nt][e];
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
        if (g == 0) {
          s.ref[warp][nt * 8 + 2 * t + e] = ref[nt][e];
          s.sum[warp][nt * 8 + 2 * t + e] = x;
        }
      }
    consumers_meet();
#pragma unroll 1
    for (int w = 0; w < kMWarps; ++w) {
      if (w == warp) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int n = nt * 8 + 2 * t + e;
            float top = s.ref[0][n];
#pragma unroll
            for (int v = 1; v < kMWarps; ++v) top = fmaxf(top, s.ref[v][n]);
            const float al = ref[nt][e] == top ? 1.f : ver_exp2(ref[nt][e] - top);
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
              float2* dst = reinterpret_cast<float2*>(&s.o[n][g * (D / 8) + 2 * j]);
              float2 x = make_float2(o[nt][j][e] * al, o[nt][j][e + 2] * al);
              if (w > 0) {
                const float2 y = *dst;
                x.x += y.x;
                x.y += y.y;
              }
              *dst = x;
            }
          }
      }
      consumers_meet();
    }
    const bool whole = p.c0 == 0 && p.c1 == p.n;
    const int64_t slot = ver_slot(blockIdx.x, p);
    for (int n = warp; n < a.M; n += kMWarps) {  // a warp per row
      const int i = n / a.grp, j = n - i * a.grp;
      if (i >= p.rows) break;
      float top = s.ref[0][n], total = 0.f;
#pragma unroll
      for (int v = 1; v < kMWarps; ++v) top = fmaxf(top, s.ref[v][n]);
#pragma unroll
      for (int v = 0; v < kMWarps; ++v)
        total += s.ref[v][n] == top ? s.sum[v][n] : s.sum[v][n] * ver_exp2(s.ref[v][n] - top);
      constexpr int kPer = D / 32;
      float v[kPer];
      const int first_nan = s.nan_at[lane * kPer / kKv4Group];
      const bool bad = first_nan != kVerNone && p.c0 * kVerChunk + first_nan < ver_limit(p, i);
      const float inv = !whole ? 1.f : (total != 0.f ? 1.f / total : 0.f);
#pragma unroll
      for (int e = 0; e < kPer; ++e) v[e] = bad ? NAN : s.o[n][lane * kPer + e] * inv;
      if (whole) {
        ver_store<kPer>(a, ver_out_at(a, p.b, i, p.hm * a.grp + j) + lane * kPer, v);
      } else {
        float* dst = a.part_o + (slot * a.MR + n) * D + lane * kPer;
#pragma unroll
        for (int e = 0; e < kPer; e += 2) *reinterpret_cast<float2*>(dst + e) = make_float2(v[e], v[e + 1]);
        if (lane == 0) {
          a.part_ml[(slot * a.MR + n) * 2] = top;
          a.part_ml[(slot * a.MR + n) * 2 + 1] = total;
        }
      }
    }
    consumers_meet();  // shared memory is free for the next piece
  }
}

template <int NT, int D>
cudaError_t launch_mma(const VerArgs& a, cudaStream_t stream) {
  const int smem = kMStages * stage_bytes(D);
  const cudaError_t e = cudaFuncSetAttribute(verify_mma_kernel<NT, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_overlapped(verify_mma_kernel<NT, D>, a.G, kMThreads, smem, stream, a);
}

}  // namespace

cudaError_t launch_verify_mma(const VerArgs& a, cudaStream_t stream) {
  const int nt = a.MR / 8;
  if (a.D == 128) {
    if (nt == 1) return launch_mma<1, 128>(a, stream);
    if (nt == 2) return launch_mma<2, 128>(a, stream);
    return launch_mma<3, 128>(a, stream);
  }
  if (nt == 1) return launch_mma<1, 64>(a, stream);
  if (nt == 2) return launch_mma<2, 64>(a, stream);
  return launch_mma<3, 64>(a, stream);
}

}  // namespace ls
