// The target's verification attention over the 4-bit paged cache (ls_verify_attend_kv4;
// Figure 2 caption (a): the target verifies the proposed block), the CUDA-core kernel and the
// kernel that joins the pieces of cut tiles.
//   o[i] = sum_t softmax_t(scale q[i] . k[t]) v[t],  t = 0 .. len - rows + i
// One pass with the running maximum and sum: o, l and the reference r (log2 units) satisfy
// o = sum_t 2^(x_t - r) v_t, l = sum_t 2^(x_t - r); joining pieces adds them after scaling
// each by 2^(r_piece - max r).
#include "ls_verify.cuh"

namespace ls {

cudaError_t launch_verify_mma(const VerArgs& a, cudaStream_t stream);
cudaError_t launch_verify_tc(const VerArgs& a, cudaStream_t stream);

namespace {

constexpr int kVThreads = 128;

// CUDA-core kernel (fp32 states, and bf16 ones with LS_FLAG_FORCE_SIMT): thread t owns key t of
// a chunk for the scores of up to 8 query rows, then an output element (of D = 64, two
// threads with every second key each).
template <typename T, int D>
__global__ void __launch_bounds__(kVThreads) verify_simt_kernel(const VerArgs a) {
  using E = Elem<T>;
  constexpr int kKeySplit = kVThreads / D;  // threads per output element
  __shared__ __align__(16) float q_s[kSimtRows][D];
  __shared__ __align__(16) float s_s[kSimtRows][kVerChunk];  // scores, then weights
  __shared__ __align__(16) __half v_s[kVerChunk][D];         // exact: see ls_kv4.cuh
  __shared__ float ref_s[kSimtRows], sum_s[kSimtRows], alpha_s[kSimtRows];
  __shared__ int nan_s[D / kKv4Group];  // first chunk-relative position, from c0 on, of a NaN value group
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_dependency_wait();
  allow_dependent_launch();
  VerCursor cur = ver_begin(a, blockIdx.x);
  VerPiece p;
  while (ver_next(a, cur, p)) {
    const int mts = a.HM / a.Hkv;
    const int g = p.hm / mts, m0 = (p.hm - g * mts) * kSimtRows;
    const int nr = min(kSimtRows, a.M - m0);
    __syncthreads();  // the piece before is done with shared memory
    for (int x = tid * E::kVec; x < kSimtRows * D; x += kVThreads * E::kVec) {
      const int r = x / D, d = x - r * D, i = (m0 + r) / a.grp, j = (m0 + r) - i * a.grp;
      float f[E::kVec];
#pragma unroll
      for (int e = 0; e < E::kVec; ++e) f[e] = 0.f;
      if (r < nr && i < p.rows)
        E::to_f32(ld_nc_v4(static_cast<const T*>(a.q) + (int64_t(p.b) * a.n_rows + i) * a.q_stride +
                           (g * a.grp + j) * D + d), f);
#pragma unroll
      for (int e = 0; e < E::kVec; ++e) q_s[r][d + e] = f[e] * a.scale_log2;
    }
    if (tid < kSimtRows) {
      ref_s[tid] = -INFINITY;
      sum_s[tid] = 0.f;
    }
    if (tid < D / kKv4Group) nan_s[tid] = kVerNone;
    float o[kSimtRows];
#pragma unroll
    for (int r = 0; r < kSimtRows; ++r) o[r] = 0.f;
    const int od = tid % D, ok = tid / D;
    for (int64_t c = p.c0; c < p.c1; ++c) {
      __syncthreads();
      const int64_t pos = c * kVerChunk + tid;
      float acc[kSimtRows];
#pragma unroll
      for (int r = 0; r < kSimtRows; ++r) acc[r] = 0.f;
      if (pos < p.len) {
        const unsigned char* block = ver_block(a, p.b, pos >> a.page_shift, g);
        const Kv4Row row = kv4_row(const_cast<unsigned char*>(block), a.page_size, D, int(pos & (a.page_size - 1)));
#pragma unroll
        for (int d0 = 0; d0 < D; d0 += kKv4Group) {
          const uint2 w = *reinterpret_cast<const uint2*>(row.k_codes + d0 / 2);
          const float sc = e4m3_to_f32(row.k_scales[d0 / kKv4Group]);
          uint32_t h[8];
          e2m1x8_to_half2(w.x, h);
          e2m1x8_to_half2(w.y, h + 4);
          float k[kKv4Group];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 f = half2_to_f2(h[j]);
            k[2 * j] = f.x * sc;
            k[2 * j + 1] = f.y * sc;
          }
#pragma unroll
          for (int r = 0; r < kSimtRows; ++r) {
#pragma unroll
            for (int j = 0; j < kKv4Group; j += 4) {
              const float4 q4 = *reinterpret_cast<const float4*>(&q_s[r][d0 + j]);
              acc[r] = fmaf(q4.x, k[j], fmaf(q4.y, k[j + 1], fmaf(q4.z, k[j + 2], fmaf(q4.w, k[j + 3], acc[r]))));
            }
          }
          const uint2 wv = *reinterpret_cast<const uint2*>(row.v_codes + d0 / 2);
          const uint32_t sb = row.v_scales[d0 / kKv4Group];
          if (nan_scale(sb)) atomicMin(&nan_s[d0 / kKv4Group], int(pos - p.c0 * kVerChunk));
          const uint32_t s2 = nan_scale(sb) ? 0u : e4m3x2_to_half2(uint16_t(sb * 0x101u));
          e2m1x8_to_half2(wv.x, h);
          e2m1x8_to_half2(wv.y, h + 4);
#pragma unroll
          for (int j = 0; j < 8; ++j) *reinterpret_cast<uint32_t*>(&v_s[tid][d0 + 2 * j]) = hmul2(h[j], s2);
        }
      } else {
#pragma unroll
        for (int d0 = 0; d0 < D; d0 += 8) *reinterpret_cast<uint4*>(&v_s[tid][d0]) = make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int r = 0; r < kSimtRows; ++r) {
        const int i = (m0 + r) / a.grp;
        s_s[r][tid] = pos < ver_limit(p, i) && pos < p.len ? acc[r] : -INFINITY;
      }
      __syncthreads();
      for (int r = warp; r < kSimtRows; r += kVThreads / 32) {
        float x[kVerChunk / 32], top = -INFINITY;
#pragma unroll
        for (int u = 0; u < kVerChunk / 32; ++u) {
          x[u] = s_s[r][lane + 32 * u];
          top = fmaxf(top, x[u]);
        }
#pragma unroll
        for (int w = 16; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
        const float old = ref_s[r], ref = fmaxf(old, top);
        const float mu = ref == -INFINITY ? 0.f : ref;  // nothing seen yet: every weight is 0
        float sum = 0.f;
#pragma unroll
        for (int u = 0; u < kVerChunk / 32; ++u) {
          x[u] = exp2f(x[u] - mu);
          sum += x[u];
          s_s[r][lane + 32 * u] = x[u];
        }
#pragma unroll
        for (int w = 16; w; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
        __syncwarp();
        if (lane == 0) {
          const float al = exp2f(old - mu);
          ref_s[r] = ref;
          sum_s[r] = sum_s[r] * al + sum;
          alpha_s[r] = al;
        }
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < kSimtRows; ++r) o[r] *= alpha_s[r];
      for (int k0 = ok * 4; k0 < kVerChunk; k0 += 4 * kKeySplit) {
        float v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = __half2float(v_s[k0 + u][od]);
#pragma unroll
        for (int r = 0; r < kSimtRows; ++r) {
          const float4 w = *reinterpret_cast<const float4*>(&s_s[r][k0]);
          o[r] = fmaf(w.x, v[0], fmaf(w.y, v[1], fmaf(w.z, v[2], fmaf(w.w, v[3], o[r]))));
        }
      }
    }
    // the piece's rows: whole tiles to the output, pieces of cut ones to their slot
    __syncthreads();
    if constexpr (kKeySplit > 1) {  // the second threads' keys (one chunk's weights are free)
      if (ok > 0) {
#pragma unroll
        for (int r = 0; r < kSimtRows; ++r) s_s[r][od] = o[r];
      }
      __syncthreads();
      if (ok == 0) {
#pragma unroll
        for (int r = 0; r < kSimtRows; ++r) o[r] += s_s[r][od];
      }
    }
    const bool whole = p.c0 == 0 && p.c1 == p.n;
    const int slot = ver_slot(blockIdx.x, p);
    if (!whole && tid < kSimtRows) {
      a.part_ml[(int64_t(slot) * a.MR + tid) * 2] = ref_s[tid];
      a.part_ml[(int64_t(slot) * a.MR + tid) * 2 + 1] = sum_s[tid];
    }
    if (ok == 0) {
#pragma unroll
      for (int r = 0; r < kSimtRows; ++r) {
        const int i = (m0 + r) / a.grp, j = (m0 + r) - i * a.grp;
        if (r >= nr || i >= p.rows) continue;
        const int first_nan = nan_s[od / kKv4Group];
        if (first_nan != kVerNone && p.c0 * kVerChunk + first_nan < ver_limit(p, i)) o[r] = NAN;
        if (whole) {
          const float x = o[r] * (sum_s[r] != 0.f ? 1.f / sum_s[r] : 0.f);
          const int64_t at = ver_out_at(a, p.b, i, g * a.grp + j) + od;
          if (a.out_f32 || a.f32_in) Elem<float>::store1(a.out, at, x);
          else Elem<__nv_bfloat16>::store1(a.out, at, x);
        } else {
          a.part_o[(int64_t(slot) * a.MR + r) * D + od] = o[r];
        }
      }
    }
  }
}

// Joins the pieces of cut tiles, zeroes the rows of empty sequences and flags arguments
// outside their range. A warp per row (one CTA per tile and four rows): its lanes take the
// pieces' references and sums, then D / 32 output elements each, piece by piece in range order.
template <int D>
__global__ void __launch_bounds__(kVThreads) verify_join_kernel(const VerArgs a) {
  constexpr int kPer = D / 32;  // output elements per lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = int(blockIdx.x) / a.HM, hm = int(blockIdx.x) - b * a.HM;
  const int mts = a.HM / a.Hkv;
  const int g = hm / mts, m0 = (hm - g * mts) * a.MR;
  const int64_t n = ver_chunks(a, b);
  const int rows = ver_rows(a, b);
  if (hm == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    if (a.kv_len[b] != ver_len(a, b)) set_err(a.err, LS_DEVERR_PREFIX_LEN);
    if (a.rows && a.rows[b] != rows) set_err(a.err, LS_DEVERR_ROWS);
  }
  const int r = int(blockIdx.y) * (kVThreads / 32) + warp;
  const int i = (m0 + r) / a.grp, j = (m0 + r) - i * a.grp;
  bool mine = r < a.MR && m0 + r < a.M && i < rows;
  int c_first = 0, c_last = -1;
  if (mine && n > 0) {  // the CTAs whose ranges hold the tile's first and last chunk
    const int64_t T = ver_chunks_before(a, a.b) * a.HM, t0 = ver_chunks_before(a, b) * a.HM + hm * n;
    const int64_t G = T < a.G ? T : a.G;
    c_first = int(((t0 + 1) * G + T - 1) / T) - 1;
    c_last = int(((t0 + n) * G + T - 1) / T) - 1;
    mine = c_first != c_last;  // else the tile's CTA has written it
  }
  // Every thread waits, those without a row too: what is launched next waits for this grid only,
  // and this grid must not be complete before the one whose output it stands for.
  grid_dependency_wait();
  if (!mine) return;
  // the first piece starts its tile (an odd slot), the others start their CTAs' ranges
  auto at = [&](int c) { return (int64_t(2 * c) + (c == c_first ? 1 : 0)) * a.MR + r; };
  float o[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) o[e] = 0.f;
  float top = -INFINITY;
  for (int c = c_first + lane; c <= c_last; c += 32) top = fmaxf(top, a.part_ml[at(c) * 2]);
#pragma unroll
  for (int w = 16; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
  const float mu = top == -INFINITY ? 0.f : top;
  float sum = 0.f;
  for (int c0 = c_first; c0 <= c_last; c0 += 32) {
    float w = 0.f;
    if (c0 + lane <= c_last) {
      const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + at(c0 + lane) * 2);
      w = exp2f(ml.x - mu);
      sum = fmaf(w, ml.y, sum);
    }
    // kBatch pieces' outputs are loaded together (past the last: that one again, with weight 0)
    constexpr int kBatch = 8;
    const int cn = min(32, c_last - c0 + 1);
    for (int u0 = 0; u0 < cn; u0 += kBatch) {
      float x[kBatch][kPer];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const float* src = a.part_o + at(c0 + min(u0 + u, cn - 1)) * D + lane * kPer;
#pragma unroll
        for (int e = 0; e < kPer; e += 2) {
          const float2 y = __ldcg(reinterpret_cast<const float2*>(src + e));
          x[u][e] = y.x;
          x[u][e + 1] = y.y;
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const float wu = __shfl_sync(0xffffffffu, w, (u0 + u) & 31);
        if (u0 + u < cn) {
#pragma unroll
          for (int e = 0; e < kPer; ++e) o[e] = fmaf(wu, x[u][e], o[e]);
        }
      }
    }
  }
#pragma unroll
  for (int w = 16; w; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll
  for (int e = 0; e < kPer; ++e) o[e] *= inv;
  ver_store<kPer>(a, ver_out_at(a, b, i, g * a.grp + j) + lane * kPer, o);
}

enum VerKernel { kVerSimt, kVerMma, kVerTc };
struct VerShape {
  VerKernel kernel;
  int MR, ctas;  // rows per tile, CTAs per SM
};
VerShape ver_shape(const ls_config& c, int n_rows) {
  const int M = n_rows * (c.n_q_heads / c.n_kv_heads);
  if (c.dtype == LS_BF16 && !(c.flags & LS_FLAG_FORCE_SIMT)) {
    if (M <= kMmaMostRows) return {kVerMma, (M + 7) / 8 * 8, mma_ctas(M)};
    if (M <= kTcRows) return {kVerTc, kTcRows, 1};
  }
  return {kVerSimt, kSimtRows, kSimtCtas};
}

}  // namespace

size_t verify_workspace_bytes(const ls_config& c, int n_rows) {
  const VerShape v = ver_shape(c, n_rows);
  return size_t(2) * kVerMaxSms * v.ctas * v.MR * (size_t(c.head_dim) + 2) * 4;
}

cudaError_t launch_verify(const Dev& p, const ls_config& c, const ls_paged_kv4& kv, int layer, const void* q,
                          int64_t q_stride, int n_rows, const int32_t* rows, const int64_t* kv_len, float scale,
                          void* out, void* ws, int sms, cudaStream_t stream) {
  const int grp = p.Hq / p.Hkv;
  const VerShape v = ver_shape(c, n_rows);
  VerArgs a{};
  a.base = static_cast<const unsigned char*>(kv.layers[layer]);
  a.page_stride = kv.page_stride;
  a.num_pages = kv.num_pages;
  a.table = kv.block_table;
  a.max_blocks = kv.max_blocks;
  a.page_size = kv.page_size;
  while ((1 << a.page_shift) < kv.page_size) ++a.page_shift;
  a.q = q;
  a.q_stride = q_stride;
  a.n_rows = n_rows;
  a.rows = rows;
  a.kv_len = kv_len;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.out = out;
  a.b = p.b;
  a.Hkv = p.Hkv;
  a.Hq = p.Hq;
  a.grp = grp;
  a.D = p.D;
  a.M = n_rows * grp;
  a.MR = v.MR;
  a.HM = p.Hkv * ((a.M + v.MR - 1) / v.MR);
  a.G = (sms < kVerMaxSms ? sms : kVerMaxSms) * v.ctas;
  a.out_f32 = p.out_f32;
  a.f32_in = p.dtype == LS_F32;
  a.err = p.err;
  a.part_o = static_cast<float*>(ws);
  a.part_ml = a.part_o + int64_t(2) * a.G * v.MR * p.D;
  if (int64_t(p.b) * a.HM > INT32_MAX) return cudaErrorNotSupported;
  cudaError_t e;
  if (v.kernel == kVerMma) {
    e = launch_verify_mma(a, stream);
  } else if (v.kernel == kVerTc) {
    e = launch_verify_tc(a, stream);
  } else if (p.dtype == LS_F32) {
    e = p.D == 128 ? launch_overlapped(verify_simt_kernel<float, 128>, a.G, kVThreads, 0, stream, a)
                   : launch_overlapped(verify_simt_kernel<float, 64>, a.G, kVThreads, 0, stream, a);
  } else {
    e = p.D == 128 ? launch_overlapped(verify_simt_kernel<__nv_bfloat16, 128>, a.G, kVThreads, 0, stream, a)
                   : launch_overlapped(verify_simt_kernel<__nv_bfloat16, 64>, a.G, kVThreads, 0, stream, a);
  }
  if (e != cudaSuccess) return e;
  const dim3 grid(p.b * a.HM, ((a.M < v.MR ? a.M : v.MR) + kVThreads / 32 - 1) / (kVThreads / 32));
  return p.D == 128 ? launch_overlapped(verify_join_kernel<128>, grid, kVThreads, 0, stream, a)
                    : launch_overlapped(verify_join_kernel<64>, grid, kVThreads, 0, stream, a);
}

}  // namespace ls
