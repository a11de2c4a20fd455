// Rows into and out of the 4-bit KV cache (ls_kv4_append, ls_kv4_read_rows): see ls_kv4.cuh
// for the format. Both kernels move each element once and are bound by those bytes: a thread
// takes the 16 bytes of a row's elements that make one full-width load or store (8 bf16 or 4 fp32
// elements of a key, and the value's), the 2 or 4 threads of a scale group share its maximum.
// 64K rows of 8 heads x 128 written (85 us) and read (70 us): 153 us together, 4.5 TB/s, 69 % of
// the copy rate (a thread per scale group with divisions: 200 us). fp32 rows: written 172 us (3.6 TB/s,
// a division per element), read 129 us (4.8 TB/s).
#include "ls_kv4.cuh"

namespace ls {

namespace {

constexpr int kKv4Threads = 256;  // at most: whole rows per CTA

struct Kv4Args {
  unsigned char* base;  // the layer's pages
  int64_t page_stride;
  int64_t num_slots;
  int32_t page_size, page_shift;
  const int64_t* slots;
  int64_t n_rows, row_stride;
  int32_t D, d_shift;
  int32_t per_row;  // threads per row: H * D elements, 16 bytes each
  int32_t per_cta;  // rows per CTA
  uint32_t per_row_inv;  // ceil(2^16 / per_row): exact for thread numbers below 256
  void* k;
  void* v;
  int32_t* err;
};

// The (page, head) block of a slot, or null (a slot outside the pool other than -1 is flagged).
__device__ inline unsigned char* kv4_block(const Kv4Args& a, int64_t slot, int head, int& off) {
  if (slot < 0 || slot >= a.num_slots) {
    if (slot != -1) set_err(a.err, LS_DEVERR_PAGE);
    return nullptr;
  }
  off = int(slot & (a.page_size - 1));
  return a.base + (slot >> a.page_shift) * a.page_stride + int64_t(head) * kv4_block_bytes(a.page_size, a.D);
}

__device__ inline uint32_t pack_e2m1(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\t"
      "cvt.u32.u8 %0, t;\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}
__device__ inline uint32_t to_e4m3(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xffu;
}

// x / s rounded enough for the nearest code with ties to even. A threshold t (half way between
// two values) times a divisor (a scale of 4 significant bits, or 6) has at most 7.
//   fp32 x: the rounded quotient lies on x's side of t, or is t where x is t s.
//   bf16 x: x (8 bits) is t s or differs from it by at least 2^-8 of it, so the product with a
//   reciprocal, off by at most 2^-21, becomes t or stays on x's side of it when it is rounded to
//   16 bits. (Divisions made the kernel issue-bound: 125 us.)
template <typename T> struct Ratio;
template <> struct Ratio<float> {
  float s;
  __device__ explicit Ratio(float d) : s(d) {}
  __device__ float operator()(float x) const { return __fdiv_rn(x, s); }
};
template <> struct Ratio<__nv_bfloat16> {
  float inv;
  __device__ explicit Ratio(float d) { asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(d)); }
  __device__ float operator()(float x) const { return __uint_as_float((__float_as_uint(x * inv) + 0x80u) & 0xffffff00u); }
};

// The largest magnitude of 16 bytes of elements; infinite if one is infinite or NaN.
template <typename T> __device__ inline float top_of(const uint4& v);
template <> __device__ inline float top_of<float>(const uint4& v) {
  // (magnitudes order as their bits do, infinities and NaN last)
  const uint32_t m = max(max(v.x & 0x7fffffffu, v.y & 0x7fffffffu), max(v.z & 0x7fffffffu, v.w & 0x7fffffffu));
  return m >= 0x7f800000u ? INFINITY : __uint_as_float(m);
}
template <> __device__ inline float top_of<__nv_bfloat16>(const uint4& v) {
  const uint32_t m2 = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
  const uint32_t m = max(m2 >> 16, m2 & 0xffffu);
  return m >= 0x7f80u ? INFINITY : __uint_as_float(m << 16);
}

// This thread's row, and its 16 bytes' first element in it; false where there is none (rows past
// the last, and the threads that fill the CTA's last warp).
__device__ inline bool kv4_place(const Kv4Args& a, int vec, int64_t& row, int& e) {
  const int in_cta = int(threadIdx.x * a.per_row_inv >> 16);  // threadIdx.x / per_row
  row = int64_t(blockIdx.x) * a.per_cta + in_cta;
  e = (int(threadIdx.x) - in_cta * a.per_row) * vec;
  return in_cta < a.per_cta && row < a.n_rows;
}

template <typename T>
__global__ void __launch_bounds__(kKv4Threads) kv4_append_kernel(const Kv4Args a) {
  using E = Elem<T>;
  grid_dependency_wait();
  allow_dependent_launch();
  constexpr int kVec = E::kVec, kLanes = kKv4Group / kVec;  // threads per scale group
  int64_t row;
  int e;
  const bool real = kv4_place(a, kVec, row, e);
  uint4 in[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  int64_t slot = -1;
  if (real) {
    in[0] = ld_nc_v4(static_cast<const T*>(a.k) + row * a.row_stride + e);
    in[1] = ld_nc_v4(static_cast<const T*>(a.v) + row * a.row_stride + e);
    slot = a.slots[row];
  }
  const int head = e >> a.d_shift, d = e & (a.D - 1);
  int off = 0;
  unsigned char* block = real ? kv4_block(a, slot, head, off) : nullptr;
  Kv4Row r{};
  if (block) r = kv4_row(block, a.page_size, a.D, off);
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    float top = top_of<T>(in[w]);
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool odd = top == INFINITY;  // an infinite or NaN element in the group
    const uint32_t sb = odd ? 0x7fu : to_e4m3(Ratio<T>(6.f)(top));
    const float s = odd ? 0.f : e4m3_to_f32(sb);
    uint32_t code = 0u;
    if (s > 0.f) {
      const Ratio<T> ratio(s);
      float x[kVec];
      E::to_f32(in[w], x);
#pragma unroll
      for (int j = 0; j < kVec; j += 2) code |= pack_e2m1(ratio(x[j]), ratio(x[j + 1])) << (4 * j);
    }
    if (block) {
      unsigned char* to = (w ? r.v_codes : r.k_codes) + d / 2;
      if constexpr (kVec == 8) *reinterpret_cast<uint32_t*>(to) = code;
      else *reinterpret_cast<uint16_t*>(to) = uint16_t(code);
      if (d % kKv4Group == 0) (w ? r.v_scales : r.k_scales)[d / kKv4Group] = static_cast<unsigned char>(sb);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kKv4Threads) kv4_read_kernel(const Kv4Args a) {
  using E = Elem<T>;
  grid_dependency_wait();
  allow_dependent_launch();
  constexpr int kVec = E::kVec;
  int64_t row;
  int e;
  if (!kv4_place(a, kVec, row, e)) return;
  const int head = e >> a.d_shift, d = e & (a.D - 1);
  int off;
  unsigned char* block = kv4_block(a, a.slots[row], head, off);
  if (!block) return;
  const Kv4Row r = kv4_row(block, a.page_size, a.D, off);
  uint32_t code[2], sb[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    // the word of the eight codes around d (fp32: its lower or upper half is this thread's)
    code[w] = *reinterpret_cast<const uint32_t*>((w ? r.v_codes : r.k_codes) + d / 8 * 4);
    sb[w] = (w ? r.v_scales : r.k_scales)[d / kKv4Group];
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const float s = e4m3_to_f32(sb[w]);
    uint32_t h[4];
    e2m1x8_to_half2(code[w], h);
    float x[kVec];
#pragma unroll
    for (int j = 0; j < kVec / 2; ++j) {
      const float2 f = half2_to_f2(kVec == 8 || !(d & 4) ? h[j] : h[j + 2]);
      x[2 * j] = f.x * s;
      x[2 * j + 1] = f.y * s;
    }
    *reinterpret_cast<uint4*>(static_cast<T*>(w ? a.v : a.k) + row * a.row_stride + e) = E::from_f32(x);
  }
}

Kv4Args kv4_args(const Dev& p, const ls_paged_kv4& kv, int layer, const int64_t* slots, int64_t n_rows, void* k, void* v,
                 int64_t row_stride) {
  Kv4Args a{};
  a.base = static_cast<unsigned char*>(kv.layers[layer]);
  a.page_stride = kv.page_stride;
  a.num_slots = kv.num_pages * kv.page_size;
  a.page_size = kv.page_size;
  while ((1 << a.page_shift) < kv.page_size) ++a.page_shift;
  a.slots = slots;
  a.n_rows = n_rows;
  a.row_stride = row_stride;
  a.D = p.D;
  a.d_shift = p.D == 128 ? 7 : 6;
  a.per_row = p.Hkv * p.D * (p.dtype == LS_BF16 ? 2 : 4) / 16;  // <= 256: 8 heads of 128 fp32 elements
  a.per_cta = kKv4Threads / a.per_row;
  a.per_row_inv = uint32_t((65536 + a.per_row - 1) / a.per_row);
  a.k = k;
  a.v = v;
  a.err = p.err;
  return a;
}

// Whole warps (at most kKv4Threads): the append's shuffles name every lane of a warp, and rows of 3
// heads of 64 or of 5 heads of 128, say, end inside one.
int kv4_threads(const Kv4Args& a) { return (a.per_cta * a.per_row + 31) / 32 * 32; }

}  // namespace

cudaError_t launch_kv4_append(const Dev& p, const ls_paged_kv4& kv, int layer, const void* k, const void* v,
                              int64_t row_stride, const int64_t* slots, int64_t n_rows, cudaStream_t stream) {
  const Kv4Args a = kv4_args(p, kv, layer, slots, n_rows, const_cast<void*>(k), const_cast<void*>(v), row_stride);
  const int threads = kv4_threads(a);
  const int64_t blocks = (n_rows + a.per_cta - 1) / a.per_cta;
  if (blocks > INT32_MAX) return cudaErrorNotSupported;
  const unsigned grid = static_cast<unsigned>(blocks);
  return p.dtype == LS_BF16 ? launch_overlapped(kv4_append_kernel<__nv_bfloat16>, dim3(grid), threads, 0, stream, a)
                            : launch_overlapped(kv4_append_kernel<float>, dim3(grid), threads, 0, stream, a);
}

cudaError_t launch_kv4_read(const Dev& p, const ls_paged_kv4& kv, int layer, const int64_t* slots, int64_t n_rows,
                            void* k, void* v, int64_t row_stride, cudaStream_t stream) {
  const Kv4Args a = kv4_args(p, kv, layer, slots, n_rows, k, v, row_stride);
  const int threads = kv4_threads(a);
  const int64_t blocks = (n_rows + a.per_cta - 1) / a.per_cta;
  if (blocks > INT32_MAX) return cudaErrorNotSupported;
  const unsigned grid = static_cast<unsigned>(blocks);
  return p.dtype == LS_BF16 ? launch_overlapped(kv4_read_kernel<__nv_bfloat16>, dim3(grid), threads, 0, stream, a)
                            : launch_overlapped(kv4_read_kernel<float>, dim3(grid), threads, 0, stream, a);
}

}  // namespace ls
