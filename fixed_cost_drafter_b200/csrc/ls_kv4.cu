// Rows into and out of the 4-bit KV cache (ls_kv4_append, ls_kv4_read_rows): see ls_kv4.cuh
// for the format. One thread per (row, KV head, group of 16 elements), keys and values in
// turn: the group's maximum stays in registers, its 16 codes leave as one 8-byte store. Both
// kernels move each element once; rows of a KV head lie 64 bytes apart in a page, so the
// stores fill whole 32-byte sectors of codes.
#include "ls_kv4.cuh"

namespace ls {

namespace {

constexpr int kKv4Threads = 256;

struct Kv4Args {
  unsigned char* base;  // the layer's pages
  int64_t page_stride;
  int64_t num_slots;
  int32_t page_size, page_shift;
  const int64_t* slots;
  int64_t n_rows, row_stride;
  int32_t H, D, groups;  // groups: H * D / 16 per row
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

// The code of x / s for s > 0: nearest e2m1 value, ties to even. The division is exact enough:
// a threshold t (half way between two values) times s has at most 7 bits, so x either equals
// t * s, and then x / s is t exactly, or differs from it by at least one part in 2^24, and
// then the rounded quotient lies on x's side of t (t * s < 2 t for the s that could be close).
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

template <typename T>
__global__ void __launch_bounds__(kKv4Threads) kv4_append_kernel(const Kv4Args a) {
  using E = Elem<T>;
  const int64_t i = int64_t(blockIdx.x) * kKv4Threads + threadIdx.x;
  const int64_t row = i / a.groups;
  if (row >= a.n_rows) return;
  const int grp = int(i - row * a.groups), per = a.D / kKv4Group;
  const int head = grp / per, gd = grp - head * per;
  int off;
  unsigned char* block = kv4_block(a, a.slots[row], head, off);
  if (!block) return;
  const Kv4Row r = kv4_row(block, a.page_size, a.D, off);
  const T* src = static_cast<const T*>(blockIdx.y ? a.v : a.k) + row * a.row_stride + grp * kKv4Group;
  float x[kKv4Group];
#pragma unroll
  for (int j = 0; j < kKv4Group; j += E::kVec) E::to_f32(ld_nc_v4(src + j), x + j);
  float top = 0.f;
  bool odd = false;  // an infinite or NaN element
#pragma unroll
  for (int j = 0; j < kKv4Group; ++j) {
    top = fmaxf(top, fabsf(x[j]));
    odd |= !(fabsf(x[j]) < INFINITY);
  }
  const uint32_t sb = odd ? 0x7fu : to_e4m3(__fdiv_rn(top, 6.f));
  const float s = odd ? 0.f : e4m3_to_f32(sb);
  uint32_t w[2] = {0u, 0u};
  if (s > 0.f) {
#pragma unroll
    for (int j = 0; j < kKv4Group; j += 2)
      w[j >> 3] |= pack_e2m1(__fdiv_rn(x[j], s), __fdiv_rn(x[j + 1], s)) << (4 * (j & 7));
  }
  *reinterpret_cast<uint2*>((blockIdx.y ? r.v_codes : r.k_codes) + gd * 8) = make_uint2(w[0], w[1]);
  (blockIdx.y ? r.v_scales : r.k_scales)[gd] = static_cast<unsigned char>(sb);
}

template <typename T>
__global__ void __launch_bounds__(kKv4Threads) kv4_read_kernel(const Kv4Args a) {
  using E = Elem<T>;
  const int64_t i = int64_t(blockIdx.x) * kKv4Threads + threadIdx.x;
  const int64_t row = i / a.groups;
  if (row >= a.n_rows) return;
  const int grp = int(i - row * a.groups), per = a.D / kKv4Group;
  const int head = grp / per, gd = grp - head * per;
  int off;
  unsigned char* block = kv4_block(a, a.slots[row], head, off);
  if (!block) return;
  const Kv4Row r = kv4_row(block, a.page_size, a.D, off);
  T* dst = static_cast<T*>(blockIdx.y ? a.v : a.k) + row * a.row_stride + grp * kKv4Group;
  const uint2 w = *reinterpret_cast<const uint2*>((blockIdx.y ? r.v_codes : r.k_codes) + gd * 8);
  const float s = e4m3_to_f32((blockIdx.y ? r.v_scales : r.k_scales)[gd]);
  uint32_t h[8];
  e2m1x8_to_half2(w.x, h);
  e2m1x8_to_half2(w.y, h + 4);
  float x[kKv4Group];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 f = half2_to_f2(h[j]);
    x[2 * j] = f.x * s;
    x[2 * j + 1] = f.y * s;
  }
#pragma unroll
  for (int j = 0; j < kKv4Group; j += E::kVec) *reinterpret_cast<uint4*>(dst + j) = E::from_f32(x + j);
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
  a.H = p.Hkv;
  a.D = p.D;
  a.groups = p.Hkv * p.D / kKv4Group;
  a.k = k;
  a.v = v;
  a.err = p.err;
  return a;
}

}  // namespace

cudaError_t launch_kv4_append(const Dev& p, const ls_paged_kv4& kv, int layer, const void* k, const void* v,
                              int64_t row_stride, const int64_t* slots, int64_t n_rows, cudaStream_t stream) {
  const Kv4Args a = kv4_args(p, kv, layer, slots, n_rows, const_cast<void*>(k), const_cast<void*>(v), row_stride);
  const int64_t blocks = (n_rows * a.groups + kKv4Threads - 1) / kKv4Threads;
  if (blocks > INT32_MAX) return cudaErrorNotSupported;
  const dim3 grid(static_cast<unsigned>(blocks), 2);
  if (p.dtype == LS_BF16) kv4_append_kernel<__nv_bfloat16><<<grid, kKv4Threads, 0, stream>>>(a);
  else kv4_append_kernel<float><<<grid, kKv4Threads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Dev& p, const ls_paged_kv4& kv, int layer, const int64_t* slots, int64_t n_rows,
                            void* k, void* v, int64_t row_stride, cudaStream_t stream) {
  const Kv4Args a = kv4_args(p, kv, layer, slots, n_rows, k, v, row_stride);
  const int64_t blocks = (n_rows * a.groups + kKv4Threads - 1) / kKv4Threads;
  if (blocks > INT32_MAX) return cudaErrorNotSupported;
  const dim3 grid(static_cast<unsigned>(blocks), 2);
  if (p.dtype == LS_BF16) kv4_read_kernel<__nv_bfloat16><<<grid, kKv4Threads, 0, stream>>>(a);
  else kv4_read_kernel<float><<<grid, kKv4Threads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace ls
