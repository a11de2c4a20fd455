// Shared by the kernels of ls_verify_attend_kv4: arguments, the split of the work over the
// CTAs and where partial results go.
//
// Work: a tile is (sequence, KV head, block of MR query rows); row m of a (sequence, KV head)
// is query row m / group of query head g * group + m mod group. A tile's keys come in chunks
// of 128. All tiles' chunks form one line (sequence by sequence), cut into G equal ranges, one
// per CTA, whatever the lengths are: no CTA has more than one chunk more than another. A CTA
// whose range holds a whole tile writes its output rows; the pieces of a tile that is cut
// leave (reference, sum, unscaled output) in fp32, and a second kernel joins them in range
// order, so repeated calls give the same bits.
#pragma once
#include "ls_kv4.cuh"

namespace ls {

constexpr int kVerChunk = 128;   // keys per chunk
constexpr int kVerMaxSms = 160;  // CTA slots are sized for at most this many SMs
// Query rows per KV head up to which the warp-level kernel runs, the tcgen05 kernel above. Both
// measured, 8 KV heads of 128, 16 requests at 56K / at 4K, us: 16 rows 488 / 69, 20 rows 634 / 72 against
// 557 / 82, 24 rows 636 / 74 against 565 / 83, 32 rows (four row tiles) 969 / 106 against 592 / 86. Head dim
// 64, 4 KV heads, at 56K: 24 rows 253 against 277, 32 rows 326 against 285. From 17 to 24 rows the faster
// one depends on the lengths, which the host does not see: the warp-level kernel loses 14 % or wins
// 12; above them it loses 14 to 70 %.
constexpr int kMmaMostRows = 24;
// its CTAs per SM: registers hold 3 with up to 8 rows (shared memory as well), then 2 and 1
__host__ __device__ constexpr int mma_ctas(int rows) { return rows <= 8 ? 3 : (rows <= 16 ? 2 : 1); }
constexpr int kTcRows = 128;      // MR of the tcgen05 kernel: a state's query rows per KV head are at most 128
constexpr int kSimtRows = 8;     // MR of the CUDA-core kernel
constexpr int kSimtCtas = 4;     // its CTAs per SM

struct VerArgs {
  const unsigned char* base;  // the layer's pages
  int64_t page_stride, num_pages;
  const int32_t* table;
  int32_t max_blocks, page_size, page_shift;
  const void* q;
  int64_t q_stride;
  int32_t n_rows;
  const int32_t* rows;
  const int64_t* kv_len;
  float scale_log2;  // softmax_scale * log2(e)
  void* out;
  float* part_ml;  // [2 G][MR][2]: reference (log2 units) and sum of a piece's rows
  float* part_o;   // [2 G][MR][D]
  int32_t b, Hkv, Hq, grp, D;
  int32_t M, MR, HM;  // rows per (sequence, KV head), rows per tile, tiles per sequence
  int32_t G;          // CTAs
  int32_t out_f32, f32_in;
  int32_t* err;
};

__device__ inline int64_t ver_len(const VerArgs& a, int b) {
  const int64_t n = a.kv_len[b];
  return n < 0 || n > int64_t(a.max_blocks) * a.page_size ? 0 : n;
}
__device__ inline int ver_rows(const VerArgs& a, int b) {
  if (!a.rows) return a.n_rows;
  const int n = a.rows[b];
  return n < 0 ? 0 : (n > a.n_rows ? a.n_rows : n);
}
// (a sequence without query rows, an idle place of a padded batch, has no work, however long it is)
__device__ inline int64_t ver_chunks(const VerArgs& a, int b) {
  return ver_rows(a, b) > 0 ? (ver_len(a, b) + kVerChunk - 1) / kVerChunk : 0;
}

__device__ inline int64_t ver_warp_sum(int64_t x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Chunks of one tile row of the sequences [0, upto), whole warp.
__device__ inline int64_t ver_chunks_before(const VerArgs& a, int upto) {
  int64_t x = 0;
  for (int i = int(threadIdx.x & 31); i < upto; i += 32) x += ver_chunks(a, i);
  return ver_warp_sum(x);
}

// A CTA's place in the line of chunks.
struct VerCursor {
  int b, hm;      // next piece: sequence, tile of it
  int64_t chunk;  // its first chunk
  int64_t left;   // chunks left in this CTA's range
};

// One piece of a tile: chunks [c0, c1) of n.
struct VerPiece {
  int b, hm, rows;
  int64_t c0, c1, n, len;
};

// Whole warp: where CTA `cta` begins in the line, and its range's length (0 where it has none).
__device__ inline VerCursor ver_begin(const VerArgs& a, int cta) {
  VerCursor u{0, 0, 0, 0};
  const int lane = threadIdx.x & 31;
  const int64_t T = ver_chunks_before(a, a.b) * a.HM;
  const int64_t G = T < a.G ? T : a.G;
  if (cta >= G) return u;
  const int64_t g0 = int64_t(cta) * T / G, g1 = int64_t(cta + 1) * T / G;
  u.left = g1 - g0;
  int64_t base = 0;  // chunks of the sequences before the 32 looked at
  for (int i0 = 0; i0 < a.b; i0 += 32) {
    const int64_t mine = i0 + lane < a.b ? ver_chunks(a, i0 + lane) * a.HM : 0;
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, base + inc > g0);
    if (hit) {
      const int w = __ffs(int(hit)) - 1;
      const int64_t n = __shfl_sync(0xffffffffu, mine, w) / a.HM;
      const int64_t r = g0 - base - __shfl_sync(0xffffffffu, inc - mine, w);
      u.b = i0 + w;
      u.hm = int(r / n);
      u.chunk = r - int64_t(u.hm) * n;
      return u;
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  u.left = 0;  // not reached: g0 < T
  return u;
}

__device__ inline bool ver_next(const VerArgs& a, VerCursor& u, VerPiece& p) {
  if (u.left <= 0) return false;
  while (u.b < a.b) {
    p.len = ver_len(a, u.b);
    p.n = ver_chunks(a, u.b);
    if (p.n > 0) break;
    ++u.b;
  }
  if (u.b >= a.b) return false;
  p.b = u.b;
  p.hm = u.hm;
  p.rows = ver_rows(a, u.b);
  p.c0 = u.chunk;
  p.c1 = p.n - p.c0 < u.left ? p.n : p.c0 + u.left;
  u.left -= p.c1 - p.c0;
  u.chunk = 0;
  if (++u.hm == a.HM) {
    u.hm = 0;
    ++u.b;
  }
  return true;
}

// The slot of a cut tile's piece: a CTA cuts at most the tile its range begins in and the one
// it ends in.
__device__ inline int ver_slot(int cta, const VerPiece& p) { return 2 * cta + (p.c0 == 0 ? 1 : 0); }

// Keys that query row i of the piece's sequence sees: positions [0, limit).
__device__ inline int64_t ver_limit(const VerPiece& p, int i) {
  const int64_t t = p.len - p.rows + i + 1;
  return t < 0 ? 0 : t;
}

// Base of the (page, KV head) block of the page at index pi of sequence b; a page id outside
// the pool is flagged and read as page 0.
__device__ inline const unsigned char* ver_block(const VerArgs& a, int b, int64_t pi, int head) {
  int64_t page = __ldg(a.table + int64_t(b) * a.max_blocks + pi);
  if (page < 0 || page >= a.num_pages) {
    set_err(a.err, LS_DEVERR_PAGE);
    page = 0;
  }
  return a.base + page * a.page_stride + int64_t(head) * kv4_block_bytes(a.page_size, a.D);
}

// A value group with a NaN scale makes the rows that see its key NaN, and only those: weights
// of unseen keys are 0, and 0 * NaN would reach the others. Such a group takes part as zeros,
// and the smallest position per group of 16 elements is kept here (per piece): a row's group
// is NaN if its limit lies behind that position.
constexpr int kVerNone = 0x7fffffff;
__device__ inline bool nan_scale(uint32_t byte) { return (byte & 0x7fu) == 0x7fu; }

// Two values as fp16, low half first; 2^x (of the tensor-core kernels' softmax).
__device__ inline uint32_t ver_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ inline float ver_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// N output elements to memory, N a multiple of 2.
template <int N>
__device__ inline void ver_store(const VerArgs& a, int64_t at, const float* v) {
  if (a.out_f32 || a.f32_in) {
    float* o = static_cast<float*>(a.out) + at;
#pragma unroll
    for (int j = 0; j < N; j += 2) *reinterpret_cast<float2*>(o + j) = make_float2(v[j], v[j + 1]);
  } else {
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + at;
#pragma unroll
    for (int j = 0; j < N; j += 2) *reinterpret_cast<__nv_bfloat162*>(o + j) = __floats2bfloat162_rn(v[j], v[j + 1]);
  }
}
// Where row i, query head h of sequence b starts in the output.
__device__ inline int64_t ver_out_at(const VerArgs& a, int b, int i, int h) {
  return ((int64_t(b) * a.n_rows + i) * a.Hq + h) * a.D;
}

// Bounded wait of a whole warp; S holds the CTA's abort flag. Every lane polls: a whole warp's
// try_wait sleeps until the phase completes, one lane's comes back after about 200 cycles and
// polls again (a wait for a complete phase costs about 200 cycles either way).
template <typename S>
__device__ inline bool ver_wait_warp(S& s, uint64_t* bar, uint32_t parity, int32_t* err) {
  bool ok = false;
#pragma unroll 1
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    ok = mbar_try_wait(bar, parity);
    if (ok || ((i & 1023) == 1023 && *reinterpret_cast<volatile uint32_t*>(&s.abort))) break;
  }
  if (!ok) {
    if (!*reinterpret_cast<volatile uint32_t*>(&s.abort)) set_err(err, LS_DEVERR_WAIT_TIMEOUT);
    *reinterpret_cast<volatile uint32_t*>(&s.abort) = 1;
  }
  return __all_sync(0xffffffffu, ok);
}

// The producer warp of both tensor-core kernels: a CTA's chunks, in order, into a ring of kRing
// stages. A stage holds blocks of min(page_size, 128) rows as a page does (K codes, V codes, K
// scales, V scales): a page's block of a KV head is one bulk copy, of a 256-row page the chunk's
// half is copied section by section. A lane looks its page up one chunk before it is copied (always
// a load, of the first entry where there is none: a value chosen after a load waits for it at once).
template <int D, int kRing, typename S>
__device__ inline void ver_produce(const VerArgs& a, S& s, uint64_t* full, uint64_t* empty, unsigned char* ring) {
  constexpr int kStage = kVerChunk * (D + D / 8);
  const int lane = threadIdx.x & 31;
  const int ps = min(a.page_size, kVerChunk), pshift = min(a.page_shift, 7);
  const bool wide = a.page_size > kVerChunk;
  const int lanes = wide ? 4 : kVerChunk >> pshift;
  VerCursor cur = ver_begin(a, blockIdx.x);
  VerPiece p;
  const int total = int(cur.left);
  int64_t pos = 0;  // of this lane's page in the chunk looked up
  int left = 0, k = 0;
  int32_t entry = 0;
  auto look_up = [&]() {
    if (left == 0) {
      if (!ver_next(a, cur, p)) return;
      left = int(p.c1 - p.c0);
      pos = p.c0 * kVerChunk + (wide ? 0 : int64_t(lane) << pshift);
    }
    entry = __ldg(a.table + (lane < lanes && pos < p.len ? int64_t(p.b) * a.max_blocks + (pos >> a.page_shift) : 0));
  };
  look_up();
  for (; k < total; ++k) {
    const bool held = lane < lanes && pos < p.len;
    int64_t page = entry;
    if (page < 0 || page >= a.num_pages) {  // flagged, and read as page 0
      if (held) set_err(a.err, LS_DEVERR_PAGE);
      page = 0;
    }
    const unsigned char* block = a.base + page * a.page_stride + int64_t(p.hm) * kv4_block_bytes(a.page_size, D);
    const int first = int(pos) & (a.page_size - 1);
    --left;
    pos += kVerChunk;
    look_up();
    const int st = k % kRing;
    if (k >= kRing && !ver_wait_warp(s, &empty[st], uint32_t(k / kRing - 1) & 1, a.err)) break;
    unsigned char* dst = ring + st * kStage;
    const int n = __popc(__ballot_sync(0xffffffffu, held));
    if (lane == 0) mbar_arrive_expect_tx(&full[st], uint32_t(wide ? kStage : n * kv4_block_bytes(ps, D)));
    __syncwarp();
    if (wide) {
      if (lane < 4) {  // 128 of the page's rows: codes (lanes 0, 1) and scales (2, 3)
        const int row = lane < 2 ? D / 2 : D / kKv4Group, bytes = kVerChunk * row;
        const int64_t from = (lane < 2 ? 0 : int64_t(a.page_size) * D) + int64_t((lane & 1) * a.page_size + first) * row;
        bulk_g2s(dst + (lane < 2 ? 0 : kVerChunk * D) + (lane & 1) * bytes, block + from, bytes, &full[st]);
      }
    } else if (held) {
      bulk_g2s(dst + lane * kv4_block_bytes(ps, D), block, kv4_block_bytes(ps, D), &full[st]);
    }
  }
  // after an abort: the copies in flight land before the shared memory is released
  if (lane == 0 && *reinterpret_cast<volatile uint32_t*>(&s.abort))
    for (int x = k > kRing ? k - kRing : 0; x < k; ++x)
      mbar_wait_bounded(&full[x % kRing], uint32_t(x / kRing) & 1, kWaitLimit);
}

}  // namespace ls
