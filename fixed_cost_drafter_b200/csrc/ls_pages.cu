// Block tables and slot maps from request lengths (ls_pages_extend, ls_pages_trim): the paged
// calls of a drafting round read them, an engine otherwise builds them on the host.
//
// With need_b = max(0, ceil((len_b + rows_b) / page_size) - held_b) and before_b the sum of
// need over the sequences before b, sequence b's j-th new page is free[count - 1 - before_b - j]
// (a stack popped in the order of the sequences), and row i of it has slot
// table[b][(len + i) / ps] * ps + (len + i) mod ps. Trim pushes the pages behind ceil(len / ps)
// so that it undoes an extend entry for entry; entries that name no page are left out.
//
// One launch each. Every CTA of a sequence sums what it needs over the sequences before it
// itself (a few loads per thread from L2, instead of a scan kernel before this one), takes new
// ids straight from the free list, and so needs nothing another CTA writes. The counts that
// all CTAs read (held, free_count) are updated by the last CTA to arrive. A round of 16 requests
// (extend and trim) takes 9.6 us, latency; 64 prompts of up to 128K rows, 34 MB of slots, 28 us,
// 23 of them the extend (its bytes take 6): some 90 warp instructions per 32 slots, each slot with a page
// id, a range check and an 8-byte store of its own, issued in 55 % of the cycles with the wait for
// page ids as the largest stall; and every prompt has the CTAs of the longest one, so that short
// prompts' are done early.
#include "ls_common.cuh"

namespace ls {

namespace {

constexpr int kPagesThreads = 256;
constexpr int kPagesAhead = 8;  // rows per thread whose page ids are loaded together

struct PagesArgs {
  ls_page_pool pool;
  const int64_t* len;  // element i at len[i * len_stride]
  int64_t len_stride;
  const int32_t* rows;
  int32_t max_rows;
  int64_t* row_begin;
  int64_t* slots;
  int64_t capacity;
  int32_t b, chunks;  // CTAs per sequence
  int32_t* arrive;
  int32_t* err;
};

// Page index and in-page offset of position pos.
__device__ inline int64_t split_pos(int64_t pos, int ps, int& off) {
  if ((ps & (ps - 1)) == 0) {
    off = int(pos & (ps - 1));
    return pos >> (__ffs(ps) - 1);
  }
  if (pos < (int64_t(1) << 32)) {
    const uint32_t q = uint32_t(pos) / uint32_t(ps);
    off = int(uint32_t(pos) - q * uint32_t(ps));
    return q;
  }
  const int64_t q = pos / ps;
  off = int(pos - q * ps);
  return q;
}
__device__ inline int64_t pages_for(int64_t rows, int ps) {
  int off;
  const int64_t q = split_pos(rows, ps, off);
  return q + (off > 0);
}

struct SeqPlan {
  int64_t len;
  int32_t n, held, pages;  // new rows; pages held; extend: pages missing, trim: pages to return
  bool bad;
};

__device__ inline SeqPlan plan_extend(const PagesArgs& a, int i) {
  SeqPlan s;
  s.len = a.len[int64_t(i) * a.len_stride];
  s.n = a.rows ? a.rows[i] : a.max_rows;
  s.held = a.pool.held[i];
  const int64_t most = int64_t(a.pool.max_blocks) * a.pool.page_size;
  s.bad = s.n < 0 || s.n > a.max_rows || s.len < 0 || s.len > most - s.n || s.held < 0 || s.held > a.pool.max_blocks;
  s.pages = 0;
  if (s.bad) {
    s.n = 0;
  } else {
    const int64_t t = pages_for(s.len + s.n, a.pool.page_size);
    if (t > s.held) s.pages = int32_t(t) - s.held;
  }
  return s;
}

__device__ inline SeqPlan plan_trim(const PagesArgs& a, int i) {
  SeqPlan s;
  s.len = a.len[int64_t(i) * a.len_stride];
  s.n = 0;
  s.held = a.pool.held[i];
  s.bad = s.len < 0 || s.held < 0 || s.held > a.pool.max_blocks;
  s.pages = 0;
  if (!s.bad) {
    const int64_t t = pages_for(s.len, a.pool.page_size);
    if (t < s.held) s.pages = s.held - int32_t(t);
  }
  return s;
}

// Sums of x and y over the block (every thread gets both).
__device__ inline void block_sum2(int64_t& x, int64_t& y) {
  __shared__ int64_t sx[kPagesThreads / 32], sy[kPagesThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    x += __shfl_xor_sync(0xffffffffu, x, o);
    y += __shfl_xor_sync(0xffffffffu, y, o);
  }
  __syncthreads();
  if (lane == 0) { sx[warp] = x; sy[warp] = y; }
  __syncthreads();
  x = y = 0;
#pragma unroll
  for (int w = 0; w < kPagesThreads / 32; ++w) { x += sx[w]; y += sy[w]; }
}

// Running sum of x over the block's threads, in order (without the thread's own); *total gets
// the block's sum.
__device__ inline int64_t block_scan(int64_t x, int64_t* total) {
  __shared__ int64_t sw[kPagesThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();
  if (lane == 31) sw[warp] = inc;
  __syncthreads();
  int64_t base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kPagesThreads / 32; ++w) {
    if (w < warp) base += sw[w];
    all += sw[w];
  }
  *total = all;
  return base + inc - x;
}

// True in every thread of the last CTA to arrive: every other CTA has read what it needs. `any`
// becomes whether `mine` was set in a thread of one of them, told by a bit of the count (a grid
// has fewer than 2^30 CTAs): reading the error word for it would cost a trip more.
constexpr int32_t kArriveMark = 1 << 30;
__device__ inline bool last_to_arrive(const PagesArgs& a, bool mine, bool& any) {
  __shared__ int32_t before;
  const bool mark = __syncthreads_or(mine);
  if (threadIdx.x == 0) {
    __threadfence();
    if (mark) atomicOr(a.arrive, kArriveMark);
    before = atomicAdd(a.arrive, 1);
    if ((before & ~kArriveMark) == int(gridDim.x) - 1) *a.arrive = 0;  // zero again for the next call
  }
  __syncthreads();
  any = (before & kArriveMark) != 0;
  return (before & ~kArriveMark) == int(gridDim.x) - 1;
}

__global__ void __launch_bounds__(kPagesThreads) pages_extend_kernel(const PagesArgs a) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int seq = int(blockIdx.x) / a.chunks, x = int(blockIdx.x) - seq * a.chunks;
  const int tid = threadIdx.x, ps = a.pool.page_size;
  const bool packed = a.row_begin != nullptr;
  const SeqPlan me = plan_extend(a, seq);
  const int count = *a.pool.free_count;
  const bool bad_count = count < 0 || count > a.pool.num_pages;
  const int64_t avail = bad_count ? 0 : count;

  int64_t before = 0, first_row = 0;  // pages and rows of the sequences before this one
  for (int i = tid; i < seq; i += kPagesThreads) {
    const SeqPlan s = plan_extend(a, i);
    before += s.pages;
    first_row += s.n;
  }
  block_sum2(before, first_row);
  const bool served = before + me.pages <= avail || me.pages == 0;
  int32_t bits = 0;
  if (me.bad) bits |= LS_DEVERR_ROWS;
  if (!served || bad_count) bits |= LS_DEVERR_POOL;

  int32_t* table = a.pool.block_table + int64_t(seq) * a.pool.max_blocks;
  const int32_t* top = a.pool.free_pages + (avail - 1 - before);  // page j of this sequence: top[-j]
  if (served) {
    for (int j = x * kPagesThreads + tid; j < me.pages; j += a.chunks * kPagesThreads)
      table[me.held + j] = top[-j];
  }
  int64_t* slots = a.slots + (packed ? first_row : int64_t(seq) * a.max_rows);
  const int64_t room = packed ? a.capacity - first_row : a.max_rows;
  const int n_out = packed ? me.n : a.max_rows;
  if (packed && n_out > room) bits |= LS_DEVERR_POOL;
  // several rows' pages are loaded together: each slot waits for its page's id
  const int step = a.chunks * kPagesThreads, n_write = int(n_out < room ? n_out : (room > 0 ? room : 0));
  const int64_t end = me.len + me.n;
  const bool simple = (ps & (ps - 1)) == 0 && end < (int64_t(1) << 31);  // 32-bit positions, shifts
  const int shift = __ffs(ps) - 1, len32 = int(me.len);
  if (simple) {
    for (int r0 = x * kPagesThreads + tid; r0 < n_write; r0 += kPagesAhead * step) {
      int32_t page[kPagesAhead];
#pragma unroll
      for (int u = 0; u < kPagesAhead; ++u) {
        const int r = r0 + u * step, pi = (len32 + r) >> shift;
        page[u] = served && r < me.n ? (pi < me.held ? table[pi] : top[me.held - pi]) : -1;
      }
#pragma unroll
      for (int u = 0; u < kPagesAhead; ++u) {
        const int r = r0 + u * step;
        if (r >= n_write) break;
        const bool ok = page[u] >= 0 && page[u] < a.pool.num_pages;
        if (!ok && served && r < me.n) bits |= LS_DEVERR_PAGE;
        slots[r] = ok ? (int64_t(page[u]) << shift) + ((len32 + r) & (ps - 1)) : -1;
      }
    }
  }
  for (int r0 = simple ? n_write : x * kPagesThreads + tid; r0 < n_write; r0 += kPagesAhead * step) {
    int64_t page[kPagesAhead];
    int off[kPagesAhead];
#pragma unroll
    for (int u = 0; u < kPagesAhead; ++u) {
      const int r = r0 + u * step;
      page[u] = -1;
      off[u] = -1;
      if (served && r < me.n && r < n_write) {
        const int64_t pi = split_pos(me.len + r, ps, off[u]);
        page[u] = pi < me.held ? table[pi] : top[-(pi - me.held)];
      }
    }
#pragma unroll
    for (int u = 0; u < kPagesAhead; ++u) {
      const int r = r0 + u * step;
      if (r >= n_write) break;
      int64_t slot = -1;
      if (off[u] >= 0) {
        if (page[u] < 0 || page[u] >= a.pool.num_pages) bits |= LS_DEVERR_PAGE;
        else slot = page[u] * ps + off[u];
      }
      slots[r] = slot;
    }
  }
  if (packed && x == 0 && tid == 0) {
    a.row_begin[seq] = first_row;
    if (seq == a.b - 1) a.row_begin[a.b] = first_row + me.n;
  }
  if (bits) set_err(a.err, bits);
  bool unused;
  if (!last_to_arrive(a, false, unused)) return;

  int64_t taken = 0;  // pages given so far, and pages needed so far
  int64_t needed = 0;
  for (int i0 = 0; i0 < a.b; i0 += kPagesThreads) {
    const int i = i0 + tid;
    SeqPlan s{};
    if (i < a.b) s = plan_extend(a, i);
    int64_t all;
    const int64_t mine = needed + block_scan(s.pages, &all);
    const bool ok = mine + s.pages <= avail;
    if (s.pages > 0 && ok) {
      a.pool.held[i] = s.held + s.pages;
      taken = mine + s.pages;
    }
    needed += all;
  }
  // the largest running sum that was served: every thread's last one, over the block
  __shared__ long long most;
  __syncthreads();
  if (tid == 0) most = 0;
  __syncthreads();
  atomicMax(&most, (long long)taken);
  __syncthreads();
  if (tid == 0 && !bad_count) *a.pool.free_count = count - int(most);
}

__global__ void __launch_bounds__(kPagesThreads) pages_trim_kernel(const PagesArgs a) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int seq = int(blockIdx.x) / a.chunks, x = int(blockIdx.x) - seq * a.chunks;
  const int tid = threadIdx.x;
  const SeqPlan me = plan_trim(a, seq);
  const int count = *a.pool.free_count;
  int64_t before = 0, total = 0;
  for (int i = tid; i < a.b; i += kPagesThreads) {
    const SeqPlan s = plan_trim(a, i);
    if (i < seq) before += s.pages;
    total += s.pages;
  }
  block_sum2(before, total);
  const bool ok = count >= 0 && count + total <= a.pool.num_pages;
  int32_t bits = 0;
  if (me.bad) bits |= LS_DEVERR_ROWS;
  if (!ok) bits |= LS_DEVERR_POOL;
  if (ok) {
    int32_t* table = a.pool.block_table + int64_t(seq) * a.pool.max_blocks + (me.held - me.pages);
    int32_t* top = a.pool.free_pages + (count + total - 1 - before);
    const int step = a.chunks * kPagesThreads;
    for (int j0 = x * kPagesThreads + tid; j0 < me.pages; j0 += kPagesAhead * step) {
      int32_t id[kPagesAhead];
#pragma unroll
      for (int u = 0; u < kPagesAhead; ++u) id[u] = table[min(j0 + u * step, me.pages - 1)];
#pragma unroll
      for (int u = 0; u < kPagesAhead; ++u) {
        const int j = j0 + u * step;
        if (j >= me.pages) break;
        if (id[u] < 0 || id[u] >= a.pool.num_pages) bits |= LS_DEVERR_PAGE;
        top[-j] = id[u];
        table[j] = -1;
      }
    }
  }
  if (bits) set_err(a.err, bits);
  bool gaps;  // a CTA met an id that names no page
  if (!last_to_arrive(a, bits & LS_DEVERR_PAGE, gaps) || !ok) return;
  for (int i = tid; i < a.b; i += kPagesThreads) {
    const SeqPlan s = plan_trim(a, i);
    if (s.pages > 0) a.pool.held[i] = s.held - s.pages;
  }
  // Such ids are dropped, or a later extend would hand them to other sequences: this CTA closes the
  // gaps. Each step's entries are read before any of its places, which lie at or before them, is
  // written (block_scan meets).
  int64_t kept = total;
  if (gaps) {
    __threadfence();
    kept = 0;
    for (int64_t i0 = 0; i0 < total; i0 += kPagesThreads) {
      const int32_t id = i0 + tid < total ? __ldcg(a.pool.free_pages + count + i0 + tid) : -1;
      const bool real = id >= 0 && id < a.pool.num_pages;
      int64_t all;
      const int64_t at = kept + block_scan(real, &all);
      if (real) a.pool.free_pages[count + at] = id;
      kept += all;
    }
  }
  if (tid == 0) *a.pool.free_count = count + int(kept);
}

PagesArgs pages_args(const Dev& p, const ls_page_pool& pool, const int64_t* len) {
  PagesArgs a{};
  a.pool = pool;
  a.len = len ? len : p.counters;
  a.len_stride = len ? 1 : int64_t(p.L) * (1 + p.nsc);
  a.b = p.b;
  a.arrive = p.arrive;
  a.err = p.err;
  return a;
}

// CTAs per sequence for `items` entries of work each: eight items a thread, at most about four
// CTAs an SM in all (more would spend their time on finding their place).
int chunks_for(int64_t items, int b, int sms) {
  const int64_t want = (items + 8 * kPagesThreads - 1) / (8 * kPagesThreads);
  const int64_t most = max(1, 4 * sms / b);
  return int(want < 1 ? 1 : (want < most ? want : most));
}

}  // namespace

cudaError_t launch_pages_extend(const Dev& p, const ls_page_pool& pool, const int64_t* len, const int32_t* rows,
                                int max_rows, int64_t* row_begin, int64_t* slots, int64_t capacity, int sms,
                                cudaStream_t stream) {
  PagesArgs a = pages_args(p, pool, len);
  a.rows = rows;
  a.max_rows = max_rows;
  a.row_begin = row_begin;
  a.slots = slots;
  a.capacity = capacity;
  a.chunks = chunks_for(max_rows, p.b, sms);
  return launch_overlapped(pages_extend_kernel, dim3(p.b * a.chunks), kPagesThreads, 0, stream, a);
}

cudaError_t launch_pages_trim(const Dev& p, const ls_page_pool& pool, const int64_t* len, int sms,
                              cudaStream_t stream) {
  PagesArgs a = pages_args(p, pool, len);
  a.chunks = chunks_for(pool.max_blocks, p.b, sms);
  return launch_overlapped(pages_trim_kernel, dim3(p.b * a.chunks), kPagesThreads, 0, stream, a);
}

}  // namespace ls
