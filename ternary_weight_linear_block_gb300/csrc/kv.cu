// The paged key/value cache around the attention of drafted tokens: block
// tables and slot maps from the requests' lengths (kv_plan), the new rows
// into their slots (kv_write), and the accepted path of every tree made
// contiguous (kv_commit).  All three move integers or 16-bit rows and do no
// arithmetic on them.
#include <algorithm>

#include "kv_internal.cuh"
#include "tern_internal.cuh"

namespace tern {
namespace {

// ------------------------------------------------------------------ plan
//
// Two sums over the requests carry everything: the rows before request b
// (its row start) and the further pages taken before it.  Every CTA adds
// them up for itself (B is at most 8192 lengths, read from L2) and keeps both,
// the cached lengths and the pages held in shared memory, so one launch is
// enough and no CTA waits for another; a row or a page then finds its request
// by bisection and has one number to read, its page.  Bound: the launch and
// two dependent round trips to L2 (16 requests, 204 rows: 4.2 us on the
// device), then the steps of the bisections before the 16 bytes written for
// each row (1024 requests, 1.17 million rows: 12.7 us, 1.5 TB/s; written at
// copy rate the rows would take 2.8).

constexpr int PLAN_THREADS = 512;
constexpr int PLAN_ROWS = 4;   // rows of one thread
constexpr int PLAN_REQS = 2;   // consecutive requests of one thread in a round of the sums

struct PlanArgs {
  const int32_t* ctx_len;
  const int32_t* new_len;
  int32_t* table;
  const int32_t* held;
  const int32_t* free_pages;
  const int32_t* free_head;
  int32_t* row_start;
  int64_t* slots;
  int32_t* positions;
  int32_t* request;
  int32_t* held_out;
  int32_t* info;
  int64_t table_stride;
  int B, shift, width, n_free, capacity;
};

// For each of N numbers the largest b with start[b] <= x (start[0] = 0, not
// decreasing, B entries): side by side, as every step waits for shared memory.
template <int N>
__device__ __forceinline__ void requests_of(const int* start, int B, const int (&x)[N], int (&b)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) b[i] = 0;
  int step = 1;
  while (step < B) step <<= 1;
  for (step >>= 1; step > 0; step >>= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) {      // without branches, or the reads do not overlap
      const int at = b[i] + step;
      const int first = start[min(at, B)];
      b[i] = (at < B) & (first <= x[i]) ? at : b[i];
    }
  }
}

// A warp has 32 ROWS consecutive rows, 32 at a time, so that its stores are
// whole lines.  Four: with eight, fewer threads wait for as many bisections
// (204 rows 5.3 us against 4.6, 80000 rows 7.1 against 5.3, 1.17 million 13.3
// against 12.7).
__global__ void __launch_bounds__(PLAN_THREADS, 2) plan_kernel(const __grid_constant__ PlanArgs a) {
  constexpr int ROWS = PLAN_ROWS;
  extern __shared__ int s_sums[];
  int* s_row = s_sums;                   // [B + 1] rows before request b
  int* s_page = s_row + a.B + 1;         // [B + 1] further pages before it
  int* s_ctx = s_page + a.B + 1;         // [B] cached tokens
  int* s_held = s_ctx + a.B;             // [B] pages in the table row
  __shared__ int64_t s_warp[2][PLAN_THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_launch_dependents();
  const int head0 = a.free_head != nullptr ? *a.free_head : 0;   // on its way with the lengths
  const int head = min(max(head0, 0), a.n_free);
  const int64_t avail = a.n_free - head;

  int64_t rows0 = 0, pages0 = 0;
  int flags = 0;
  for (int base = 0; base < a.B; base += PLAN_THREADS * PLAN_REQS) {
    int64_t n[PLAN_REQS], more[PLAN_REQS], rows = 0, pages = 0;
    const int b0 = base + tid * PLAN_REQS;
#pragma unroll
    for (int i = 0; i < PLAN_REQS; ++i) {
      const int b = b0 + i;
      const int cl = b < a.B ? a.ctx_len[b] : 0, nl = b < a.B ? a.new_len[b] : 0;
      const int c = max(cl, 0);
      if (cl < 0 || nl < 0) flags |= 8;
      n[i] = max(nl, 0);
      const int64_t up = (int64_t(1) << a.shift) - 1;
      const int64_t all = (int64_t(c) + n[i] + up) >> a.shift;
      int64_t held = (int64_t(c) + up) >> a.shift;
      if (a.held != nullptr) held = b < a.B ? max(a.held[b], 0) : 0;
      held = held < a.width ? held : a.width;
      if (all > a.width) flags |= 2;
      more[i] = max((all < a.width ? all : a.width) - held, int64_t(0));
      rows += n[i];
      pages += more[i];
      if (b < a.B) {
        s_ctx[b] = c;
        s_held[b] = static_cast<int>(held);
      }
    }
    const int64_t mine_r = rows, mine_p = pages;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t r = __shfl_up_sync(~0u, rows, d), p = __shfl_up_sync(~0u, pages, d);
      if (lane >= d) {
        rows += r;
        pages += p;
      }
    }
    __syncthreads();
    if (lane == 31) {
      s_warp[0][warp] = rows;
      s_warp[1][warp] = pages;
    }
    __syncthreads();
    int64_t before_r = rows0 + rows - mine_r, before_p = pages0 + pages - mine_p;
#pragma unroll
    for (int w = 0; w < PLAN_THREADS / 32; ++w) {
      const int64_t r = s_warp[0][w], p = s_warp[1][w];
      if (w < warp) {
        before_r += r;
        before_p += p;
      }
      rows0 += r;
      pages0 += p;
    }
#pragma unroll
    for (int i = 0; i < PLAN_REQS; ++i) {
      // held: what it has and what it gets of the free pages, which may run out
      if (a.held_out != nullptr && blockIdx.x == 0 && b0 + i < a.B)
        a.held_out[b0 + i] = s_held[b0 + i] + static_cast<int>(min(max(avail - before_p, int64_t(0)), more[i]));
      before_r += n[i];
      before_p += more[i];
      if (b0 + i < a.B) {   // sums past 2^31 stay at its end: past every row asked for
        s_row[b0 + i + 1] = static_cast<int>(min(before_r, int64_t(INT32_MAX)));
        s_page[b0 + i + 1] = static_cast<int>(min(before_p, int64_t(INT32_MAX)));
      }
    }
  }
  if (tid == 0) s_row[0] = s_page[0] = 0;
  if (blockIdx.x == 0) {
    const int too_long = __syncthreads_or(flags & 2) ? 2 : 0;
    const int negative = __syncthreads_or(flags & 8) ? 8 : 0;
    for (int b = tid; b <= a.B; b += PLAN_THREADS) a.row_start[b] = s_row[b];
    if (tid == 0) {
      const int taken = static_cast<int>(min(pages0, avail));
      a.info[0] = s_row[a.B];
      a.info[1] = taken;
      a.info[2] = head + taken;
      a.info[3] = too_long | negative | (pages0 > avail ? 1 : 0) | (rows0 > a.capacity ? 4 : 0);
    }
  } else {
    __syncthreads();
  }
  const int total = s_row[a.B];
  const int pages_all = s_page[a.B];

  // the rows
  const int64_t warps = int64_t(gridDim.x) * (PLAN_THREADS / 32);
  for (int64_t w = int64_t(blockIdx.x) * (PLAN_THREADS / 32) + warp; w * (32 * ROWS) < a.capacity;
       w += warps) {
    int row[ROWS], b[ROWS], page[ROWS];
    int64_t p[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) row[i] = static_cast<int>(min(w * (32 * ROWS) + i * 32 + lane, int64_t(INT32_MAX)));
    // long requests: the warp's first and last rows have the same one
    const int ends[2] = {static_cast<int>(w * (32 * ROWS)),
                         static_cast<int>(min(w * (32 * ROWS) + 32 * ROWS - 1, int64_t(INT32_MAX)))};
    int of[2];
    requests_of<2>(s_row, a.B, ends, of);
    if (of[0] == of[1]) {
#pragma unroll
      for (int i = 0; i < ROWS; ++i) b[i] = of[0];
    } else {
      requests_of<ROWS>(s_row, a.B, row, b);
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      // one address each and no branches, so that all the reads are on their
      // way together
      const int bi = min(b[i], a.B - 1);
      const bool in = (row[i] < total) & (row[i] < a.capacity);
      const int c = bi >= 0 ? s_ctx[bi] : 0, held = bi >= 0 ? s_held[bi] : 0;
      const int start = bi >= 0 ? s_row[bi] : 0, more = bi >= 0 ? s_page[bi] : 0;
      p[i] = in ? int64_t(c) + (row[i] - start) : 0;
      const int64_t at = p[i] >> a.shift, taken = more + (at - held);
      const bool known = at < held;
      const int32_t* from = known ? a.table + bi * a.table_stride + at : a.free_pages + head + taken;
      page[i] = in & (known | ((at < a.width) & (taken < avail))) ? __ldg(from) : -1;
      b[i] = in ? bi : -1;
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (row[i] < a.capacity) {
        a.slots[row[i]] = page[i] < 0 ? -1 : (int64_t(page[i]) << a.shift) +
                                                 (p[i] & ((int64_t(1) << a.shift) - 1));
        a.positions[row[i]] = static_cast<int>(min(p[i], int64_t(INT32_MAX)));
        a.request[row[i]] = b[i];
      }
    }
  }
  // the further pages into the table (entries that no row reads)
  const int64_t threads = int64_t(gridDim.x) * PLAN_THREADS;
  for (int64_t q = int64_t(blockIdx.x) * PLAN_THREADS + tid; q < pages_all; q += threads) {
    const int x[1] = {static_cast<int>(q)};
    int b[1];
    requests_of<1>(s_page, a.B, x, b);
    const int64_t at = s_held[b[0]] + (q - s_page[b[0]]);
    if (at < a.width) a.table[b[0] * a.table_stride + at] = q < avail ? a.free_pages[head + q] : -1;
  }
}

// ------------------------------------------------------------------ write
//
// A copy of 16-byte chunks to slots: `tpt` threads (a power of two) share a
// row, so that a few rows still use many threads and many rows keep a warp's
// accesses in one row.  Bound: the rows read and written once (95601 rows of
// 8 heads of 128: 784 MB in 122 us, 6.4 TB/s, 0.96 of a copy's rate; 16 rows of
// 20 heads: 1.7 us, the launch).

constexpr int COPY_THREADS = 256;

struct WriteArgs {
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* ck;
  uint16_t* cv;
  const int64_t* slots;
  int64_t k_token, k_head, v_token, v_head;
  int64_t page_stride, token_stride, head_stride;
  int64_t T, n_slots;
  int chunks;                             // 16-byte chunks of a row of all heads
  int dim_shift, page_shift, tpt_shift;   // log2 of chunks a head, of the page size, of tpt
};

__global__ void __launch_bounds__(COPY_THREADS) write_kernel(const WriteArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int tpt = 1 << a.tpt_shift;
  const int64_t step = (int64_t(gridDim.x) * COPY_THREADS) >> a.tpt_shift;
  const int part = threadIdx.x & (tpt - 1);
  for (int64_t t = (int64_t(blockIdx.x) * COPY_THREADS + threadIdx.x) >> a.tpt_shift; t < a.T;
       t += step) {
    const int64_t slot = a.slots[t];
    if (slot < 0 || slot >= a.n_slots) continue;
    const int64_t to = (slot >> a.page_shift) * a.page_stride +
                       (slot & ((int64_t(1) << a.page_shift) - 1)) * a.token_stride;
    const uint16_t* k = a.k + t * a.k_token;
    const uint16_t* v = a.v + t * a.v_token;
#pragma unroll 4
    for (int c = part; c < a.chunks; c += tpt) {
      const int64_t h = c >> a.dim_shift;
      const int64_t d = (c & ((1 << a.dim_shift) - 1)) * 8;
      const uint4 kk = *reinterpret_cast<const uint4*>(k + h * a.k_head + d);
      const uint4 vv = *reinterpret_cast<const uint4*>(v + h * a.v_head + d);
      *reinterpret_cast<uint4*>(a.ck + to + h * a.head_stride + d) = kk;
      *reinterpret_cast<uint4*>(a.cv + to + h * a.head_stride + d) = vv;
    }
  }
}

// ------------------------------------------------------------------ commit
//
// A thread owns one 16-byte column of a request's rows and moves it for the
// whole path.  A path increases, so path[j] >= j: row j is written only
// after it was read as a source (path[j'] = j needs j' <= j), and a later
// source path[j'] > path[j] >= j is never a row already written.  So loads
// may run ahead of stores and no thread waits for another.  Bound: the
// moved rows read and written once (61 requests of up to 64 drafts, 16 layers:
// 452 MB in 73 us, 6.2 TB/s); at decode sizes the launch and three dependent
// round trips (path, table, rows: 2 requests, 16 layers 4.9 us with the write).

constexpr int MAX_PATH = 256;
constexpr int COMMIT_LAYERS = 64;   // layers of one launch: their pointers are kernel arguments

struct CommitArgs {
  uint16_t* ptr[2 * COMMIT_LAYERS];   // keys, values of each layer
  const int32_t* table;
  const int32_t* ctx_len;
  const int32_t* path;
  const int32_t* path_len;
  int32_t* ctx_out;
  int64_t table_stride, path_stride;
  int64_t page_stride, token_stride, head_stride, pages;
  int width, path_width, chunks, dim_shift, page_shift;
};

__global__ void __launch_bounds__(COPY_THREADS) commit_kernel(const __grid_constant__ CommitArgs a) {
  __shared__ int64_t s_from[MAX_PATH], s_to[MAX_PATH];
  __shared__ int s_count;
  const int b = blockIdx.y, tid = threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const int ctx = a.ctx_len[b];
  const int len = ctx < 0 ? 0 : min(max(a.path_len[b], 0), a.path_width);
  if (tid == 0) s_count = len;
  __syncthreads();
  // row of position p in the cache, or -1
  const auto place = [&](int64_t p) -> int64_t {
    const int64_t at = p >> a.page_shift;
    if (at >= a.width) return -1;
    const int64_t page = a.table[b * a.table_stride + at];
    if (page < 0 || page >= a.pages) return -1;
    return page * a.page_stride + (p & ((int64_t(1) << a.page_shift) - 1)) * a.token_stride;
  };
  for (int j = tid; j < len; j += COPY_THREADS) {
    const int p = a.path[b * a.path_stride + j];
    const int prev = j > 0 ? a.path[b * a.path_stride + j - 1] : -1;
    int64_t from = -1, to = -1;
    if (p >= 0 && p > prev) {
      from = place(int64_t(ctx) + p);
      to = p == j ? from : place(int64_t(ctx) + j);
    }
    if (from < 0 || to < 0) atomicMin(&s_count, j);
    s_from[j] = from;
    s_to[j] = to;
  }
  __syncthreads();
  const int count = s_count;
  if (a.ctx_out != nullptr && blockIdx.x == 0 && blockIdx.z == 0 && tid == 0)
    a.ctx_out[b] = ctx + count;
  const int c = blockIdx.x * COPY_THREADS + tid;
  if (c >= a.chunks) return;
  const int64_t col = int64_t(c >> a.dim_shift) * a.head_stride +
                      (c & ((1 << a.dim_shift) - 1)) * 8;
  uint16_t* x = a.ptr[blockIdx.z] + col;   // keys and values are two planes of z
  constexpr int U = 4;
  for (int j0 = 0; j0 < count; j0 += U) {
    uint4 r[U];
    bool move[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      move[i] = j0 + i < count && s_from[j0 + i] != s_to[j0 + i];
      if (move[i]) r[i] = *reinterpret_cast<const uint4*>(x + s_from[j0 + i]);
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (move[i]) *reinterpret_cast<uint4*>(x + s_to[j0 + i]) = r[i];
  }
}

int log2_of(int64_t v) {
  int s = 0;
  while ((int64_t(1) << s) < v) ++s;
  return s;
}

}  // namespace

// SMs of the current device (asked once per device; 152, GB300's, without one).
int kv_sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  n = known[dev].load(std::memory_order_relaxed);
  if (n > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 152;
  known[dev].store(n, std::memory_order_relaxed);
  return n;
}

cudaError_t launch_kv_plan(const int32_t* ctx_len, const int32_t* new_len, int64_t B,
                           int64_t page_size, int32_t* table, int64_t table_stride,
                           int64_t table_width, const int32_t* held, const int32_t* free_pages,
                           int64_t n_free, const int32_t* free_head, int32_t* row_start,
                           int64_t capacity, int64_t* slots, int32_t* positions, int32_t* request,
                           int32_t* held_out, int32_t* info, cudaStream_t st) {
  static std::atomic<unsigned long long> attr_done{0};
  const size_t smem = static_cast<size_t>(4 * B + 2) * sizeof(int);
  const cudaError_t e = once_per_device(attr_done, [] {
    constexpr int most = (4 * 8192 + 2) * static_cast<int>(sizeof(int));
    return cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  });
  if (e != cudaSuccess) return e;
  PlanArgs a{ctx_len, new_len, table, held, free_pages, free_head, row_start, slots, positions,
             request, held_out, info, table_stride, static_cast<int>(B), log2_of(page_size),
             static_cast<int>(table_width), static_cast<int>(n_free), static_cast<int>(capacity)};
  const int64_t per_block = int64_t(PLAN_THREADS) * PLAN_ROWS;
  const int64_t blocks = std::min(std::max<int64_t>((capacity + per_block - 1) / per_block, 1),
                                  int64_t(2) * kv_sm_count());
  return launch(plan_kernel, dim3(static_cast<unsigned>(blocks)), dim3(PLAN_THREADS), smem, st, a);
}

cudaError_t launch_kv_write(const tern_kv_cache& c, const void* k, const void* v, int64_t k_token,
                            int64_t k_head, int64_t v_token, int64_t v_head, const int64_t* slots,
                            int64_t T, cudaStream_t st) {
  WriteArgs a{static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
              static_cast<uint16_t*>(c.k), static_cast<uint16_t*>(c.v), slots, k_token, k_head,
              v_token, v_head, c.page_stride, c.token_stride, c.head_stride, T,
              c.pages * c.page_size, static_cast<int>(c.heads * c.dim / 8), log2_of(c.dim / 8),
              log2_of(c.page_size), 0};
  // one chunk a thread while that fits the GPU once, at most a warp a row beyond
  // (a warp a row always: 16 rows of 20 heads 4.0 us against 1.9; one chunk a
  // thread always: 95601 rows of 8 heads 126 us against 122)
  const int64_t room = int64_t(kv_sm_count()) * 2048;
  int shift = 0;
  while (shift < 8 && (2 << shift) <= a.chunks && (shift < 5 || (T << (shift + 1)) <= room)) ++shift;
  a.tpt_shift = shift;
  const int64_t blocks = std::min<int64_t>(((T << shift) + COPY_THREADS - 1) / COPY_THREADS,
                                           int64_t(kv_sm_count()) * 8);
  return launch(write_kernel, dim3(static_cast<unsigned>(blocks)), dim3(COPY_THREADS), 0, st, a);
}

cudaError_t launch_kv_commit(const tern_kv_cache* caches, int64_t layers, const int32_t* table,
                             int64_t table_stride, int64_t table_width, const int32_t* ctx_len,
                             const int32_t* path, int64_t path_width, const int32_t* path_len,
                             int32_t* ctx_out, int64_t B, cudaStream_t st) {
  const tern_kv_cache& c = caches[0];
  const int chunks = static_cast<int>(c.heads * c.dim / 8);
  for (int64_t l0 = 0; l0 < layers; l0 += COMMIT_LAYERS) {
    const int n = static_cast<int>(std::min<int64_t>(layers - l0, COMMIT_LAYERS));
    CommitArgs a{};
    for (int l = 0; l < n; ++l) {
      a.ptr[2 * l] = static_cast<uint16_t*>(caches[l0 + l].k);
      a.ptr[2 * l + 1] = static_cast<uint16_t*>(caches[l0 + l].v);
    }
    a.table = table;
    a.ctx_len = ctx_len;
    a.path = path;
    a.path_len = path_len;
    a.ctx_out = l0 == 0 ? ctx_out : nullptr;
    a.table_stride = table_stride;
    a.path_stride = path_width;
    a.page_stride = c.page_stride;
    a.token_stride = c.token_stride;
    a.head_stride = c.head_stride;
    a.pages = c.pages;
    a.width = static_cast<int>(table_width);
    a.path_width = static_cast<int>(path_width);
    a.chunks = chunks;
    a.dim_shift = log2_of(c.dim / 8);
    a.page_shift = log2_of(c.page_size);
    const dim3 grid(static_cast<unsigned>((chunks + COPY_THREADS - 1) / COPY_THREADS),
                    static_cast<unsigned>(B), static_cast<unsigned>(2 * n));
    const cudaError_t e = launch(commit_kernel, grid, dim3(COPY_THREADS), 0, st, a);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace tern
