// Device code shared by the tree-attention kernels: what a call's arguments
// are, how the work is divided among the CTAs, and what a row sees.
//
// Work is counted in tiles of TK keys.  Request b has H key heads, rts row
// tiles of RT rows (a row is a new token with one of the `group` query heads
// of a key head) and `tiles` key tiles; an item is one (row tile, key head)
// of a request, and the items' tiles in order form one line, of which each
// CTA takes an equal piece.  So a single long context uses every SM and
// uneven contexts balance without the host knowing the lengths; a CTA's
// piece begins and ends inside an item at most once each, and those partial
// results (running maximum, sum and unnormalised output) go to the
// workspace, where combine_kernel joins them.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv_internal.cuh"
#include "sm100_ptx.cuh"
#include "tern_internal.cuh"

namespace tern {
namespace attn {

struct Args {
  const uint16_t* q;
  const uint16_t* v;        // the cache's values (non-finite drafts are read again)
  uint16_t* out;
  float* lse;
  const int32_t* table;
  const int32_t* ctx_len;
  const int32_t* row_start;
  const uint64_t* mask;
  float* part_o;            // [2 grid][RT][D] unnormalised outputs
  float2* part_ml;          // [2 grid][RT] (maximum, sum), base 2
  struct Join* join;        // [grid]
  int64_t q_token, q_head, table_stride;
  int64_t page_stride, token_stride, head_stride;
  int width, pages, page_shift, mask_words, B, T, H, group, Hq;
  float scale_log2;
};

// What a CTA leaves to be joined: the item that its piece begins but does
// not end (slot 1 of this CTA, then slot 0 of the next `follow` CTAs).
struct Join {
  int follow;   // 0: nothing
  int row0;     // first row of the request
  int r0;       // first row of the row tile
  int rows;     // its rows
  int head;     // key head
  int pad[3];
};

// One request.
struct Req {
  int ctx, n, row0, len, tiles, rts;
};

template <int TK, int RT>
__device__ __forceinline__ Req load_req(const Args& a, int b) {
  Req r;
  const int s0 = a.row_start[b], s1 = a.row_start[b + 1];
  const int cap = a.width << a.page_shift;
  const bool ok = s0 >= 0 && s1 >= s0 && s1 <= a.T;
  r.row0 = s0;
  r.n = ok ? s1 - s0 : 0;
  r.ctx = min(max(a.ctx_len[b], 0), cap);
  r.len = static_cast<int>(min(int64_t(r.ctx) + r.n, int64_t(cap)));
  r.tiles = r.n > 0 ? max((r.len + TK - 1) / TK, 1) : 0;
  r.rts = static_cast<int>((int64_t(r.n) * a.group + RT - 1) / RT);
  return r;
}

// A CTA's piece [lo, hi) of the line of tiles, and the request where it
// begins (`base`: tiles before that request).
struct Piece {
  int64_t lo, hi, total, base;
  int b, ctas;
  Req r;   // request b
};

// Shared scratch of find_piece for a CTA of NT threads.
template <int NT>
struct PieceScratch {
  int64_t warp[NT / 32];
  int64_t base;
  int b;
  Req r;
};

// Every thread of a CTA of NT threads (it synchronises them).
template <int TK, int RT, int NT>
__device__ __forceinline__ Piece find_piece(const Args& a, PieceScratch<NT>& s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int W = NT / 32;
  Piece p{};
  int64_t carry = 0;
  int64_t mine = 0, before = 0;   // of this thread's request in the last round of the scan
  Req r{};
  const auto round = [&](int base) {
    const int b = base + tid;
    mine = 0;
    if (b < a.B) {
      r = load_req<TK, RT>(a, b);
      mine = int64_t(a.H) * r.rts * r.tiles;
    }
    int64_t x = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(~0u, x, d);
      if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 31) s.warp[warp] = x;
    __syncthreads();
    int64_t below = carry;
    for (int w = 0; w < W; ++w) {
      const int64_t y = s.warp[w];
      if (w < warp) below += y;
      carry += y;
    }
    before = below + x - mine;
  };
  for (int base = 0; base < a.B; base += NT) round(base);
  p.total = carry;
  p.ctas = static_cast<int>(min(int64_t(gridDim.x), p.total));
  p.b = 0;
  p.base = 0;
  p.lo = p.hi = 0;
  if (static_cast<int>(blockIdx.x) >= p.ctas) return p;
  p.lo = p.total * blockIdx.x / p.ctas;
  p.hi = p.total * (blockIdx.x + 1) / p.ctas;
  const auto found = [&](int b) {
    if (before <= p.lo && p.lo < before + mine) {
      s.base = before;
      s.b = b;
      s.r = r;
    }
  };
  if (a.B <= NT) {
    found(tid);
  } else {
    carry = 0;
    for (int base = 0; base < a.B && carry <= p.lo; base += NT) {
      round(base);
      found(base + tid);
    }
  }
  __syncthreads();
  p.base = s.base;
  p.b = s.b;
  p.r = s.r;
  return p;
}

// Last CTA whose piece touches tile x of the line.
__device__ __forceinline__ int cta_of(const Piece& p, int64_t x) {
  return static_cast<int>(((x + 1) * p.ctas - 1) / p.total);
}

// One item's part in a CTA's piece.
struct Seg {
  Req r;
  int b, h, rt, t0, t1;   // key tiles [t0, t1)
  int64_t end;            // first tile of the line past the item
};

// Steps through a piece item by item.  Each role of a CTA walks on its own.
template <int TK, int RT>
struct Walk {
  const Args& a;
  int64_t w, hi, base;
  int b;
  Req r;
  int64_t size;

  __device__ __forceinline__ Walk(const Args& args, const Piece& p)
      : a(args), w(p.lo), hi(p.hi), base(p.base), b(p.b), r(p.r) {
    size = int64_t(a.H) * r.rts * r.tiles;
  }
  __device__ __forceinline__ bool next(Seg& s) {
    if (w >= hi) return false;
    while (w - base >= size) {   // total covers w: a request with tiles follows
      base += size;
      ++b;
      r = load_req<TK, RT>(a, b);
      size = int64_t(a.H) * r.rts * r.tiles;
    }
    const int64_t off = w - base;
    const int64_t item = off / r.tiles;
    s.r = r;
    s.b = b;
    s.t0 = static_cast<int>(off - item * r.tiles);
    s.t1 = static_cast<int>(min(int64_t(r.tiles), s.t0 + (hi - w)));
    s.h = static_cast<int>(item / r.rts);
    s.rt = static_cast<int>(item - int64_t(s.h) * r.rts);
    s.end = base + (item + 1) * r.tiles;
    w += s.t1 - s.t0;
    return true;
  }
};

// Whether a row (new token i, mask words mw) sees new token j.
__device__ __forceinline__ bool sees(const Args& a, const uint64_t* mw, int i, int j, int n) {
  if (j >= n) return false;
  if (a.mask == nullptr) return j <= i;
  return (j >> 6) < a.mask_words && ((mw[j >> 6] >> (j & 63)) & 1);
}

// The same for the N (16 or 32) keys from position k0 on, as bits: cached keys
// are seen, keys past the request's last are not.
template <int N>
__device__ __forceinline__ uint32_t sees_bits(const Args& a, const uint64_t* mw, int i, int k0,
                                              const Req& r) {
  const int j0 = k0 - r.ctx;              // k0 as a new token, below 0: cached
  const int lo = max(j0, 0), skip = min(lo - j0, N);
  uint64_t x = 0;
  if (skip < N) {
    if (a.mask == nullptr) {
      const int up = i - lo + 1;          // new tokens lo .. i
      x = up <= 0 ? 0 : up >= N ? 0xFFFFFFFFu : (1u << up) - 1;
    } else {
      const int w = lo >> 6, sh = lo & 63;
      if (w < a.mask_words) x = mw[w] >> sh;
      if (sh > 64 - N && w + 1 < a.mask_words) x |= mw[w + 1] << (64 - sh);
    }
  }
  const uint64_t bits = (x << skip) | ((uint64_t(1) << skip) - 1);
  const int valid = min(max(r.len - k0, 0), N);
  return static_cast<uint32_t>(bits & ((uint64_t(1) << valid) - 1));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}
template <bool BF16>
__device__ __forceinline__ float widen(uint16_t x) {
  if constexpr (BF16) return __uint_as_float(uint32_t(x) << 16);
  return __half2float(*reinterpret_cast<const __half*>(&x));
}
// Which of the two 16-bit values of a word are infinite or NaN (bits 0, 1).
template <bool BF16>
__device__ __forceinline__ uint32_t nonfinite2(uint32_t x) {
  constexpr uint32_t E = BF16 ? 0x7F80u : 0x7C00u;
  return ((x & E) == E ? 1u : 0u) | (((x >> 16) & E) == E ? 2u : 0u);
}

constexpr float kLn2 = 0.69314718055994530942f;

}  // namespace attn
}  // namespace tern
