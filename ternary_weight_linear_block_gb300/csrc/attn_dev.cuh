// Device code shared by the tree-attention kernels: what a call's arguments
// are, how the work is divided among the CTAs, and what a row sees.
//
// Work is counted in tiles of TK keys.  Request b has H key heads, rts row
// tiles of RT rows (a row is a new token with one of the `group` query heads
// of a key head) and `tiles` key tiles; an item is one (row tile, key head)
// of a request, and the items' tiles in order form one line, of which each
// CTA takes an equal piece.  An item counts PAD tiles more than it has, for
// what it costs beside its tiles (queries, masks, output), so that a CTA with
// many short items has as long as one with a long one.  So a single long context uses every SM and
// uneven contexts balance without the host knowing the lengths; a CTA's
// piece begins and ends inside an item at most once each, and those partial
// results (running maximum, sum and unnormalised output) go to the
// workspace, where they are joined: by the last of the item's CTAs to arrive
// (join_piece, few rows) or by a second kernel (combine_kernel, many).
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
  float* part_o;            // [2 grid][D / 4][RT][4] unnormalised outputs
  float2* part_ml;          // [2 grid pieces, 2 grid sums][RT] (maximum, sum), base 2
  int* arrived;             // [3 grid] pieces that have arrived, 0 between calls
  struct Item* items;       // [grid] the item that each CTA's piece begins but does not end
  int64_t q_token, q_head, table_stride;
  int64_t page_stride, token_stride, head_stride;
  int width, pages, page_shift, mask_words, B, T, H, group, Hq;
  uint32_t group_mul;       // 2^32 / group + 1, or 0 (div_group)
  int tile_rows;            // rows of an item, RT or (tile kernel) whole tokens of it
  float scale_log2;
};

// One request.
struct Req {
  int ctx, n, row0, len, tiles, rts;
};

// Row r of a request on a key head -> its new token.  r is below T group,
// whatever the lengths on the GPU are, and the product with 2^32 / group + 1 is
// exact while r group < 2^32: the host gives the factor only then.
__device__ __forceinline__ int div_group(const Args& a, int r) {
  if (a.group_mul != 0) return static_cast<int>(__umulhi(static_cast<uint32_t>(r), a.group_mul));
  return a.group == 1 ? r : r / a.group;
}

// Tiles that an item counts for.
template <int PAD>
__device__ __forceinline__ int64_t line_of(const Args& a, const Req& r) {
  return r.n > 0 ? int64_t(a.H) * r.rts * (r.tiles + PAD) : 0;
}

template <int TK>
__device__ __forceinline__ Req load_req(const Args& a, int b) {
  Req r;
  const int s0 = a.row_start[b], s1 = a.row_start[b + 1];
  const int cap = a.width << a.page_shift;
  const bool ok = s0 >= 0 && s1 >= s0 && s1 <= a.T;
  r.row0 = s0;
  r.n = ok ? s1 - s0 : 0;
  r.ctx = min(max(a.ctx_len[b], 0), cap);
  r.len = static_cast<int>(min(int64_t(r.ctx) + r.n, int64_t(cap)));
  r.tiles = r.n > 0 ? max(r.len - 1, 0) / TK + 1 : 0;   // (a position may be the last of 31 bits)
  const uint32_t rt = a.tile_rows;
  r.rts = static_cast<int>((uint32_t(r.n) * uint32_t(a.group) + rt - 1) / rt);   // below 2^28 rows
  return r;
}

// a / b of numbers that are not negative; two of 32 bits are the usual case and
// cost a fifth of a 64-bit division.
__device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
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
template <int TK, int PAD, int LEAST, int NT>
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
      r = load_req<TK>(a, b);
      mine = line_of<PAD>(a, r);
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
  // no more CTAs than have LEAST places each: a part smaller than that costs
  // more in starting and joining than it saves
  p.ctas = static_cast<int>(min(int64_t(gridDim.x), max(quot(p.total, LEAST), min(p.total, int64_t(1)))));
  p.b = 0;
  p.base = 0;
  p.lo = p.hi = 0;
  if (static_cast<int>(blockIdx.x) >= p.ctas) return p;
  p.lo = quot(p.total * blockIdx.x, p.ctas);
  p.hi = quot(p.total * (blockIdx.x + 1), p.ctas);
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
  return static_cast<int>(quot((x + 1) * p.ctas - 1, p.total));
}

// One item's part in a CTA's piece.
struct Seg {
  Req r;
  int b, h, rt, t0, t1;   // key tiles [t0, t1)
  int64_t first, end;     // the item's first tile on the line, and the place past its last
};

// Steps through a piece item by item.  Each role of a CTA walks on its own.
template <int TK, int PAD>
struct Walk {
  const Args& a;
  int64_t w, hi, base;
  int b;
  Req r;
  int64_t size;

  __device__ __forceinline__ Walk(const Args& args, const Piece& p)
      : a(args), w(p.lo), hi(p.hi), base(p.base), b(p.b), r(p.r), size(line_of<PAD>(args, p.r)) {}
  __device__ __forceinline__ bool next(Seg& s) {
    while (w < hi) {
      while (w - base >= size) {   // the line covers w: a request with tiles follows
        base += size;
        ++b;
        r = load_req<TK>(a, b);
        size = line_of<PAD>(a, r);
      }
      const int64_t off = w - base;
      const int span = r.tiles + PAD;            // PAD places, then the tiles
      const int64_t item = quot(off, span);
      const int at = static_cast<int>(off - item * span);
      const int to = static_cast<int>(min(int64_t(span), at + (hi - w)));
      w += to - at;
      if (to <= PAD) continue;                   // no tile of it: the next CTA begins it
      s.r = r;
      s.b = b;
      s.t0 = max(at - PAD, 0);
      s.t1 = to - PAD;
      s.h = static_cast<int>(quot(item, r.rts));
      s.rt = static_cast<int>(item - int64_t(s.h) * r.rts);
      s.first = base + item * span + PAD;
      s.end = base + (item + 1) * span;
      return true;
    }
    return false;
  }
};

// Whether a row (new token i, mask words mw) sees new token j.
__device__ __forceinline__ bool sees(const Args& a, const uint64_t* mw, int i, int j, int n) {
  if (j >= n) return false;
  if (a.mask == nullptr) return j <= i;
  return (j >> 6) < a.mask_words && ((mw[j >> 6] >> (j & 63)) & 1);
}

// The first word of a row's mask, which covers most trees: read with the row's
// queries, so that the tiles of new tokens do not wait for it.
__device__ __forceinline__ uint64_t first_word(const Args& a, const uint64_t* mw) {
  return a.mask != nullptr ? __ldg(mw) : 0;
}

// The same for the N (16 or 32) keys from position k0 on, as bits: cached keys
// are seen, keys past the request's last are not.
template <int N>
__device__ __forceinline__ uint32_t sees_bits(const Args& a, const uint64_t* mw, uint64_t word0,
                                              int i, int k0, int ctx, int len) {
  const int j0 = k0 - ctx;              // k0 as a new token, below 0: cached
  const int lo = max(j0, 0), skip = min(lo - j0, N);
  uint64_t x = 0;
  if (skip < N) {
    if (a.mask == nullptr) {
      const int up = i - lo + 1;          // new tokens lo .. i
      x = up <= 0 ? 0 : up >= N ? 0xFFFFFFFFu : (1u << up) - 1;
    } else {
      const int w = lo >> 6, sh = lo & 63;
      if (w < a.mask_words) x = (w == 0 ? word0 : mw[w]) >> sh;
      if (sh > 64 - N && w + 1 < a.mask_words) x |= mw[w + 1] << (64 - sh);
    }
  }
  const uint64_t bits = (x << skip) | ((uint64_t(1) << skip) - 1);
  const int valid = min(max(len - k0, 0), N);
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

// The rare paths are functions of their own, not inlined: a kernel whose loop
// does not fit the instruction cache fetches it again from an L2 that its
// copies keep busy, 1.5 us a miss.

// sees_bits for 64 keys, and for 16.
__device__ __noinline__ uint64_t sees64(const Args& a, const uint64_t* mw, uint64_t word0, int i,
                                        int k0, int ctx, int len) {
  return sees_bits<32>(a, mw, word0, i, k0, ctx, len) |
         static_cast<uint64_t>(sees_bits<32>(a, mw, word0, i, k0 + 32, ctx, len)) << 32;
}
__device__ __noinline__ uint32_t sees16(const Args& a, const uint64_t* mw, uint64_t word0, int i,
                                        int k0, int ctx, int len) {
  return sees_bits<16>(a, mw, word0, i, k0, ctx, len);
}

// Values of a tile (64-column parts `part` bytes apart, rows of 128 swizzled
// bytes) in rows [r0, r1), of which row 0 is key k0: those past the request's
// last token become zero, and so do non-finite ones of new tokens, which
// s_bad (by token) and s_any_bad note; add_bad adds them to the rows that see
// them.  For `count` threads.
template <bool BF16, int D>
__device__ __noinline__ void clean_values(uint8_t* tile, int part, int k0, int r0, int r1, int ctx,
                                          int len, int thread, int count, unsigned int* s_bad,
                                          int* s_any_bad) {
  r0 = max(r0, ctx - k0);
#pragma unroll 1
  for (int i = thread; i < (r1 - r0) * (D / 8); i += count) {
    const int r = r0 + i / (D / 8), c = i % (D / 8);
    uint4* at = reinterpret_cast<uint4*>(tile + (c >> 3) * part + r * 128 + (((c & 7) ^ (r & 7)) << 4));
    if (k0 + r >= len) {
      *at = make_uint4(0, 0, 0, 0);
      continue;
    }
    uint4 x = *at;
    uint32_t bad = 0;
    uint32_t* xw = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t b = nonfinite2<BF16>(xw[e]);
      if (b & 1) xw[e] &= 0xFFFF0000u;
      if (b & 2) xw[e] &= 0x0000FFFFu;
      bad |= b;
    }
    if (bad) {
      *at = x;
      const int j = k0 + r - ctx;
      if (j < 256) atomicOr(&s_bad[j >> 5], 1u << (j & 31));
      *s_any_bad = 1;
    }
  }
  ptx::fence_proxy_async_smem();   // before an MMA's reading and the ring's next copy
}

// Adds the non-finite values of the new tokens that a row sees to columns
// [d0, d0 + n_cols) of what this thread stored for the row: its output
// (`out`), or its part of a piece (`part`, four columns every `step` floats).
template <bool BF16>
__device__ __noinline__ void add_bad(const Args& a, const unsigned int* s_bad, int b, int h, int ctx,
                                     int n, int row0, int token, int d0, int n_cols, uint16_t* out,
                                     float* part, int step) {
  const uint64_t* mw = a.mask != nullptr ? a.mask + (row0 + int64_t(token)) * a.mask_words : nullptr;
#pragma unroll 1
  for (int j = 0; j < min(n, 256); ++j) {
    if (!((s_bad[j >> 5] >> (j & 31)) & 1) || !sees(a, mw, token, j, n)) continue;
    const int64_t pos = int64_t(ctx) + j;
    const int pg = a.table[int64_t(b) * a.table_stride + (pos >> a.page_shift)];
    if (pg < 0 || pg >= a.pages) continue;
    const uint16_t* v = a.v + int64_t(pg) * a.page_stride +
                        (pos & ((1 << a.page_shift) - 1)) * a.token_stride + int64_t(h) * a.head_stride + d0;
#pragma unroll 1
    for (int d = 0; d < n_cols; ++d) {
      if (!(nonfinite2<BF16>(v[d]) & 1)) continue;
      if (out != nullptr)
        out[d] = static_cast<uint16_t>(pack2<BF16>(widen<BF16>(out[d]) + widen<BF16>(v[d]), 0.f));
      else
        part[d / 4 * step + d % 4] += widen<BF16>(v[d]);
    }
  }
}

constexpr float kLn2 = 0.69314718055994530942f;

// The reference that a row's exponents are taken from is its maximum less this
// much: 2^7 is then the largest probability when the reference is set and 2^15
// before it moves on.  fp16 has no numbers below 2^-24 and loses bits below
// 2^-14, so that with the maximum itself a probability of 2^-24.6 counted half as
// much again and one of 2^-25 nothing, beside a sum that had both; so it is off
// by at most 2^-32 of the largest, or relatively as the type rounds.  bf16 has
// the exponents of 32 bits.
template <bool BF16>
constexpr float kLift = BF16 ? 0.f : 7.f;

// lse of a row with a sum l > 0 referred to m (which is less by kLift than the
// maximum).
template <bool BF16>
__device__ __forceinline__ float lse_of(float m, float l) {
  if constexpr (BF16) return (m + log2f(l)) * kLn2;
  return ((m + kLift<BF16>) + log2f(l * (1.f / 128.f))) * kLn2;
}

// ------------------------------------------------------------------ join
//
// out = sum 2^(m_i - m) out_i / sum 2^(m_i - m) l_i over the pieces of an item
// that several CTAs share: slot 1 of CTA `first`, then slot 0 of the next
// `follow` CTAs.  Each CTA stores its piece and counts itself; whoever counts
// last adds all pieces, in the order of the keys, so the result does not
// depend on who that was.  From JOIN_ALL pieces on they are first added in
// groups of about their square root, by each group's last, then the groups:
// one long context on one key head makes hundreds.  For up to 16 rows: with
// more, adding up is work for more than one SM.
constexpr int JOIN_ALL = 24;

// An item that several CTAs share.
struct Item {
  int first, follow;        // CTAs: the one that begins it, and how many follow
  int row0, r0, rows, head; // first row of the request and of the tile, its rows, key head
};

// One piece more to a running (m, l, o).
__device__ __forceinline__ void add_piece(float& m, float& l, float4& o, float2 ml, float4 x) {
  const float mn = fmaxf(m, ml.x), ms = mn == -INFINITY ? 0.f : mn;
  const float f = ex2(m - ms), e = ex2(ml.x - ms);
  m = mn;
  l = l * f + ml.y * e;
  o = make_float4(o.x * f + x.x * e, o.y * f + x.y * e, o.z * f + x.z * e, o.w * f + x.w * e);
}

// Four columns of a joined row to the output.
template <bool BF16, int D>
__device__ __forceinline__ void write_joined(const Args& a, const Item& it, int r, int d4, float m,
                                             float l, float4 o) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int token = div_group(a, it.r0 + r);
  const int head = it.head * a.group + (it.r0 + r - token * a.group);
  const int64_t at = (int64_t(it.row0) + token) * a.Hq + head;
  *reinterpret_cast<uint2*>(a.out + at * D + d4 * 4) =
      make_uint2(pack2<BF16>(o.x * inv, o.y * inv), pack2<BF16>(o.z * inv, o.w * inv));
  if (d4 == 0 && a.lse != nullptr)
    a.lse[at] = l == 0.f ? -INFINITY : lse_of<BF16>(m, l);
}

// The one or two items whose parts a CTA stored (the first and the last of its
// piece), after both: N threads with `tid` 0 .. N - 1, synchronised by named
// barrier 1.
template <bool BF16, int D, int RT, int N>
__device__ __forceinline__ void join_pieces(const Args& a, const Item (&items)[2], int n, int tid,
                                            int* s_last) {
  const int grid = static_cast<int>(gridDim.x);
  const auto slot_of = [](const Item& it, int i) { return 2 * (int64_t(it.first) + i) + (i == 0 ? 1 : 0); };
  const auto group_of = [](const Item& it) {     // pieces that are added first
    int size = it.follow + 1;
    if (size >= JOIN_ALL) {
      size = 5;
      while (size * size < it.follow + 1) ++size;
    }
    return size;
  };
  // Counts one arrival each; which were the last ones, for every thread.  The
  // barrier and thread 0's fence publish what all of them stored.
  const auto count = [&](int* c0, int all0, int* c1, int all1) {
    ptx::named_sync(1, N);
    if (tid == 0) {
      __threadfence();
      const int at0 = atomicAdd(c0, 1);
      const int at1 = c1 != nullptr ? atomicAdd(c1, 1) : -2;
      const int last = (at0 == all0 - 1 ? 1 : 0) | (at1 == all1 - 1 ? 2 : 0);
      if (last & 1) *c0 = 0;
      if (last & 2) *c1 = 0;
      __threadfence();
      *s_last = last;
    }
    ptx::named_sync(1, N);
    return *reinterpret_cast<volatile int*>(s_last);
  };
  // pieces i0, i0 + step, .. below i1: to the output, or as the group's sum to
  // piece i0's place.  A group's (m, l) has a place of its own, 2 grid slots
  // on, since every column's thread reads the piece's.
  const auto add_up = [&](const Item& it, int i0, int i1, int step, bool out) {
    const int64_t sums = step > 1 ? 2 * int64_t(grid) : 0;
    // a thread has W groups of four columns of a row: with 16 rows or fewer
    // nearly everything is read at once
    constexpr int W = 4, CG = D / 4 / W;
#pragma unroll 1
    for (int p = tid; p < it.rows * CG; p += N) {
      const int c = p / it.rows, r = p - c * it.rows;
      float m = -INFINITY, l = 0.f;
      float4 o[W];
#pragma unroll
      for (int k = 0; k < W; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
      for (int i = i0; i < i1; i += step) {
        const int64_t slot = slot_of(it, i);
        const float2 ml = __ldcg(a.part_ml + (sums + slot) * RT + r);
        float4 x[W];
#pragma unroll
        for (int k = 0; k < W; ++k)
          x[k] = __ldcg(reinterpret_cast<const float4*>(a.part_o + ((slot * (D / 4) + c + k * CG) * RT + r) * 4));
        const float m0 = m, l0 = l;
#pragma unroll
        for (int k = 0; k < W; ++k) {
          m = m0;
          l = l0;
          add_piece(m, l, o[k], ml, x[k]);
        }
      }
      if (out) {
#pragma unroll
        for (int k = 0; k < W; ++k) write_joined<BF16, D>(a, it, r, c + k * CG, m, l, o[k]);
      } else {
        const int64_t slot = slot_of(it, i0);
#pragma unroll
        for (int k = 0; k < W; ++k)
          *reinterpret_cast<float4*>(a.part_o + ((slot * (D / 4) + c + k * CG) * RT + r) * 4) = o[k];
        if (c == 0) a.part_ml[(2 * int64_t(grid) + slot) * RT + r] = make_float2(m, l);
      }
    }
  };
  // where item k's arrival is counted first, and how many are awaited there
  const auto first_count = [&](const Item& it, int*& c, int& all) {
    const int size = group_of(it), pieces = it.follow + 1;
    const int i0 = (static_cast<int>(blockIdx.x) - it.first) / size * size;
    c = size == pieces ? a.arrived + it.first : a.arrived + grid + slot_of(it, i0);
    all = min(size, pieces - i0);
  };
  int *c0 = nullptr, *c1 = nullptr, all0 = 0, all1 = 0;
  first_count(items[0], c0, all0);
  if (n > 1) first_count(items[1], c1, all1);
  const int last = count(c0, all0, c1, all1);
#pragma unroll 1
  for (int k = 0; k < n; ++k) {
    if (!((last >> k) & 1)) continue;
    const Item it = k == 0 ? items[0] : items[1];
    const int size = group_of(it), pieces = it.follow + 1;
    const int i0 = (static_cast<int>(blockIdx.x) - it.first) / size * size;
    int from = i0, to = min(i0 + size, pieces), step = 1;
    bool out = size == pieces;
#pragma unroll 1
    while (true) {
      add_up(it, from, to, step, out);
      if (out || !(count(a.arrived + it.first, (pieces + size - 1) / size, nullptr, 0) & 1)) break;
      from = 0;
      to = pieces;
      step = size;
      out = true;
    }
  }
}

}  // namespace attn
}  // namespace tern
