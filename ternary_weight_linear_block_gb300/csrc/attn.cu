// Attention of drafted tokens over the paged cache.
//
// For a row (new token with a query head) over the keys j that it sees:
//   t_j = scale log2(e) q . k_j,  m = max t_j,  l = sum 2^(t_j - m),
//   out = sum 2^(t_j - m) v_j / l,  lse = (m + log2 l) ln 2,
// kept over the tiles of a piece as (m, l, unnormalised out) in 32 bits and
// rescaled where m grows.  The probabilities are rounded to the cache's type
// for the second product, as its values are (the matrix instructions take both
// operands in one type, and splitting a probability into two would double that
// product); l sums them unrounded.  m is less than the maximum by kLift.
//
// attn_rows_kernel: up to 16 rows an item, tiles of 64 keys.  A producer warp
// copies each page's part of a tile with TMA into a ring; four warps take 16
// keys of a tile each and keep their own (m, l, out) of all the item's rows,
// so that no warp waits for another inside an item; they join at its end.
// The products are mma.sync m16n8k16 with the keys (and the values' columns)
// on the 16 side and 8 rows on the other: one to eight rows cost one
// instruction of a tile, not two of which half is padding, and each
// ldmatrix of keys or values serves all the rows.
// Bound: the keys and values, read once (64 requests of up to 16001 keys, 8
// heads of 128, 4 query heads on each: 2.63 GB in 397 us, 6.62 TB/s, 0.99 of a
// copy's rate); a small call starts, finds its pieces and joins them beside that
// (16 requests of up to 700 keys, 20 heads of 128: 70 MB in 21.8 us, of which
// 10.5 at copy rate, and 16.3 where L2 has the keys; 4 requests of 3 keys, heads
// of 64, 5.4 us).  A second kernel that joins the pieces, in place of the last CTA
// to arrive, took 22.6 us against 19.7.
#include <algorithm>

#include "attn_tile.cuh"

namespace tern {

__device__ unsigned int g_attn_error;

namespace {

using namespace attn;

__device__ __forceinline__ void fail(volatile int* abort_flag, unsigned int code) {
  *abort_flag = 1;
  atomicOr(&g_attn_error, code);
}

// ------------------------------------------------------------------ rows kernel

constexpr int TK = 64;             // keys of a tile
constexpr int NW = 4;              // warps that share a tile's keys, 16 each

// NT: eights of rows in an item.  The accumulators (D / 4 * NT registers a
// thread) and the query fragments (D / 8 * NT) decide how many CTAs an SM
// holds, and so the ring's size.  Joining the warps takes two buffers of the
// item's rows, `COLS` columns of them at a time.
template <int D, int NT>
struct Rows {
  static constexpr int RT = 8 * NT;
  // an item's cost beside its tiles, which also bounds a piece (LEAST).  8 heads
  // of 128, 16 rows: 2 requests of up to 20000 keys 35.7 us with 1, 32.6 with 3, 29.9
  // with 6, but 1 of 1000 keys 14.5 with 3 and 17.8 with 6
  static constexpr int PAD = D == 64 ? 4 : 3;
  static constexpr int LEAST = PAD + 1;                   // places of a CTA's piece at least
  static constexpr int THREADS = (NW + 2) * 32;           // and a producer each of K and V
  static constexpr int STAGE = 2 * TK * D * 2;            // keys and values of a tile
  static constexpr int CTAS = D < 256 ? 2 : 1;            // per SM
  static constexpr int COLS = D * NT <= 128 || NT == 1 ? D : D / 2;
  static constexpr int LD = COLS + 4;                     // no two lanes of a store share a bank
  static constexpr int MERGE = 2 * RT * LD * 4;
  static constexpr int QLD = D * 2 + 16;                  // bytes of a query row
  static constexpr int QBYTES = RT * QLD;
  static constexpr int ROOM = (CTAS == 2 ? 115200 : 232448) - MERGE - QBYTES - 1024 - 1536;
  static constexpr int FIT = ROOM / STAGE;
  static constexpr int STAGES = FIT < 8 ? FIT : 8;
  static constexpr size_t SMEM = size_t(STAGES) * STAGE + MERGE + QBYTES + 1024;
  static_assert(STAGES >= 2, "ring");
};

// Keys or values of tile t into `dst` (64-column halves of TKEYS rows of 128
// swizzled bytes), one box and half a lane; the warp first announces the
// bytes on `bar`.
template <int D, int TKEYS>
__device__ __forceinline__ void load_tile(const Args& a, const CUtensorMap* map, uint8_t* dst,
                                          uint64_t* bar, const Seg& s, int t, int page,
                                          int box_shift, int lane) {
  constexpr int HALVES = D / 64;
  const int k0 = t * TKEYS;
  const int keys = min(TKEYS, s.r.len - k0);
  const int boxes = keys > 0 ? (keys + (1 << box_shift) - 1) >> box_shift : 0;
  if (lane == 0)
    ptx::mbar_arrive_expect_tx(bar, static_cast<uint32_t>(boxes << box_shift) * D * 2u);
  __syncwarp();
  const int box = lane / HALVES, half = lane % HALVES;   // at most 32: 8 keys a box or more
  const int pg = __shfl_sync(~0u, page, box);
  if (box < boxes)
    tma_load_4d(dst + half * (TKEYS * 128) + (box << box_shift) * 128, map, bar, half * 64,
                k0 & ((1 << a.page_shift) - 1), s.h, pg);
}

template <bool BF16, int D, int NT>
__global__ void __launch_bounds__((Rows<D, NT>::THREADS), (Rows<D, NT>::CTAS))
    attn_rows_kernel(const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Args a) {
  using C = Rows<D, NT>;
  constexpr int RT = C::RT, THREADS = C::THREADS;
  constexpr int HALVES = D / 64;
  constexpr int HB = TK * 128;
  constexpr int KS = D / 16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  float* merge = reinterpret_cast<float*>(ring + C::STAGES * C::STAGE);
  uint8_t* sq = ring + C::STAGES * C::STAGE + C::MERGE;
  __shared__ uint64_t full[C::STAGES], empty[C::STAGES], q_full, q_empty;
  __shared__ __align__(16) Part s_part;
  __shared__ uint64_t s_word0[RT];      // of each row's mask
  __shared__ PieceScratch<THREADS> scratch;
  __shared__ float2 s_ml[NW][RT];
  __shared__ unsigned int s_bad[8];     // new tokens with a non-finite value, by index
  __shared__ int s_any_bad, s_last;
  __shared__ int s_abort;
  volatile int* abort_flag = &s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      ptx::mbar_init(&full[s], 2);
      ptx::mbar_init(&empty[s], NW);
    }
    ptx::mbar_init(&q_full, 1);
    ptx::mbar_init(&q_empty, NW);
    s_abort = 0;
    s_any_bad = 0;
    for (int i = 0; i < 8; ++i) s_bad[i] = 0;
    ptx::mbar_fence_init();
    ptx::prefetch_tmap(&tm_k);
    ptx::prefetch_tmap(&tm_v);
  }
  pdl_wait();
  pdl_launch_dependents();
  const Piece piece = find_piece<TK, C::PAD, C::LEAST, THREADS>(a, scratch);   // synchronises the CTA
  if (piece.lo >= piece.hi) return;

  if (warp >= NW) {
    // ---------------- producers: one warp copies the keys, one the values
    // (issued by one warp, pages of 16 rows held a long context to two thirds
    // of its rate).  The keys' also copies each item's queries and says what
    // the item is, while the consumers are still at the one before: found out
    // by themselves, that was a third of a short item's time.
    const bool vals = warp > NW;
    const CUtensorMap* map = vals ? &tm_v : &tm_k;
    Walk<TK, C::PAD> walk(a, piece);
    Seg s{};
    int st = 0;
    uint32_t phase = 0, q_phase = 1;
    long issued = 0, q_issued = 0;
    bool ok = true;
    const int box_shift = min(a.page_shift, 6);      // rows of a box: a page, or the tile
    const auto give_up = [&](bool good) {
      if (!good && lane == 0 && !*abort_flag) fail(abort_flag, ERR_PRODUCER);
      return good;
    };
    uint64_t word0 = 0;      // lane r: of the mask of the item's row r
    const auto rows_of = [&] { return min(RT, s.r.n * a.group - s.rt * RT); };
    // the item's queries, once the one before needs its own no more
    const auto post_queries = [&] {
      ok = give_up(ptx::mbar_wait_warp(&q_empty, q_phase, abort_flag, WAIT_LIMIT));
      if (!ok) return;
      q_phase ^= 1u;
      ++q_issued;
      const int r = s.rt * RT + lane;
      if (lane < rows_of()) {
        const int tok = div_group(a, r);
        ptx::bulk_load(sq + lane * C::QLD,
                       a.q + (s.r.row0 + int64_t(tok)) * a.q_token +
                           int64_t(s.h * a.group + (r - tok * a.group)) * a.q_head,
                       D * 2, &q_full);
      }
    };
    // what the item is, or (none) that there is no further one
    const auto post = [&](bool item) {
      const int rows = item ? rows_of() : 0;
      if (lane < rows) s_word0[lane] = word0;
      if (lane == 0) {
        const bool whole = s.t0 == 0 && s.t1 == s.r.tiles;
        const int first = whole ? 0 : cta_of(piece, s.first);
        s_part = Part{s.b, s.h, s.rt * RT, rows, s.r.row0, s.r.ctx, s.r.n, s.r.len, s.t0,
                      item ? s.t1 : s.t0, whole, s.t0 == 0, first,
                      whole ? 0 : cta_of(piece, s.end - 1) - first, {0, 0}};
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_expect_tx(&q_full, static_cast<uint32_t>(rows) * D * 2);
    };
    while (ok && walk.next(s)) {
      int page = page_at<TK>(a, s, s.t0, box_shift, lane);
      if (!vals && a.mask != nullptr && lane < rows_of())
        word0 = a.mask[(s.r.row0 + int64_t(div_group(a, s.rt * RT + lane))) * a.mask_words];
      // the queries go first where their place is free (a CTA's first item:
      // they are on their way while the page numbers are), else after a tile
      bool posted = vals;
      if (!vals && __all_sync(~0u, ptx::mbar_test_wait(&q_empty, q_phase))) {
        post_queries();
        posted = true;
      }
      for (int t = s.t0; t < s.t1 && ok; ++t) {
        const int ahead = t + 1 < s.t1 ? page_at<TK>(a, s, t + 1, box_shift, lane) : 0;
        ok = give_up(ptx::mbar_wait_warp(&empty[st], phase ^ 1u, abort_flag, WAIT_LIMIT));
        if (!ok) break;
        load_tile<D, TK>(a, map, ring + st * C::STAGE + (vals ? HALVES * HB : 0), &full[st], s, t,
                         page, box_shift, lane);
        page = ahead;
        ++issued;
        if (++st == C::STAGES) {
          st = 0;
          phase ^= 1u;
        }
        if (!vals && t == s.t0) {
          if (!posted) post_queries();
          if (ok) post(true);
        }
      }
    }
    if (ok && !vals) {
      ok = give_up(ptx::mbar_wait_warp(&q_empty, q_phase, abort_flag, WAIT_LIMIT));
      if (ok) post(false);
    }
    // something gave up: the copies land before the CTA exits
    const long back = ok && !*abort_flag ? 0 : issued < C::STAGES ? issued : C::STAGES;
    for (long i = 0; i < back; ++i) {
      if (--st < 0) {
        st = C::STAGES - 1;
        phase ^= 1u;
      }
      if (!ptx::mbar_wait_bounded(&full[st], phase, WAIT_LIMIT)) atomicOr(&g_attn_error, ERR_DRAIN);
    }
    if (q_issued > 0 && (!ok || *abort_flag) && !ptx::mbar_wait_bounded(&q_full, q_phase, WAIT_LIMIT))
      atomicOr(&g_attn_error, ERR_DRAIN);
    return;
  }

  // ---------------- consumers: warp w has keys 16 w .. 16 w + 15 of each tile
  int st = 0;
  uint32_t phase = 0;
  const uint32_t ring_u = ptx::smem_u32(ring);
  const int row_b = lane >> 2;           // query row (of 8) whose fragment this lane holds
  const int row_c = (lane & 3) * 2;      // score rows of this lane: row_c, row_c + 1
  // ldmatrix: keys (matrices: keys 0-7 d 0-7, keys 8-15 d 0-7, keys 0-7 d 8-15, ...)
  const int k_row = warp * 16 + (lane & 15);
  const int k_chunk = lane >> 4;
  // values transposed (matrices: keys 0-7 d 0-7, keys 0-7 d 8-15, keys 8-15 d 0-7, ...)
  const int v_row = warp * 16 + (lane & 7) + ((lane >> 4) << 3);
  const int v_chunk = (lane >> 3) & 1;
  bool ok = true;
  uint32_t q_phase = 0;
  Item joins[2];
  int n_joins = 0;
  while (true) {
    ok = ok && ptx::mbar_wait_warp(&q_full, q_phase, abort_flag, WAIT_LIMIT);
    q_phase ^= 1u;
    // all four warps go on or none does (and the buffers below are free again)
    if (named_any(1, NW * 32, !ok)) {
      if (lane == 0 && !*abort_flag) fail(abort_flag, ERR_CONSUMER);
      break;
    }
    const Part s = s_part;
    if (s.t1 <= s.t0) break;
    const int rows = s.rows, r0 = s.r0;
    // query fragments (rows past the item's last are what the place held
    // before: they reach only their own scores), and of this lane's score
    // rows the new token and its mask's first word
    uint32_t qf[KS][NT][2];
    int tok[NT][2];
    uint64_t word0[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint8_t* q = sq + (n * 8 + row_b) * C::QLD + (lane & 3) * 4;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qf[k][n][0] = *reinterpret_cast<const uint32_t*>(q + k * 32);
        qf[k][n][1] = *reinterpret_cast<const uint32_t*>(q + k * 32 + 16);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = n * 8 + row_c + e;
        tok[n][e] = r < rows ? div_group(a, r0 + r) : 0;
        word0[n][e] = r < rows ? s_word0[r] : 0;
      }
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&q_empty);
    float o[KS][NT][4];
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
    }

    for (int t = s.t0; t < s.t1; ++t) {
      const int k0 = t * TK + warp * 16;         // this warp's first key
      const bool edge = k0 > s.ctx - 16;     // new tokens, or past the last
      uint32_t vis[NT][2];
      if (edge) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            vis[n][e] = sees16(a, a.mask + (s.row0 + int64_t(tok[n][e])) * a.mask_words,
                               word0[n][e], tok[n][e], k0, s.ctx, s.len);
      }
      // a warp whose wait gave up reads no more tiles, but still meets the
      // others at the barriers below
      if (ok) {
        ok = ptx::mbar_wait_warp(&full[st], phase, abort_flag, WAIT_LIMIT);
        if (!ok && lane == 0 && !*abort_flag) fail(abort_flag, ERR_CONSUMER);
      }
      if (!ok) break;
      const uint32_t kbase = ring_u + st * C::STAGE;
      const uint32_t vbase = kbase + HALVES * HB;
      if (k0 < s.len || k0 == 0) {     // else past the last token: nothing to add
        if (edge) {
          clean_values<BF16, D>(ring + st * C::STAGE + HALVES * HB, HB, t * TK, warp * 16,
                                warp * 16 + 16, s.ctx, s.len, lane, 32, s_bad, &s_any_bad);
          __syncwarp();
        }
        float c[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t x[4];
          const int chunk = (k & 3) * 2 + k_chunk;
          ldsm_x4(kbase + (k >> 2) * HB + k_row * 128 + ((chunk ^ (k_row & 7)) << 4), x);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816<BF16>(c[n], x, qf[k][n][0], qf[k][n][1]);
        }
        // c[n]: keys lane / 4 and + 8, rows row_c and + 1
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            c[n][e] *= a.scale_log2;
            if (edge && !((vis[n][e & 1] >> (row_b + (e >> 1) * 8)) & 1)) c[n][e] = -INFINITY;
          }
        float al[NT][2];
        bool moved = false;
        uint32_t p[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float ms[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = fmaxf(c[n][e], c[n][e + 2]);
            x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
            x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
            x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
            const float mn = fmaxf(m[n][e], x - kLift<BF16>);
            ms[e] = mn == -INFINITY ? 0.f : mn;
            al[n][e] = ex2(m[n][e] - ms[e]);
            moved |= mn != m[n][e];
            m[n][e] = mn;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) c[n][e] = ex2(c[n][e] - ms[e & 1]);
#pragma unroll
          for (int e = 0; e < 2; ++e) l[n][e] = l[n][e] * al[n][e] + (c[n][e] + c[n][e + 2]);
          p[n][0] = movm(pack2<BF16>(c[n][0], c[n][1]));
          p[n][1] = movm(pack2<BF16>(c[n][2], c[n][3]));
        }
        if (__any_sync(~0u, moved)) {
#pragma unroll
          for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[i][n][e] *= al[n][e & 1];
        }
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          uint32_t x[4];
          const int chunk = (i & 3) * 2 + v_chunk;
          ldsm_x4_t(vbase + (i >> 2) * HB + v_row * 128 + ((chunk ^ (v_row & 7)) << 4), x);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816<BF16>(o[i][n], x, p[n][0], p[n][1]);
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&empty[st]);
      if (++st == C::STAGES) {
        st = 0;
        phase ^= 1u;
      }
    }

    // ---- join the four warps: factors from every warp's (m, l); two of them
    // store, the other two add to what they stored, and the two sums are added
    // as they are read
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[n][e] += __shfl_xor_sync(~0u, l[n][e], 4);
        l[n][e] += __shfl_xor_sync(~0u, l[n][e], 8);
        l[n][e] += __shfl_xor_sync(~0u, l[n][e], 16);
        if (lane < 4) s_ml[warp][n * 8 + row_c + e] = make_float2(m[n][e], l[n][e]);
      }
    ptx::named_sync(1, NW * 32);
    float f[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) mm = fmaxf(mm, s_ml[w][n * 8 + row_c + e].x);
        f[n][e] = mm == -INFINITY ? 0.f : ex2(m[n][e] - mm);
      }
    const bool whole = s.whole != 0;
    const int64_t slot = 2 * int64_t(blockIdx.x) + s.begins;
    const bool any_bad = *reinterpret_cast<volatile int*>(&s_any_bad) != 0;
    float* mine = merge + (warp & 1) * (RT * C::LD);
#pragma unroll
    for (int c0 = 0; c0 < D; c0 += C::COLS) {
      if (c0 > 0) ptx::named_sync(1, NW * 32);
#pragma unroll 1
      for (int round = 0; round < 2; ++round) {
        if ((warp >> 1) == round) {
#pragma unroll
          for (int i = 0; i < C::COLS / 16; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float* at = mine + (n * 8 + row_c + (e & 1)) * C::LD + i * 16 + row_b + (e >> 1) * 8;
                float x = o[c0 / 16 + i][n][e] * f[n][e & 1];
                if (round > 0) x += *at;
                *at = x;
              }
        }
        ptx::named_sync(1, NW * 32);
      }
      // ---- write: thread -> 4 consecutive values of a row
#pragma unroll 1
      for (int i = tid; i < RT * (C::COLS / 4); i += NW * 32) {
        const int r = i % RT, dc = i / RT * 4, d = c0 + dc;
        if (r >= rows) continue;
        float4 x = *reinterpret_cast<const float4*>(merge + r * C::LD + dc);
        const float4 y = *reinterpret_cast<const float4*>(merge + (RT + r) * C::LD + dc);
        x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
        const int token = div_group(a, r0 + r), head = s.h * a.group + (r0 + r - token * a.group);
        float mm = -INFINITY, ll = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) mm = fmaxf(mm, s_ml[w][r].x);
#pragma unroll
        for (int w = 0; w < NW; ++w)
          ll += s_ml[w][r].y * (mm == -INFINITY ? 0.f : ex2(s_ml[w][r].x - mm));
        if (whole) {
          const float inv = ll == 0.f ? 0.f : 1.f / ll;
          const int64_t at = (int64_t(s.row0) + token) * a.Hq + head;
          *reinterpret_cast<uint2*>(a.out + at * D + d) =
              make_uint2(pack2<BF16>(x.x * inv, x.y * inv), pack2<BF16>(x.z * inv, x.w * inv));
          if (d == 0 && a.lse != nullptr)
            a.lse[at] = ll == 0.f ? -INFINITY : lse_of<BF16>(mm, ll);
        } else {
          *reinterpret_cast<float4*>(a.part_o + ((slot * (D / 4) + d / 4) * RT + r) * 4) = x;
          if (d == 0) a.part_ml[slot * RT + r] = make_float2(mm, ll);
        }
        if (any_bad)
          add_bad<BF16>(a, s_bad, s.b, s.h, s.ctx, s.n, s.row0, token, d, 4,
                        whole ? a.out + ((int64_t(s.row0) + token) * a.Hq + head) * D + d : nullptr,
                        a.part_o + ((slot * (D / 4) + d / 4) * RT + r) * 4, 4);
      }
    }
    if (!whole) {
      const Item it{s.first, s.follow, s.row0, r0, rows, s.h};
      if (n_joins++ == 0) joins[0] = it; else joins[1] = it;
    }
    if (any_bad) {
      ptx::named_sync(1, NW * 32);
      if (tid < 8) s_bad[tid] = 0;
      if (tid == 0) s_any_bad = 0;
    }
  }
  if (n_joins > 0) join_pieces<BF16, D, RT, NW * 32>(a, joins, n_joins, tid, &s_last);
}

// ------------------------------------------------------------------ tile kernel
//
// Up to 128 or 256 rows an item (whole tokens: 128 / group of them a stream)
// on tcgen05: S = Q K^T with 128 rows on the M
// side, the accumulator in tensor memory; a thread reads one row of S, writes
// the row's probabilities over it as 16-bit values, and out += P V takes P
// from tensor memory and V from the ring as its pages hold it (columns of V
// along the MMA's N side: the MN-major operand).  Keys and values arrive in a
// ring of slots in the order K0 K1 V0 K2 V1 K3 ...
//
// Two warpgroups, so that one's softmax runs beside the MMAs for the other:
//   SHARED rows <= 128: they take the key tiles in turn and share the out
//          accumulator.  A row's reference maximum goes from one to the other
//          through shared memory, tile by tile, and whoever has to move it
//          waits for the MMA before and rescales.  S has three buffers and
//          runs two tiles ahead.  (An accumulator for each, joined at the end,
//          measured the same with head size 128 and 64; with 256 columns it
//          does not fit, and a half of the columns for each, S computed twice,
//          took 109 us against 82 on 8 requests of up to 20003 keys.)
//   ROWS   rows <= 256, head size 128: each has 128 rows with their own S and
//          accumulator (a stream); a key tile serves both.
// The maximum that a row's exponents refer to only moves when it grows by
// more than 2^8: until then nothing is rescaled (probabilities above one round
// as others do, kLift leaves fp16 room for them, and sums are in 32 bits), so the
// pass over the accumulator is rare.  Rows past the item's last cost their MMAs alone:
// whole warps of them skip the softmax.
//
// Bound: keys and values up to about 64 rows of head size 128 (a context of
// 131001 keys, 16 drafts, 8 heads of 128, 64 rows on each: 537 MB in 90 us,
// 6.0 TB/s, 0.89 of a copy's rate).  Above that each tile's chain of S, its
// softmax and P V, which two streams only partly hide from each other (4
// requests of 64 drafts over up to 32768 keys, 512 rows on each of 8 heads:
// 156 us, 930 TFLOP/s, 0.48 of the matrix rate; 8 requests of 29 drafts over up
// to 20003 keys, 232 rows on each of 2 heads of 256: 79 us, 525 TFLOP/s).  Short
// items are bound by filling and draining each part (16 requests of 23 drafts
// over up to 4099 keys, 16 heads of 64: 47 us, 3.9 TB/s).
// A tile of 128 rows and keys took a stream 3800 cycles when the first of these
// chains was 167 us: 1320 until S is there, 500 for the maximum, 1380 for the
// reference, the exponentials and P, the rest in handing over.  Measured and
// slower (512 rows): the streams' softmax in turns 257 us against 247 at that
// step; four warpgroups, two threads a row, 183 against 167; 64-key tiles with
// S two ahead 217; P V in two halves while the second is still exponents 171.
// For 64-wide heads two CTAs an SM took 66 us against 50.

constexpr int TILE_THREADS = 384;   // K producer, MMA, queries, V producer; two warpgroups
enum Mode { SHARED, ROWS };

template <int D, int MODE>
struct Tile {
  static constexpr int TKT = D == 256 ? 64 : 128;        // keys of a tile
  static constexpr int RT = MODE == ROWS ? 256 : 128;
  // an item's cost beside its tiles: 16 requests of up to 4099 keys, 16 heads of 64:
  // 51.2 us with 1, 47.6 with 3, 48.9 with 6
  static constexpr int PAD = D == 64 ? 3 : 2;
  static constexpr int LEAST = PAD + 1;                   // places of a CTA's piece at least
  static constexpr int SLOT = TKT * D * 2;
  static constexpr int QB = 128 * D * 2;                 // one Q tile
  static constexpr int QBYTES = MODE == ROWS ? 2 * QB : QB;
  static constexpr int FIT = (232448 - 1024 - 6144 - QBYTES) / SLOT;
  static constexpr int SLOTS = FIT < 8 ? FIT : 8;
  static constexpr size_t SMEM = size_t(SLOTS) * SLOT + QBYTES + 1024;
  static constexpr int AHEAD = MODE == SHARED ? 2 : 1;    // tiles that S runs ahead
  static constexpr int NS = MODE == SHARED ? 3 : 2;      // buffers of S
  static constexpr int S_STEP = MODE == SHARED ? TKT : 128;
  // accumulators: stream x at O_COL + 128 x; SHARED: one
  static constexpr uint32_t S_COL = 0, O_COL = MODE == SHARED && D < 256 ? 384 : 256;
  static_assert(SLOTS >= 4, "ring");
};

template <bool BF16, int D, int MODE>
__global__ void __launch_bounds__(TILE_THREADS, 1)
    attn_tile_kernel(const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ Args a) {
  using C = Tile<D, MODE>;
  constexpr int TKT = C::TKT, RT = C::RT, SLOTS = C::SLOTS, NS = C::NS;
  constexpr int HALVES = D / 64;
  constexpr int HB = TKT * 128;          // 64 columns of a key or value tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sq = ring + SLOTS * C::SLOT;
  __shared__ uint64_t full[SLOTS], empty[SLOTS], q_full, q_empty, o_full, done, s_full[NS], p_full[NS];
  // SHARED: out of an even or odd tile added (of the two, only one can be in
  // flight when its phase is awaited); a tile's maximum known
  __shared__ uint64_t o_step[2], m_ready[4];
  __shared__ float s_m[MODE == SHARED ? 128 : 1];
  __shared__ PieceScratch<TILE_THREADS> scratch;
  __shared__ float2 s_ml[2][128];
  __shared__ unsigned int s_bad[8];
  __shared__ int s_any_bad;
  __shared__ int s_abort;
  __shared__ uint32_t s_tmem;
  volatile int* abort_flag = &s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < SLOTS; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 1);
    }
    ptx::mbar_init(&q_full, 1);
    ptx::mbar_init(&q_empty, 1);
    ptx::mbar_init(&o_full, 1);
    ptx::mbar_init(&done, 1);
    for (int x = 0; x < NS; ++x) {
      ptx::mbar_init(&s_full[x], 1);
      ptx::mbar_init(&p_full[x], 4);
    }
    for (int e = 0; e < 2; ++e) ptx::mbar_init(&o_step[e], 1);
    for (int q = 0; q < 4; ++q) ptx::mbar_init(&m_ready[q], 1);
    s_abort = 0;
    s_any_bad = 0;
    for (int i = 0; i < 8; ++i) s_bad[i] = 0;
    ptx::mbar_fence_init();
    ptx::prefetch_tmap(&tm_k);
    ptx::prefetch_tmap(&tm_v);
    ptx::prefetch_tmap(&tm_q);
  }
  if (warp == 2) {
    ptx::tmem_alloc(&s_tmem, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  pdl_wait();
  pdl_launch_dependents();
  const Piece piece = find_piece<TKT, C::PAD, C::LEAST, TILE_THREADS>(a, scratch);   // synchronises the CTA
  ptx::tc_fence_after();
  const uint32_t tmem = s_tmem;
  if (tid == 128) a.items[blockIdx.x].follow = 0;   // the thread that may set it below
  const int stream_rows = MODE == ROWS ? a.tile_rows / 2 : a.tile_rows;   // at most 128
  Walk<TKT, C::PAD> walk(a, piece);
  Seg s{};

  if (warp == 0 || warp == 3) {
    // ---------------- producers: warp 0 copies the keys, warp 3 the values
    const bool vals = warp == 3;
    const CUtensorMap* map = vals ? &tm_v : &tm_k;
    uint32_t seq0 = 0;
    uint32_t mine = 0, parity = 0;      // slots this warp filled last, and their phases
    bool ok = true;
    const int box_shift = min(a.page_shift, TKT == 128 ? 7 : 6);
    while (ok && walk.next(s)) {
      const int cnt = s.t1 - s.t0;
      int page = page_at<TKT>(a, s, s.t0, box_shift, lane);
      for (int i = 0; i < cnt; ++i) {
        const int ahead = i + 1 < cnt ? page_at<TKT>(a, s, s.t0 + i + 1, box_shift, lane) : 0;
        const uint32_t n = seq0 + (vals ? v_place<C::AHEAD>(i, cnt) : k_place<C::AHEAD>(i));
        const uint32_t sl = n % SLOTS, par = (n / SLOTS) & 1u;
        ok = ptx::mbar_wait_warp(&empty[sl], par ^ 1u, abort_flag, WAIT_LIMIT);
        if (!ok) {
          if (lane == 0 && !*abort_flag) fail(abort_flag, ERR_PRODUCER);
          break;
        }
        load_tile<D, TKT>(a, map, ring + sl * C::SLOT, &full[sl], s, s.t0 + i, page, box_shift, lane);
        mine |= 1u << sl;
        parity = (parity & ~(1u << sl)) | (par << sl);
        page = ahead;
      }
      seq0 += 2u * cnt;
    }
    // something gave up: the copies land before the CTA exits
    for (int sl = 0; (!ok || *abort_flag) && sl < SLOTS; ++sl)
      if (((mine >> sl) & 1u) && !ptx::mbar_wait_bounded(&full[sl], (parity >> sl) & 1u, WAIT_LIMIT))
        atomicOr(&g_attn_error, ERR_DRAIN);
  } else if (warp == 1) {
    // ---------------- MMA issuer: the whole warp waits and counts, one elected
    // lane issues.  Counters are made uniform over the warp (shuffles, votes),
    // so that descriptors are built in uniform registers: issued from a
    // lane-dependent branch an MMA took 65 to 90 cycles, more than the 32 to
    // 64 that it runs.
    bool ok = true;
    uint32_t seq0 = 0, q_phase = 0, p_phase = 0;
    uint32_t tile0 = 0;      // tiles of the items before
    const auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!ok) return;
      ok = ptx::mbar_wait_warp(bar, parity, abort_flag, WAIT_LIMIT);
      if (!ok && lane == 0 && !*abort_flag) fail(abort_flag, ERR_CONSUMER);
      ptx::tc_fence_after();
    };
    // addresses stay below 2^18, so offsets add to a descriptor's address field
    const uint64_t q_desc = ptx::sw128_kmajor_desc(ptx::smem_u32(sq));
    const uint64_t k_desc = ptx::sw128_kmajor_desc(ptx::smem_u32(ring));
    const uint64_t v_desc = sw128_mn_desc(ptx::smem_u32(ring), HB);
    const uint32_t tm = __shfl_sync(~0u, tmem, 0);
    // a negative scale turns the queries' signs
    const uint32_t s_idesc = idesc<BF16>(TKT, false) | (a.scale_log2 < 0.f ? 1u << 13 : 0u);
    while (ok && __any_sync(~0u, walk.next(s))) {
      const int cnt = __shfl_sync(~0u, s.t1 - s.t0, 0);
      // S of stream x from the keys in slot sl (one lane): 16 values further
      // is 32 bytes (2 in the descriptor) in a swizzled row, or the next 64
      // columns
      const auto issue_s = [&](uint32_t sl, int i, int x, bool last) {
        const uint64_t da = q_desc + (MODE == ROWS ? x * (C::QB >> 4) : 0);
        const uint64_t db = k_desc + sl * (C::SLOT >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          ptx::mma_f16_ss(tm + C::S_COL + C::S_STEP * x,
                          da + ((k >> 2) * (128 * 128 >> 4) + 2 * (k & 3)),
                          db + ((k >> 2) * (HB >> 4) + 2 * (k & 3)), s_idesc, k > 0);
        if (last) ptx::mma_commit(&empty[sl]);
        ptx::mma_commit(&s_full[x]);
        if (last && i == cnt - 1) ptx::mma_commit(&q_empty);   // the item's queries were read
      };
      // one stream's step: out += P V of tile i, then S of its next tile j
      // (none: j >= cnt).  The ring's barriers are waited for before the
      // stream's P, which is the last to be ready.
      const auto step = [&](int i, int j, int x, bool first, bool ring, bool last) {
        const uint32_t nv = seq0 + v_place<C::AHEAD>(i, cnt), nk = seq0 + k_place<C::AHEAD>(j);
        const uint32_t sv = nv % SLOTS, sk = nk % SLOTS;
        if (ring) {
          wait(&full[sv], (nv / SLOTS) & 1u);
          if (j < cnt) wait(&full[sk], (nk / SLOTS) & 1u);
        }
        wait(&p_full[x], (p_phase >> x) & 1u);
        p_phase ^= 1u << x;
        if (!ok) return;
        const uint64_t dv = v_desc + sv * (C::SLOT >> 4);
        // steps of 16 keys up to the request's last
        const int steps = __shfl_sync(~0u, (min(s.r.len - (s.t0 + i) * TKT, TKT) + 15) >> 4, 0);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < TKT / 16; ++k)
            if (k == 0 || k < steps) ptx::mma_f16_ts(tm + C::O_COL + (MODE == SHARED ? 0 : 128 * x),
                            tm + C::S_COL + C::S_STEP * x + TKT / 2 + k * 8, dv + k * (2048 >> 4),
                            idesc<BF16>(D, true), (!first || k > 0) ? 1u : 0u);
          if (MODE == SHARED) ptx::mma_commit(&o_step[(tile0 + i) & 1u]);
          if (last) ptx::mma_commit(&empty[sv]);
          if (j < cnt) issue_s(sk, j, x, last);
        }
        __syncwarp();
      };
      const auto begin = [&](int i, int x, bool ring, bool last) {
        const uint32_t nk = seq0 + k_place<C::AHEAD>(i), sk = nk % SLOTS;
        if (ring) wait(&full[sk], (nk / SLOTS) & 1u);
        if (ok && elect_one()) issue_s(sk, i, x, last);
        __syncwarp();
      };
      wait(&q_full, q_phase);
      q_phase ^= 1u;
      if constexpr (MODE == SHARED) {
        // S of tile i + 2 goes to the buffer whose P the MMA before read
        for (int i = 0; i < min(cnt, 2); ++i) begin(i, (tile0 + i) % NS, true, true);
        for (int i = 0; i < cnt && ok; ++i) {
          if (i + 2 < cnt) begin(i + 2, (tile0 + i + 2) % NS, true, true);
          step(i, cnt, (tile0 + i) % NS, i == 0, true, true);
        }
        tile0 += cnt;
      } else {
        const bool two = __any_sync(~0u, s.r.n * a.group - s.rt * a.tile_rows > stream_rows);
        begin(0, 0, true, !two);
        if (two) begin(0, 1, false, true);
        for (int i = 0; i < cnt && ok; ++i) {
          step(i, i + 1, 0, i == 0, true, !two);
          if (two) step(i, i + 1, 1, i == 0, false, true);
        }
      }
      if (ok && elect_one()) ptx::mma_commit(&o_full);
      __syncwarp();
      seq0 += 2u * cnt;
    }
    // every MMA issued has completed once `done` fires
    if (elect_one()) ptx::mma_commit(&done);
    __syncwarp();
    if (!ptx::mbar_wait_bounded(&done, 0, WAIT_LIMIT)) atomicOr(&g_attn_error, ERR_DRAIN);
  } else if (warp == 2) {
    // ---------------- queries: an item's rows, as soon as the item before
    // needs its own no more.  A stream's rows are whole tokens with the heads
    // of the group, which is how a box of [tokens][heads][64 values] lies in
    // shared memory.  Rows past the request's last token are another's or
    // zero: they reach only their own rows of S.
    bool ok = true;
    uint32_t parity = 1;
    const int tokens = stream_rows / a.group;
    while (ok && walk.next(s)) {
      ok = ptx::mbar_wait_warp(&q_empty, parity, abort_flag, WAIT_LIMIT);
      if (!ok) {
        if (lane == 0 && !*abort_flag) fail(abort_flag, ERR_PRODUCER);
        break;
      }
      parity ^= 1u;
      const bool two = MODE == ROWS && s.r.n * a.group - s.rt * a.tile_rows > stream_rows;
      if (lane == 0)
        ptx::mbar_arrive_expect_tx(&q_full, static_cast<uint32_t>(stream_rows) * D * (two ? 4 : 2));
      __syncwarp();
      const int x = lane / HALVES, half = lane % HALVES;
      if (x < (two ? 2 : 1))
        ptx::tma_load_3d(sq + x * C::QB + half * (128 * 128), &tm_q, &q_full, half * 64,
                         s.h * a.group, s.r.row0 + (s.rt * (MODE == ROWS ? 2 : 1) + x) * tokens);
    }
    if (!ptx::mbar_wait_bounded(&q_full, parity, WAIT_LIMIT)) atomicOr(&g_attn_error, ERR_DRAIN);
  } else if (warp >= 4) {
    // ---------------- softmax and output: warpgroup x has stream x, a thread
    // one row of it
    const int x = (warp - 4) >> 2;
    const int lrow = (warp & 3) * 32 + lane;           // row of the stream's tile, its lane
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    uint32_t s_addr = tmem + C::S_COL + 128 * x + lane_addr;
    const uint32_t o_addr = tmem + C::O_COL + (MODE == SHARED ? 0 : 128 * x) + lane_addr;
    const int wid = tid - 128;                         // 0 .. 255
    // the maximum is taken of the products themselves, so the scale must not
    // be negative (the MMA turns the queries' signs instead) nor zero
    const float scale = fmaxf(fabsf(a.scale_log2), 1e-37f);
    bool ok = true;
    uint32_t seq0 = 0, s_phase = 0, o_phase = 0;
    uint32_t tile0 = 0;                                // tiles of the items before
    const auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!ok) return;
      ok = ptx::mbar_wait_warp(bar, parity, abort_flag, WAIT_LIMIT);
      if (!ok && lane == 0 && !*abort_flag) fail(abort_flag, ERR_CONSUMER);
      ptx::tc_fence_after();
    };
    while (walk.next(s)) {
      const int rows_all = s.r.n * a.group;
      const int r0 = s.rt * a.tile_rows;
      const int rows = min(a.tile_rows, rows_all - r0);
      const int cnt = s.t1 - s.t0;
      // row of the item, of which the stream has some from `base` on
      const int base = MODE == ROWS ? stream_rows * x : 0;
      const bool has = lrow < stream_rows && base + lrow < rows;
      const int my = base + lrow;
      const bool active = base + (warp & 3) * 32 < rows;
      const int tok = has ? div_group(a, r0 + my) : 0;
      const uint64_t* mw = a.mask != nullptr ? a.mask + (s.r.row0 + int64_t(tok)) * a.mask_words : nullptr;
      const uint64_t word0 = first_word(a, mw);
      float m = -INFINITY, l = 0.f;
      bool any = false;
      // SHARED: the tiles of this warpgroup's parity, counted over all items
      // (ROWS: a stream without rows has no S either)
      for (int i = MODE == SHARED ? (tile0 + x) & 1 : base < rows ? 0 : cnt; i < cnt;
           i += MODE == ROWS ? 1 : 2) {
        const int buf = MODE == SHARED ? (tile0 + i) % NS : x;
        if constexpr (MODE == SHARED) {
          s_addr = tmem + C::S_COL + C::S_STEP * buf + lane_addr;
          s_phase = ((tile0 + i) / NS) & 1u;
        }
        const int k0 = (s.t0 + i) * TKT;
        const bool edge = k0 > s.r.ctx - TKT;
        uint64_t vis[TKT / 64];
        if (edge && active) {
#pragma unroll
          for (int c = 0; c < TKT / 64; ++c)
            vis[c] = sees64(a, mw, word0, tok, k0 + 64 * c, s.r.ctx, s.r.len);
        }
        wait(&s_full[buf], s_phase);
        s_phase ^= 1u;
        if (!ok) break;
        if (active) {
          // a row of S is read twice, 64 columns at a time: held whole it would
          // not fit the registers.  The last 64 of the first pass are the first
          // of the second, so P starts in the upper half of S.
          uint32_t v[2][32];
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int c = 0; c < TKT / 32; c += 2) {
            ptx::tmem_ld_32x32b_x32(s_addr + 32 * c, v[0]);
            ptx::tmem_ld_32x32b_x32(s_addr + 32 * c + 32, v[1]);
            tmem_ld_wait_for(v[0]);
            tmem_ld_wait_for(v[1]);
            if (edge) {
              const uint64_t bits = TKT == 64 || c == 0 ? vis[0] : vis[TKT / 64 - 1];
              mask_out(v[0], static_cast<uint32_t>(bits));
              mask_out(v[1], static_cast<uint32_t>(bits >> 32));
            }
#pragma unroll
            for (int e = 0; e < 64; e += 2)
              mx[(e >> 1) & 3] = fmaxf(mx[(e >> 1) & 3], fmaxf(__uint_as_float(v[e >> 5][e & 31]),
                                                               __uint_as_float(v[e >> 5][(e & 31) + 1])));
          }
          const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale - kLift<BF16>;
          float f = 1.f;            // of this thread's sum
          bool move = false;        // of the accumulator, by `fo`
          float fo = 1.f;
          if constexpr (MODE == SHARED) {
            float mp = -INFINITY;   // the other warpgroup's, of the tile before
            if (i > 0) {
              wait(&m_ready[warp & 3], (tile0 + i - 1) & 1u);
              mp = *reinterpret_cast<volatile float*>(&s_m[lrow]);
            }
            float mn = mp;
            if (mt > mp + 8.f || (mp == -INFINITY && mt != mp)) mn = mt;
            *reinterpret_cast<volatile float*>(&s_m[lrow]) = mn;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&m_ready[warp & 3]);
            if (mn != m) f = ex2(m - mn);
            m = mn;
            if (mn != mp) fo = ex2(mp - mn);
            move = i > 0 && __any_sync(~0u, fo != 1.f);
            if (move) {
              wait(&o_step[(tile0 + i - 1) & 1u], ((tile0 + i - 1) >> 1) & 1u);
              move = ok;
            }
          } else {
            if (mt > m + 8.f || (m == -INFINITY && mt != m)) {
              f = ex2(m - mt);
              m = mt;
            }
            fo = f;
            move = any && __any_sync(~0u, f != 1.f);
          }
          if (move) {
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              ptx::tmem_ld_32x32b_x16(o_addr + 16 * c, o);
              tmem_ld_wait_for(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * fo);
              tmem_st_x16(o_addr + 16 * c, o);
            }
          }
          any = true;
          const float ms = m == -INFINITY ? 0.f : m;
          const float2 sc2 = make_float2(scale, scale), ms2 = make_float2(-ms, -ms);
          float2 sum[4] = {};
#pragma unroll
          for (int c = TKT / 32 - 2; c >= 0; c -= 2) {
            if (c < TKT / 32 - 2) {
              tmem_ld_wait_for(v[0]);
              tmem_ld_wait_for(v[1]);
              if (edge) {
                mask_out(v[0], static_cast<uint32_t>(vis[0]));
                mask_out(v[1], static_cast<uint32_t>(vis[0] >> 32));
              }
            }
            uint32_t w[2][16];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float2 t = fma2(make_float2(__uint_as_float(v[e >> 4][2 * (e & 15)]),
                                                __uint_as_float(v[e >> 4][2 * (e & 15) + 1])), sc2, ms2);
              const float2 p = make_float2(ex2(t.x), ex2(t.y));
              sum[e & 3] = add2(sum[e & 3], p);
              w[e >> 4][e & 15] = pack2<BF16>(p.x, p.y);
            }
            if (c > 0) {
              ptx::tmem_ld_32x32b_x32(s_addr, v[0]);
              ptx::tmem_ld_32x32b_x32(s_addr + 32, v[1]);
            }
            tmem_st_x16(s_addr + TKT / 2 + 16 * c, w[0]);
            tmem_st_x16(s_addr + TKT / 2 + 16 * c + 16, w[1]);
          }
          const float2 all = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
          l = l * f + (all.x + all.y);
          ptx::tmem_st_wait();
        } else if (MODE == SHARED && lane == 0) {
          ptx::mbar_arrive(&m_ready[warp & 3]);    // its phases count tiles, whoever is active
        }
        if (edge && (MODE == SHARED || x == 0)) {
          // values past the last token count as zero, and so does a non-finite
          // value of a new token here (added at the item's end)
          const uint32_t n = seq0 + v_place<C::AHEAD>(i, cnt);
          // SHARED: S runs so far ahead that the values of two tiles before may
          // still be on their way to this slot; a wait for a phase is only one
          // once the phase before it is over
          if (MODE == SHARED && i >= 2) wait(&o_step[(tile0 + i) & 1u], ((tile0 + i - 2) >> 1) & 1u);
          wait(&full[n % SLOTS], (n / SLOTS) & 1u);
          if (!ok) break;
          clean_values<BF16, D>(ring + (n % SLOTS) * C::SLOT, HB, k0, 0,
                                min(TKT, (max(s.r.len - k0, 1) + 15) & ~15), s.r.ctx, s.r.len, lrow,
                                128, s_bad, &s_any_bad);
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&p_full[buf]);
      }
      // ---- the item's part is complete
      wait(&o_full, o_phase);
      o_phase ^= 1u;
      seq0 += 2u * cnt;
      tile0 += cnt;
      if constexpr (MODE == SHARED) s_ml[x][lrow] = make_float2(m, l);
      ptx::named_sync(1, 256);
      const bool any_bad = *reinterpret_cast<volatile int*>(&s_any_bad) != 0;
      const bool whole = s.t0 == 0 && s.t1 == s.r.tiles;
      const int64_t slot = 2 * int64_t(blockIdx.x) + (s.t0 == 0 ? 1 : 0);
      if (ok && active) {
        if constexpr (MODE == SHARED) {      // the sums of both warpgroups' tiles
          const float2 y = s_ml[x ^ 1][lrow];
          const float mm = fmaxf(m, y.x);
          l = l * (mm == -INFINITY ? 0.f : ex2(m - mm)) + y.y * (mm == -INFINITY ? 0.f : ex2(y.x - mm));
          m = mm;
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t at = (int64_t(s.r.row0) + tok) * a.Hq + s.h * a.group + (r0 + my - tok * a.group);
        // SHARED: this warpgroup's half of the columns, which refer to the larger
        // maximum already; ROWS: all columns of its rows
        constexpr int NC = MODE == ROWS ? D : D / 2;
        const int col0 = MODE == ROWS ? 0 : x * NC;
#pragma unroll 1
        for (int c = 0; c < NC / 16; ++c) {
          uint32_t u[16];
          ptx::tmem_ld_32x32b_x16(o_addr + col0 + 16 * c, u);
          tmem_ld_wait_for(u);
          float o[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __uint_as_float(u[e]);
          if (has) {
            const int d = col0 + 16 * c;
            if (whole) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                uint4 w;
                w.x = pack2<BF16>(o[8 * e] * inv, o[8 * e + 1] * inv);
                w.y = pack2<BF16>(o[8 * e + 2] * inv, o[8 * e + 3] * inv);
                w.z = pack2<BF16>(o[8 * e + 4] * inv, o[8 * e + 5] * inv);
                w.w = pack2<BF16>(o[8 * e + 6] * inv, o[8 * e + 7] * inv);
                *reinterpret_cast<uint4*>(a.out + at * D + d + 8 * e) = w;
              }
            } else {
              float* po = a.part_o + ((slot * (D / 4) + d / 4) * RT + my) * 4;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                *reinterpret_cast<float4*>(po + 4 * RT * e) =
                    make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            }
            if (any_bad)
              add_bad<BF16>(a, s_bad, s.b, s.h, s.r.ctx, s.r.n, s.r.row0, tok, d, 16,
                            whole ? a.out + at * D + d : nullptr,
                            a.part_o + ((slot * (D / 4) + d / 4) * RT + my) * 4, 4 * RT);
          }
        }
        if (has && (MODE == ROWS || x == 0)) {
          if (!whole)
            a.part_ml[slot * RT + my] = make_float2(m, l);
          else if (a.lse != nullptr)
            a.lse[at] = l == 0.f ? -INFINITY : lse_of<BF16>(m, l);
        }
      }
      if (!whole && s.t0 == 0 && wid == 0) {
        const int first = static_cast<int>(blockIdx.x);
        a.items[first] = Item{first, cta_of(piece, s.end - 1) - first, s.r.row0, r0, rows, s.h};
      }
      ptx::tc_fence_before();
      ptx::named_sync(1, 256);   // accumulators, s_ml and s_bad are free again
      if (any_bad) {
        if (wid < 8) s_bad[wid] = 0;
        if (wid == 0) s_any_bad = 0;
        ptx::named_sync(1, 256);
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 2) ptx::tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ host

// The cache as [pages][heads][rows][dim]: boxes of `rows` rows of one page
// and head, 64 values wide (128 bytes, swizzled).
bool make_map(CUtensorMap* map, const tern_kv_cache& c, void* base, int rows) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.dim), static_cast<cuuint64_t>(c.page_size),
                              static_cast<cuuint64_t>(c.heads), static_cast<cuuint64_t>(c.pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.token_stride) * 2,
                                 static_cast<cuuint64_t>(c.head_stride) * 2,
                                 static_cast<cuuint64_t>(c.page_stride) * 2};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(rows), 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const auto type = c.dtype == TERN_KV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                            : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return enc(map, type, 4, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Which kernel serves requests of up to `rows` rows on a key head, as its
// rows an item and its CTAs an SM.  8 key heads, device time:
//   16 rows, 16 requests of up to 1000 keys / 1 of 100000: rows kernel 14.8 / 44.4 us
//     with head size 64, 20.1 / 74.7 with 128, 31.8 / 136 with 256; tile kernel
//     18.5 / 44.6, 21.1 / 72.7, 24.0 / 127.  Over 26 sizes from 3 to 20000 keys
//     the tile kernel takes 1.15 of the rows kernel's time with head size 64,
//     0.99 with 128, 0.80 with 256 (and 1.16 with 256 and 1, 4 and 8 rows).
//   256 rows, 16 requests of up to 6000 keys / 4 of up to 30000: ROWS 58.9 / 75.2 us with
//     head size 64, 75.5 / 96.1 with 128; SHARED twice, the second reading the
//     keys from L2 where it keeps pace, 59.7 / 81.1 and 88.9 / 133.  144 rows:
//     56.2 / 64.8 and 70.3 / 77.6 against 45.8 / 52.4 and 67.6 / 71.7; over
//     nine counts of rows from 144 to 512 SHARED takes 0.96 of ROWS's time with
//     head size 64 and 1.11 of it with 128.
// The tile kernel takes whole tokens, so a group above 128 heads is the rows
// kernel's.
struct Choice {
  int nt;         // rows kernel: eights of rows; 0: tile kernel
  int mode;       // tile kernel
  int rt, ctas;
};
Choice choose(int64_t max_new, int64_t group, int64_t D) {
  const int64_t rows = max_new * group;
  const int ctas = D == 256 ? 1 : 2;
  if (rows <= 8) return {1, 0, 8, ctas};
  if ((rows <= 16 && D < 256) || group > 128) return {2, 0, 16, ctas};
  if (D != 128 || rows <= 128 / group * group) return {0, SHARED, 128, 1};
  return {0, ROWS, 256, 1};
}

cudaError_t set_up(const TreeAttnCall& call, int keys, int grid, int rt, Args& a, CUtensorMap& tk,
                   CUtensorMap& tv) {
  const int box = static_cast<int>(std::min<int64_t>(call.cache.page_size, keys));
  if (!make_map(&tk, call.cache, call.cache.k, box) || !make_map(&tv, call.cache, call.cache.v, box))
    return cudaErrorInvalidValue;
  const Ws w = ws_layout(grid, rt, call.cache.dim);
  uint8_t* ws = static_cast<uint8_t*>(call.ws);
  a.part_o = reinterpret_cast<float*>(ws + w.o);
  a.part_ml = reinterpret_cast<float2*>(ws + w.ml);
  a.arrived = reinterpret_cast<int*>(ws);
  a.items = reinterpret_cast<Item*>(ws + w.items);
  a.tile_rows = rt;
  return cudaSuccess;
}

template <bool BF16, int D, int NT>
cudaError_t launch_rows(const TreeAttnCall& call, Args a, cudaStream_t st) {
  using C = Rows<D, NT>;
  static std::atomic<unsigned long long> attr_done{0};
  cudaError_t e = once_per_device(attr_done, [] {
    return cudaFuncSetAttribute(attn_rows_kernel<BF16, D, NT>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(C::SMEM));
  });
  if (e != cudaSuccess) return e;
  const int grid = std::min(kv_sm_count() * C::CTAS, MAX_GRID);
  CUtensorMap tk, tv;
  e = set_up(call, TK, grid, C::RT, a, tk, tv);
  if (e != cudaSuccess) return e;
  return launch(attn_rows_kernel<BF16, D, NT>, dim3(grid), dim3(C::THREADS), C::SMEM, st, tk, tv, a);
}

template <bool BF16, int D, int MODE>
cudaError_t launch_tile(const TreeAttnCall& call, Args a, cudaStream_t st) {
  using C = Tile<D, MODE>;
  static std::atomic<unsigned long long> attr_done{0};
  cudaError_t e = once_per_device(attr_done, [] {
    return cudaFuncSetAttribute(attn_tile_kernel<BF16, D, MODE>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(C::SMEM));
  });
  if (e != cudaSuccess) return e;
  const int grid = std::min(kv_sm_count(), MAX_GRID);
  CUtensorMap tk, tv;
  e = set_up(call, C::TKT, grid, C::RT, a, tk, tv);
  if (e != cudaSuccess) return e;
  // the queries as [T][Hq][D]: boxes of a stream's tokens and the group's heads
  const int tokens = 128 / a.group;
  a.tile_rows = tokens * a.group * (MODE == ROWS ? 2 : 1);
  CUtensorMap tq;
  if (!make_query_map(&tq, call.q, call.cache.dtype == TERN_KV_BF16, D, call.Hq, call.T, call.q_head_stride,
                      call.q_token_stride, tokens, a.group))
    return cudaErrorInvalidValue;
  e = launch(attn_tile_kernel<BF16, D, MODE>, dim3(grid), dim3(TILE_THREADS), C::SMEM, st, tk, tv, tq, a);
  if (e != cudaSuccess) return e;
  return launch(combine_kernel<BF16, D>, dim3(4 * kv_sm_count()), dim3(JOIN_THREADS), 0, st, a, C::RT,
                grid);
}

template <bool BF16, int D>
cudaError_t launch_dim(const TreeAttnCall& call, const Args& a, cudaStream_t st) {
  const Choice c = choose(call.max_new, a.group, D);
  if (c.nt == 1) return launch_rows<BF16, D, 1>(call, a, st);
  if (c.nt == 2) return launch_rows<BF16, D, 2>(call, a, st);
  if constexpr (D != 128) {
    return launch_tile<BF16, D, SHARED>(call, a, st);
  } else {
    return c.mode == ROWS ? launch_tile<BF16, D, ROWS>(call, a, st)
                          : launch_tile<BF16, D, SHARED>(call, a, st);
  }
}

}  // namespace

size_t tree_attention_workspace_bytes(int64_t max_new, int64_t Hq, int64_t H, int64_t D) {
  const Choice c = choose(max_new, Hq / H, D);
  return ws_layout(std::min(kv_sm_count() * c.ctas, MAX_GRID), c.rt, D).bytes;
}

cudaError_t launch_tree_attention(const TreeAttnCall& call, cudaStream_t st) {
  const tern_kv_cache& c = call.cache;
  Args a{};
  a.q = static_cast<const uint16_t*>(call.q);
  a.v = static_cast<const uint16_t*>(c.v);
  a.out = static_cast<uint16_t*>(call.out);
  a.lse = call.lse;
  a.table = call.table;
  a.ctx_len = call.ctx_len;
  a.row_start = call.row_start;
  a.mask = call.mask;
  a.q_token = call.q_token_stride;
  a.q_head = call.q_head_stride;
  a.table_stride = call.table_stride;
  a.page_stride = c.page_stride;
  a.token_stride = c.token_stride;
  a.head_stride = c.head_stride;
  a.width = static_cast<int>(call.table_width);
  a.pages = static_cast<int>(c.pages);
  while ((int64_t(1) << a.page_shift) < c.page_size) ++a.page_shift;
  a.mask_words = static_cast<int>(call.mask_words);
  a.B = static_cast<int>(call.B);
  a.T = static_cast<int>(call.T);
  a.H = static_cast<int>(c.heads);
  a.Hq = static_cast<int>(call.Hq);
  a.group = static_cast<int>(call.Hq / c.heads);
  // exact for every row that T tokens can have: r group < 2^32 for r < T group
  a.group_mul = a.group > 1 && call.T < (int64_t(1) << 32) / (int64_t(a.group) * a.group)
                    ? static_cast<uint32_t>((uint64_t(1) << 32) / a.group + 1) : 0;
  a.scale_log2 = call.scale * 1.4426950408889634f;
  const bool bf = c.dtype == TERN_KV_BF16;
  if (c.dim == 64) return bf ? launch_dim<true, 64>(call, a, st) : launch_dim<false, 64>(call, a, st);
  if (c.dim == 128)
    return bf ? launch_dim<true, 128>(call, a, st) : launch_dim<false, 128>(call, a, st);
  return bf ? launch_dim<true, 256>(call, a, st) : launch_dim<false, 256>(call, a, st);
}

cudaError_t attn_read_clear_error(unsigned int* err) {
  cudaError_t e = cudaMemcpyFromSymbol(err, g_attn_error, sizeof(unsigned int));
  if (e != cudaSuccess || *err == 0) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_attn_error, &zero, sizeof(unsigned int));
}

}  // namespace tern
