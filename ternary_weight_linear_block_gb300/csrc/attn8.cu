// Attention of drafted tokens over the 8-bit paged cache (tern_tree_attention8).
//
// A key is code * ku and a value code * vu, with a unit of its row each.  For a
// row (new token with a query head) over the keys j that it sees:
//   t_j = scale log2(e) ku_j (q . code_j),   p_j = 2^(t_j - m),
//   l = sum p_j,   out = sum (p_j vu_j) code_j / l,   lse = (m + log2 l) ln 2.
// Codes become fp16 exactly, so the products are mma.sync of fp16 with 32-bit
// sums whatever the rows' type: a row of bf16 queries is turned into fp16 by the
// power of two that brings its largest to 2^13 .. 2^14 and keeps its 8 bits; the
// power goes into the row's scale.  p_j vu_j is rounded to fp16 for the second
// product.  So that it keeps its bits whatever the units are, m is the maximum of
// t_j + log2 vu_j (less kLift's 7), not of t_j: p_j vu_j <= 2^7 when m is set.
// l and lse do not depend on which reference was taken.
//
// attn8_rows_kernel: up to 16 rows an item.  Work division, the ring of tiles and
// the join of pieces are those of attn_rows_kernel; a tile of a stage has the codes
// as their pages hold them, and 4 bytes a key for its unit.
//
// The cache's bytes bound it, half of the 16-bit cache's, but widening a code costs
// about as many instructions as its two products, so the SM has twice as many a
// byte: 64 requests of one token over up to 16001 keys take 264 us (5.2 TB/s, 0.76
// of the copy rate; 274 with two CTAs an SM and a longer ring, 272 before each
// warp's units were read ahead), 16 of them over up to 700 keys 22.5 (two CTAs
// 20.5: one rule for both is kept, that of the long case).  A profile of 16 requests
// has 0.57 instructions a cycle and scheduler, DRAM at 58 %, waits for fixed
// latencies 1.6 and for memory 1.0 cycles an instruction.  4 drafts of 6 heads of
// 256 over 131001 keys are 24 rows, the tile kernel's: 116 us.
#include <algorithm>

#include "attn8_dev.cuh"

namespace tern {

__device__ unsigned int g_attn8_error;

namespace {

using namespace attn;

__device__ __forceinline__ void fail(volatile int* abort_flag, unsigned int code) {
  *abort_flag = 1;
  atomicOr(&g_attn8_error, code);
}

// NT eights of rows an item, NW warps that share a tile's keys, 16 each.
template <int D, int NT>
struct Rows8 {
  static constexpr int NW = 4;
  static constexpr int TK = 16 * NW;
  static constexpr int RT = 8 * NT;
  static constexpr int PAD = D == 64 ? 4 : 3;             // as for the 16-bit cache
  static constexpr int LEAST = PAD + 1;
  static constexpr int THREADS = (NW + 2) * 32;
  static constexpr int ROWB = D < 128 ? D : 128;          // bytes of a row of a tile's part
  static constexpr int HALVES = D / ROWB;
  static constexpr int PART = TK * ROWB;
  static constexpr int CODES = TK * D;
  static constexpr int UNITS = TK * 4;
  static constexpr int STAGE = 2 * CODES;                 // keys, values
  static constexpr int CTAS = D == 256 ? (NT > 1 ? 1 : 2) : NT == 1 ? 3 : 2;
  static constexpr int IC = D == 64 || NT > 1 ? 4 : 8;    // value tiles that are joined at a time
  static constexpr int COLS = 16 * IC;
  static constexpr int LD = COLS + 4;
  static constexpr int MERGE = 2 * RT * LD * 4;
  static constexpr int QLD = D * 2 + 16;
  static constexpr int QBYTES = RT * QLD;
  static constexpr int ROOM = (CTAS == 3 ? 76800 : CTAS == 2 ? 115200 : 232448) - MERGE - QBYTES - 1024 - 2048;
  static constexpr int FIT = ROOM / (STAGE + 2 * UNITS);
  static constexpr int STAGES = FIT < 8 ? FIT : 8;
  static constexpr size_t SMEM = size_t(STAGES) * (STAGE + 2 * UNITS) + MERGE + QBYTES + 1024;
  static_assert(STAGES >= 2, "ring");
};

template <bool BF16, int KIND, int D, int NT>
__global__ void __launch_bounds__((Rows8<D, NT>::THREADS), (Rows8<D, NT>::CTAS))
    attn8_rows_kernel(const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Args8 g) {
  using C = Rows8<D, NT>;
  constexpr int RT = C::RT, THREADS = C::THREADS, NW = C::NW, TK = C::TK;
  constexpr int KS = D / 16;
  const Args& a = g.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  float* merge = reinterpret_cast<float*>(ring + C::STAGES * C::STAGE);
  uint8_t* sq = ring + C::STAGES * C::STAGE + C::MERGE;
  float* units = reinterpret_cast<float*>(sq + C::QBYTES);      // [stage][keys, values][TK]
  __shared__ uint64_t full[C::STAGES], empty[C::STAGES], q_full, q_empty;
  __shared__ __align__(16) Part s_part;
  __shared__ uint64_t s_word0[RT];      // of each row's mask
  __shared__ PieceScratch<THREADS> scratch;
  __shared__ float2 s_ml[NW][RT];
  __shared__ int s_last;
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
    ptx::mbar_fence_init();
    ptx::prefetch_tmap(&tm_k);
    ptx::prefetch_tmap(&tm_v);
  }
  pdl_wait();
  pdl_launch_dependents();
  const Piece piece = find_piece<TK, C::PAD, C::LEAST, THREADS>(a, scratch);   // synchronises the CTA
  if (piece.lo >= piece.hi) return;

  if (warp >= NW) {
    // ---------------- producers: one warp copies the keys, one the values; the
    // keys' also copies each item's queries and says what the item is
    const bool vals = warp > NW;
    const CUtensorMap* map = vals ? &tm_v : &tm_k;
    const float* unit = vals ? g.vu : g.ku;
    Walk<TK, C::PAD> walk(a, piece);
    Seg s{};
    int st = 0;
    uint32_t phase = 0, q_phase = 1;
    long issued = 0, q_issued = 0;
    bool ok = true;
    const int box_shift = min(a.page_shift, TK == 128 ? 7 : 6);      // rows of a box: a page, or the tile
    const auto give_up = [&](bool good) {
      if (!good && lane == 0 && !*abort_flag) fail(abort_flag, ERR_PRODUCER);
      return good;
    };
    uint64_t word0 = 0;      // lane r: of the mask of the item's row r
    const auto rows_of = [&] { return min(RT, s.r.n * a.group - s.rt * RT); };
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
    // codes and units of tile t: a lane has one page's box of one half, the
    // first half's lanes also its units.  A page out of range gives zeros: of
    // codes by the copy, of units by this lane.
    const auto load = [&](int t, int page) {
      const int k0 = t * TK;
      const int keys = min(TK, s.r.len - k0);
      const int boxes = keys > 0 ? (keys + (1 << box_shift) - 1) >> box_shift : 0;
      const int box = lane / C::HALVES, half = lane % C::HALVES;
      const int pg = __shfl_sync(~0u, page, box);
      const bool mine = box < boxes, known = pg < a.pages;
      float* to = units + (st * 2 + (vals ? 1 : 0)) * TK + (box << box_shift);
      if (mine && half == 0 && !known)
        for (int i = 0; i < (1 << box_shift); ++i) to[i] = 0.f;
      const int with_units = __popc(__ballot_sync(~0u, mine && half == 0 && known));
      __syncwarp();
      if (lane == 0)
        ptx::mbar_arrive_expect_tx(&full[st], static_cast<uint32_t>(boxes * D + with_units * 4) << box_shift);
      __syncwarp();
      if (mine) {
        const int row = k0 & ((1 << a.page_shift) - 1);
        uint8_t* dst = ring + st * C::STAGE + (vals ? C::CODES : 0) + half * C::PART + (box << box_shift) * C::ROWB;
        tma_load_4d(dst, map, &full[st], half * 128, row, s.h, pg);
        if (half == 0 && known)
          ptx::bulk_load(to, unit + pg * g.unit_page + s.h * g.unit_head + row, 4u << box_shift, &full[st]);
      }
    };
    while (ok && walk.next(s)) {
      int page = page_at<TK>(a, s, s.t0, box_shift, lane);
      if (!vals && a.mask != nullptr && lane < rows_of())
        word0 = a.mask[(s.r.row0 + int64_t(div_group(a, s.rt * RT + lane))) * a.mask_words];
      bool posted = vals;
      if (!vals && __all_sync(~0u, ptx::mbar_test_wait(&q_empty, q_phase))) {
        post_queries();
        posted = true;
      }
      for (int t = s.t0; t < s.t1 && ok; ++t) {
        const int ahead = t + 1 < s.t1 ? page_at<TK>(a, s, t + 1, box_shift, lane) : 0;
        ok = give_up(ptx::mbar_wait_warp(&empty[st], phase ^ 1u, abort_flag, WAIT_LIMIT));
        if (!ok) break;
        load(t, page);
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
      if (!ptx::mbar_wait_bounded(&full[st], phase, WAIT_LIMIT)) atomicOr(&g_attn8_error, ERR_DRAIN);
    }
    if (q_issued > 0 && (!ok || *abort_flag) && !ptx::mbar_wait_bounded(&q_full, q_phase, WAIT_LIMIT))
      atomicOr(&g_attn8_error, ERR_DRAIN);
    return;
  }

  // ---------------- consumers: warp w has keys 16 w .. 16 w + 15 of each tile
  int st = 0;
  uint32_t phase = 0;
  const uint32_t ring_u = ptx::smem_u32(ring);
  const int row_b = lane >> 2;           // query row (of 8) whose fragment this lane holds
  const int row_c = (lane & 3) * 2;      // score rows of this lane: row_c, row_c + 1
  // ldmatrix of bytes: keys 0-7 and 8-15 of one 16-byte chunk, then of the next.
  // A lane gets 4 codes of a key, columns 4 c .. 4 c + 3 of a 16-column step,
  // as the fragment's pairs (0, 1) and (2, 3); the queries' fragments take the
  // same order.
  const int k_row = warp * 16 + (lane & 15);
  const int k_chunk = lane >> 4;
  // values: a lane has a 16-byte chunk (or half of one) of four keys
  const int v_key = warp * 16 + row_c;
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
    uint32_t qf[KS][NT][2];
    float row_scale[NT][2];
    int tok[NT][2];
    uint64_t word0[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint8_t* q = sq + (n * 8 + row_b) * C::QLD + (lane & 3) * 8;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const uint2 w = *reinterpret_cast<const uint2*>(q + k * 32);
        qf[k][n][0] = w.x;
        qf[k][n][1] = w.y;
      }
      float f = a.scale_log2;
      if constexpr (BF16) {
        // the row's largest exponent; a row with an infinity or NaN stays as it is
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            top = max(top, max(qf[k][n][e] & 0x7F80u, (qf[k][n][e] >> 16) & 0x7F80u));
        top = max(top, __shfl_xor_sync(~0u, top, 1));
        top = max(top, __shfl_xor_sync(~0u, top, 2));
        // 2^13 / 2^exponent, in two factors as it may pass 2^127
        const int up = top == 0x7F80u ? 0 : 140 - max(static_cast<int>(top >> 7), 1);
        const float f0 = __int_as_float((127 + up / 2) << 23), f1 = __int_as_float((127 + up - up / 2) << 23);
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t w = qf[k][n][e];
            qf[k][n][e] = pack2<false>(__uint_as_float(w << 16) * f0 * f1, __uint_as_float(w & 0xFFFF0000u) * f0 * f1);
          }
        f = f * __int_as_float((127 - up / 2) << 23) * __int_as_float((127 - (up - up / 2)) << 23);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        row_scale[n][e] = __shfl_sync(~0u, f, (row_c + e) * 4);
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
      const uint8_t* vbase = ring + st * C::STAGE + C::CODES;
      if (k0 < s.len || k0 == 0) {     // else past the last token: nothing to add
        const float* un = units + st * 2 * TK + warp * 16 + row_b;
        const float ku[2] = {un[0], un[8]}, vu[2] = {un[TK], un[TK + 8]};
        // two sums, of alternate steps: an MMA waits for the one before in its own
        float c[NT][4], c2[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) c[n][e] = c2[n][e] = 0.f;
#pragma unroll
        for (int k = 0; k < KS; k += 2) {
          uint32_t x[4], f[2][4];
          const int chunk = k + k_chunk;
          ldsm_x4(kbase + (chunk >> 3) * C::PART + chunk_at<C::ROWB>(k_row, chunk & 7), x);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            widen<KIND>(x[2 * e], f[e][0], f[e][2]);
            widen<KIND>(x[2 * e + 1], f[e][1], f[e][3]);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816<false>(e ? c2[n] : c[n], f[e], qf[k + e][n][0], qf[k + e][n][1]);
          }
        }
        // c[n]: keys lane / 4 and + 8, rows row_c and + 1
        const float lu[2] = {__log2f(fmaxf(vu[0], kLeastUnit)), __log2f(fmaxf(vu[1], kLeastUnit))};
        bool hid[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            c[n][e] = (c[n][e] + c2[n][e]) * (ku[e >> 1] * row_scale[n][e & 1]);
            hid[n][e] = edge && !((vis[n][e & 1] >> (row_b + (e >> 1) * 8)) & 1);
            if (hid[n][e]) c[n][e] = -INFINITY;
          }
        float al[NT][2];
        bool moved = false;
        uint32_t p[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float ms[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = fmaxf(c[n][e] + lu[0], c[n][e + 2] + lu[1]);
            x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
            x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
            x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
            const float mn = fmaxf(m[n][e], x - kLift<false>);
            ms[e] = mn == -INFINITY ? 0.f : mn;
            al[n][e] = ex2(m[n][e] - ms[e]);
            moved |= mn != m[n][e];
            m[n][e] = mn;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) c[n][e] = ex2(c[n][e] - ms[e & 1]);
#pragma unroll
          for (int e = 0; e < 2; ++e) l[n][e] = l[n][e] * al[n][e] + (c[n][e] + c[n][e + 2]);
#pragma unroll
          for (int e = 0; e < 4; ++e) c[n][e] = hid[n][e] ? 0.f : c[n][e] * vu[e >> 1];
          p[n][0] = movm(pack2<false>(c[n][0], c[n][1]));
          p[n][1] = movm(pack2<false>(c[n][2], c[n][3]));
        }
        if (__any_sync(~0u, moved)) {
#pragma unroll
          for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[i][n][e] *= al[n][e & 1];
        }
        // values: of keys row_c, row_c + 1, row_c + 8, row_c + 9 the lane's
        // columns; two keys' bytes side by side are a fragment's pairs
        constexpr int WORDS = C::ROWB / 32;       // words of a key and part
#pragma unroll
        for (int h = 0; h < C::HALVES; ++h) {
          uint32_t w[4][WORDS];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int r = v_key + (y & 1) + (y >> 1) * 8;
            const uint8_t* at = vbase + h * C::PART;
            if constexpr (D == 64) {
              const uint2 v = *reinterpret_cast<const uint2*>(at + chunk_at<64>(r, row_b >> 1) + (row_b & 1) * 8);
              w[y][0] = v.x, w[y][1] = v.y;
            } else {
              const uint4 v = *reinterpret_cast<const uint4*>(at + chunk_at<128>(r, row_b));
              w[y][0] = v.x, w[y][1] = v.y, w[y][2] = v.z, w[y][3] = v.w;
            }
            // what stands past the last token may be no number
            if (KIND == E4M3 && edge && t * TK + r >= s.len) {
#pragma unroll
              for (int j = 0; j < WORDS; ++j) w[y][j] = 0;
            }
          }
#pragma unroll
          for (int j = 0; j < WORDS; ++j)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              uint32_t f[4];
              widen<KIND>(__byte_perm(w[0][j], w[1][j], b ? 0x7362 : 0x5140), f[0], f[1]);
              widen<KIND>(__byte_perm(w[2][j], w[3][j], b ? 0x7362 : 0x5140), f[2], f[3]);
              // value tile i: columns 2 i and 2 i + 1 of the lane's
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma16816<false>(o[h * 2 * WORDS + 2 * j + b][n], f, p[n][0], p[n][1]);
            }
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
    // pieces and bf16's lse refer to the maximum itself
    constexpr float kDown = BF16 ? 1.f / 128.f : 1.f;
    float f[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) mm = fmaxf(mm, s_ml[w][n * 8 + row_c + e].x);
        f[n][e] = mm == -INFINITY ? 0.f : ex2(m[n][e] - mm) * kDown;
      }
    const bool whole = s.whole != 0;
    const int64_t slot = 2 * int64_t(blockIdx.x) + s.begins;
    float* mine = merge + (warp & 1) * (RT * C::LD);
    constexpr int IC = C::IC, EACH = 2 * IC;     // columns of a lane at a time
#pragma unroll
    for (int i0 = 0; i0 < KS; i0 += IC) {
      if (i0 > 0) ptx::named_sync(1, NW * 32);
#pragma unroll 1
      for (int round = 0; round < NW / 2; ++round) {
        if ((warp >> 1) == round) {
#pragma unroll
          for (int i = 0; i < IC; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float2* at = reinterpret_cast<float2*>(mine + (n * 8 + row_c + e) * C::LD + row_b * EACH + 2 * i);
                float2 x = make_float2(o[i0 + i][n][e] * f[n][e], o[i0 + i][n][e + 2] * f[n][e]);
                if (round > 0) {
                  const float2 y = *at;
                  x = make_float2(x.x + y.x, x.y + y.y);
                }
                *at = x;
              }
        }
        ptx::named_sync(1, NW * 32);
      }
      // ---- write: thread -> 4 consecutive values of a row
#pragma unroll 1
      for (int i = tid; i < RT * (C::COLS / 4); i += NW * 32) {
        const int r = i % RT, place = i / RT * 4;
        // a lane has ROWB / 8 columns in a row, EACH of them in this round
        const int d = i0 / (C::ROWB / 16) * C::ROWB + place / EACH * (C::ROWB / 8) +
                      2 * (i0 % (C::ROWB / 16)) + place % EACH;
        if (r >= rows) continue;
        float4 x = *reinterpret_cast<const float4*>(merge + r * C::LD + place);
        const float4 y = *reinterpret_cast<const float4*>(merge + (RT + r) * C::LD + place);
        x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
        float mm = -INFINITY, ll = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) mm = fmaxf(mm, s_ml[w][r].x);
#pragma unroll
        for (int w = 0; w < NW; ++w)
          ll += s_ml[w][r].y * (mm == -INFINITY ? 0.f : ex2(s_ml[w][r].x - mm) * kDown);
        if (BF16) mm += kLift<false>;
        if (whole) {
          const int token = div_group(a, r0 + r), head = s.h * a.group + (r0 + r - token * a.group);
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
      }
    }
    if (!whole) {
      const Item it{s.first, s.follow, s.row0, r0, rows, s.h};
      if (n_joins++ == 0) joins[0] = it; else joins[1] = it;
    }
  }
  if (n_joins > 0) join_pieces<BF16, D, RT, NW * 32>(a, joins, n_joins, tid, &s_last);
}

// ------------------------------------------------------------------ host

// Eights of rows an item of the rows kernel for requests of up to `max_new` tokens,
// 0: the tile kernel (which takes whole tokens, so a group above 128 heads is
// not its).  Items of 16 rows read the keys again for every 16, from L2 for the
// most part, and are still ahead up to the counts below (rows kernel / tile
// kernel, us, int8, 8 requests of up to 20003 keys and 32 of up to 1500; 16, 8 and 4
// key heads of 64, 128 and 256):
//    64   32 rows 167 / 226 and 69 / 110, 48 rows 259 / 248 and 93 / 116,
//         64 rows 305 / 228 and 112 / 112
//   128   24 rows 89 / 111 and 46 / 61, 32 rows 126 / 130 and 59 / 67,
//         48 rows 188 / 142 and 78 / 70
//   256   16 rows 77 / 100 and 42 / 53, 24 rows 100 / 97 and 54 / 52
// Items of 32 rows of head size 64 took 187 and 83 for 32 rows: a loop that no
// longer fits the instruction cache.
int eights_of(int64_t max_new, int64_t group, int64_t D) {
  const int64_t rows = max_new * group;
  if (rows <= 8) return 1;
  return group > 128 || rows <= (D == 64 ? 48 : D == 128 ? 32 : 16) ? 2 : 0;
}

template <bool BF16, int KIND, int D, int NT>
cudaError_t launch_rows8(const TreeAttn8Call& call, Args8 g, cudaStream_t st) {
  using C = Rows8<D, NT>;
  static std::atomic<unsigned long long> attr_done{0};
  const cudaError_t e = once_per_device(attr_done, [] {
    return cudaFuncSetAttribute(attn8_rows_kernel<BF16, KIND, D, NT>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(C::SMEM));
  });
  if (e != cudaSuccess) return e;
  const int grid = std::min(kv_sm_count() * C::CTAS, MAX_GRID8);
  const int box = static_cast<int>(std::min<int64_t>(call.cache.page_size, C::TK));
  CUtensorMap tk, tv;
  if (!make_map8(&tk, call.cache, call.cache.k, box) || !make_map8(&tv, call.cache, call.cache.v, box))
    return cudaErrorInvalidValue;
  const Ws w = ws_layout(grid, C::RT, D);
  uint8_t* ws = static_cast<uint8_t*>(call.ws);
  g.a.part_o = reinterpret_cast<float*>(ws + w.o);
  g.a.part_ml = reinterpret_cast<float2*>(ws + w.ml);
  g.a.arrived = reinterpret_cast<int*>(ws);
  g.a.items = reinterpret_cast<Item*>(ws + w.items);
  g.a.tile_rows = C::RT;
  return launch(attn8_rows_kernel<BF16, KIND, D, NT>, dim3(grid), dim3(C::THREADS), C::SMEM, st, tk, tv, g);
}

template <bool BF16, int KIND, int D>
cudaError_t launch_dim8(const TreeAttn8Call& call, const Args8& g, cudaStream_t st) {
  const int nt = eights_of(call.max_new, g.a.group, D);
  return nt == 1 ? launch_rows8<BF16, KIND, D, 1>(call, g, st) : launch_rows8<BF16, KIND, D, 2>(call, g, st);
}

template <bool BF16, int KIND>
cudaError_t launch_kind8(const TreeAttn8Call& call, const Args8& g, cudaStream_t st) {
  if (call.cache.dim == 64) return launch_dim8<BF16, KIND, 64>(call, g, st);
  if (call.cache.dim == 128) return launch_dim8<BF16, KIND, 128>(call, g, st);
  return launch_dim8<BF16, KIND, 256>(call, g, st);
}

}  // namespace

size_t tree_attention8_workspace_bytes(int64_t max_new, int64_t Hq, int64_t H, int64_t D) {
  const int nt = eights_of(max_new, Hq / H, D);
  if (nt == 0) return ws_layout(std::min(kv_sm_count(), MAX_GRID8), 128, D).bytes;
  return ws_layout(std::min(kv_sm_count() * 3, MAX_GRID8), 8 * nt, D).bytes;
}

cudaError_t launch_tree_attention8(const TreeAttn8Call& call, cudaStream_t st) {
  const tern_kv_cache8& c = call.cache;
  Args8 g{};
  Args& a = g.a;
  a.q = static_cast<const uint16_t*>(call.q);
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
  g.ku = c.k_scale;
  g.vu = c.v_scale;
  g.unit_page = c.scale_page_stride;
  g.unit_head = c.scale_head_stride;
  if (eights_of(call.max_new, a.group, c.dim) == 0) return launch_attn8_tile(call, g, st);
  if (call.dtype == TERN_KV_BF16)
    return c.dtype == TERN_KV_I8 ? launch_kind8<true, I8>(call, g, st) : launch_kind8<true, E4M3>(call, g, st);
  return c.dtype == TERN_KV_I8 ? launch_kind8<false, I8>(call, g, st) : launch_kind8<false, E4M3>(call, g, st);
}

cudaError_t attn8_read_clear_error(unsigned int* err) {
  unsigned int tile = 0;
  cudaError_t e = attn8_tile_read_clear_error(&tile);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(err, g_attn8_error, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  if (*err != 0) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_attn8_error, &zero, sizeof(unsigned int));
  }
  *err |= tile;
  return e;
}

}  // namespace tern
