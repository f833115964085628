// Attention of many rows over the 8-bit paged cache, on tcgen05 (the rows of up to
// 16 are attn8.cu's, which states the mathematics).
//
// The SHARED kernel of the 16-bit cache (attn.cu) with a stage more: tiles of
// codes arrive in a ring of their own, and four warps turn them into fp16 tiles,
// exactly, as the MMAs want them.  They also turn bf16 queries into fp16 by a
// power of two for each row.  A score column is multiplied by its key's unit in 32
// bits as the softmax reads a row.  The values' units:
//   folded  bf16 rows, a tile of cached tokens whose units are within 2^8 of each
//           other: code * unit / 2^E goes to the fp16 tile (one rounding, as
//           relatively small as that of the probabilities, which then take 2^E;
//           beside an fp16 output's it would show), E the largest unit's
//           exponent, so the softmax has nothing to read
//   exact   others, and a tile with new tokens (which a row may not see):
//           probabilities are multiplied by the unit in 32 bits
// The reference m of a row's exponents is the largest t_j + log2 vu_j of the tile
// that set it.  A tile of cached tokens first takes a bound of its own: the largest
// score times the largest (or, below zero, the least) key's unit, one pass over
// the scores alone.  Only where fp16 could not hold what the bound allows, and
// in tiles with new tokens, is the maximum itself looked for.  What a folded tile
// rounds to fp16 is 2^(t_j - m + E), of a key whose unit is less than 2^E more than
// m knows of, so there m is also at least the largest t_j + E - kTop; as its t_j +
// log2 vu_j is 2^8 below at most, the product keeps 2^7.
//
// Neither memory nor the tensor cores bound it but what the warps issue: widening,
// and two passes over the scores.  4 requests of 29 drafts of 4 heads (116 rows) of
// 128 over up to 20003 keys: 94 us, 162 MB of codes at 1.7 TB/s; 24 rows of 256 over
// 131001 keys: 116 us, 2.4 TB/s.  Steps of the first: 254 as items of 16 rows; 123
// as tiles; 106 with the units folded and the loops rolled; 102 and 89 with a tile's
// bound in place of its maximum and short code for exact tiles, 94 with more bits
// for small probabilities (kRef).  The code matters
// twice: a profile of the first version waited 1.9 cycles an instruction for the
// instruction itself, since eight kinds of warps run as many loops, so loops stay
// rolled and short (widening unrolled eight times 159, against 124).  Not better:
// 640 threads with two widening groups 122 (106), 3 fp16 and 5 code tiles 127, 5 and
// 1 173, scores 32 columns at a time 129 (spills), a reference that moves by 2^2 128.
// One warp copies and in ring order: with two, one could pass a wait of a slot's
// older phase.  Units are released by the softmax and by the widening warps.
#include <algorithm>

#include "attn8_dev.cuh"
#include "attn_tile.cuh"

namespace tern {

__device__ unsigned int g_attn8_tile_error;

namespace {

using namespace attn;

// a warp each for copies, MMAs, queries and units; two warpgroups of softmax; four
// warps that widen codes
constexpr int THREADS = 512;

template <int D>
struct Tile8 {
  static constexpr int TKT = D == 256 ? 64 : 128;        // keys of a tile
  static constexpr int RT = 128;
  static constexpr int PAD = D == 64 ? 3 : 2;             // as for the 16-bit cache
  static constexpr int LEAST = PAD + 1;
  static constexpr int SLOT = TKT * D * 2;               // a tile in fp16
  static constexpr int RAW = TKT * D;                    // and as codes
  static constexpr int ROWB = D < 128 ? D : 128;
  static constexpr int QB = 128 * D * 2;
  static constexpr int SLOTS = D == 256 ? 3 : D == 128 ? 4 : 6;
  static constexpr int RAWS = D == 64 ? 6 : 3;
  static constexpr size_t SMEM = size_t(SLOTS) * SLOT + size_t(RAWS) * RAW + QB + 1024;
  static constexpr int AHEAD = 2;                         // tiles that S runs ahead
  static constexpr int NS = 3;                            // buffers of S
  static constexpr int NU = 4;                            // tiles' units that are held (even)
  static constexpr uint32_t S_COL = 0, O_COL = D < 256 ? 384 : 256;
  static_assert(SMEM + 18 * 1024 <= 232448, "shared memory");
};

__device__ __forceinline__ void fail(volatile int* abort_flag, unsigned int code) {
  *abort_flag = 1;
  atomicOr(&g_attn8_tile_error, code);
}

// What a row's exponents refer to is the largest t_j + log2 vu_j less kRef, when it
// is set; it moves when that grows by more than 2^kMove.  Up to 2^kTop, which a
// bound has to say for a tile, fp16 holds what is rounded to it (its largest is just
// below 2^16).  So what is rounded has 2^-25 where it has no exponent left and
// 2^kRef at the row's largest: 2^-33 of that, 2^-32 in folded tiles, whose values
// are multiplied by the unit's fraction of up to 2 behind it.  A reference 2^3 below
// lost small probabilities that 32-bit sums count, but looked for the maximum less
// often: 4 x 29 drafts over up to 20003 keys 89 us, now 94.
constexpr float kRef = 8.f, kMove = 7.9f, kTop = 15.9f;

// The units of a tile: the largest and least of the keys, and of the values.  A
// value unit of 0 (a row of zeros, or a page out of range) bounds no probability,
// so a tile that has one is exact: there it is multiplied by the probability in
// 32 bits, before that is rounded.
struct TileUnits {
  float k_most, k_least, v_most;
  int e;             // exponent of v_most
  bool fold;         // the values' units are within 2^8 of each other
};
__device__ __forceinline__ TileUnits tile_units(const float4& q) {
  TileUnits u;
  u.k_most = q.x;
  u.k_least = q.y;
  u.v_most = q.z;
  u.fold = q.z >= 0x1p-100f && q.z <= 256.f * q.w;
  u.e = q.z == 0.f ? 0 : (__float_as_int(q.z) >> 23) - 127;
  return u;
}

__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(x)), "l"(reinterpret_cast<uint64_t&>(y)));
  return d;
}

__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
      : "memory");
}

template <bool BF16, int KIND, int D>
__global__ void __launch_bounds__(THREADS, 1)
    attn8_tile_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ Args8 g) {
  using C = Tile8<D>;
  constexpr int TKT = C::TKT, RT = C::RT, SLOTS = C::SLOTS, RAWS = C::RAWS, NS = C::NS, NU = C::NU;
  constexpr int HB = TKT * 128;          // 64 columns of a key or value tile in fp16
  const Args& a = g.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sq = ring + SLOTS * C::SLOT;
  uint8_t* codes = sq + C::QB;
  __shared__ uint64_t full[SLOTS], empty[SLOTS], raw_full[RAWS], raw_empty[RAWS], u_full[NU], u_ready[NU],
      u_empty[NU];
  __shared__ uint64_t q_full, q_ready, q_empty, o_full, done, s_full[NS], p_full[NS];
  // out of an even or odd tile added (of the two, only one can be in flight when
  // its phase is awaited); a tile's maximum known
  __shared__ uint64_t o_step[2], m_ready[4];
  __shared__ __align__(16) float s_ku[NU][TKT], s_vu[NU][TKT], s_lu[NU][TKT];   // units, log2 of the values'
  __shared__ __align__(16) uint2 s_fold[NU][TKT];  // folded tiles: a value's unit over 2^E in two fp16 parts
  __shared__ __align__(16) float4 s_range[NU];     // units: largest and least of keys, of values
  __shared__ float s_scale[4][128];      // of four items' rows: S may run three items ahead
  __shared__ float s_m[128];
  __shared__ PieceScratch<THREADS> scratch;
  __shared__ float2 s_ml[2][128];
  __shared__ int s_abort;
  __shared__ uint32_t s_tmem;
  volatile int* abort_flag = &s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < SLOTS; ++s) {
      ptx::mbar_init(&full[s], 4);
      ptx::mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < RAWS; ++s) {
      ptx::mbar_init(&raw_full[s], 1);
      ptx::mbar_init(&raw_empty[s], 4);
    }
    for (int s = 0; s < NU; ++s) {
      ptx::mbar_init(&u_full[s], 1);
      ptx::mbar_init(&u_ready[s], 1);
      ptx::mbar_init(&u_empty[s], 8);      // softmax and widening of values
    }
    ptx::mbar_init(&q_full, 1);
    ptx::mbar_init(&q_ready, 4);
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
    ptx::mbar_fence_init();
    ptx::prefetch_tmap(&tm_k);
    ptx::prefetch_tmap(&tm_v);
    ptx::prefetch_tmap(&tm_q);
  }
  s_scale[tid >> 7][tid & 127] = 1.f;
  if (warp == 2) {
    ptx::tmem_alloc(&s_tmem, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  pdl_wait();
  pdl_launch_dependents();
  const Piece piece = find_piece<TKT, C::PAD, C::LEAST, THREADS>(a, scratch);   // synchronises the CTA
  ptx::tc_fence_after();
  const uint32_t tmem = s_tmem;
  if (tid == 128) a.items[blockIdx.x].follow = 0;   // the thread that may set it below
  const int stream_rows = a.tile_rows;              // at most 128, whole tokens
  Walk<TKT, C::PAD> walk(a, piece);
  Seg s{};

  if (warp == 0) {
    // ---------------- producer: codes in the ring's order, and the keys' and
    // values' units with a tile's keys.  One warp for both: a wait for a slot's
    // phase tells it from the phase two uses before only if the warp knows that
    // one to be over, which two warps of a short ring do not.
    uint32_t seq0 = 0, tile0 = 0;
    uint32_t mine = 0, parity = 0;      // slots filled last, and their phases
    uint32_t u_mine = 0, u_parity = 0;
    bool ok = true;
    const int box_shift = min(a.page_shift, TKT == 128 ? 7 : 6);
    // a lane has one page's box of one part; the first part's lanes also the units.
    // A page out of range gives zeros: of codes by the copy, of units by the lane.
    constexpr int PARTS = D / C::ROWB;
    const int box = lane / PARTS, part = lane % PARTS;
    while (ok && walk.next(s)) {
      const int cnt = s.t1 - s.t0;
      int pages[3] = {0, 0, 0};         // of the tiles whose values are still to come
      int next = page_at<TKT>(a, s, s.t0, box_shift, lane);
      int ik = 0, iv = 0;
      for (int n = 0; n < 2 * cnt; ++n) {
        const bool key = ik < cnt && k_place<C::AHEAD>(ik) == static_cast<uint32_t>(n);
        const int i = key ? ik++ : iv++;
        int page;
        if (key) {
          page = next;
          if (i + 1 < cnt) next = page_at<TKT>(a, s, s.t0 + i + 1, box_shift, lane);
          const int held = i - iv;      // at most AHEAD
          if (held == 0) pages[0] = page;
          else if (held == 1) pages[1] = page;
          else pages[2] = page;
        } else {
          page = pages[0];
          pages[0] = pages[1];
          pages[1] = pages[2];
        }
        const uint32_t nn = seq0 + n, sl = nn % RAWS, par = (nn / RAWS) & 1u;
        const uint32_t us = (tile0 + i) % NU, u_par = ((tile0 + i) / NU) & 1u;
        ok = ptx::mbar_wait_warp(&raw_empty[sl], par ^ 1u, abort_flag, WAIT_LIMIT);
        if (ok && key) ok = ptx::mbar_wait_warp(&u_empty[us], u_par ^ 1u, abort_flag, WAIT_LIMIT);
        if (!ok) {
          if (lane == 0 && !*abort_flag) fail(abort_flag, ERR_PRODUCER);
          break;
        }
        const int k0 = (s.t0 + i) * TKT;
        const int keys = min(TKT, s.r.len - k0);
        const int boxes = keys > 0 ? (keys + (1 << box_shift) - 1) >> box_shift : 0;
        const int pg = __shfl_sync(~0u, page, box);
        const bool here = box < boxes, known = pg < a.pages;
        const bool units = key && here && part == 0;
        if (units && !known)
          for (int e = 0; e < (1 << box_shift); ++e)
            s_ku[us][(box << box_shift) + e] = s_vu[us][(box << box_shift) + e] = 0.f;
        const int with_units = __popc(__ballot_sync(~0u, units && known));
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(&raw_full[sl], static_cast<uint32_t>(boxes * D) << box_shift);
          if (key) ptx::mbar_arrive_expect_tx(&u_full[us], static_cast<uint32_t>(with_units * 8) << box_shift);
        }
        __syncwarp();
        if (here) {
          const int row = k0 & ((1 << a.page_shift) - 1);
          tma_load_4d(codes + sl * C::RAW + part * (TKT * C::ROWB) + (box << box_shift) * C::ROWB,
                      key ? &tm_k : &tm_v, &raw_full[sl], part * 128, row, s.h, pg);
          if (units && known) {
            const int64_t from = pg * g.unit_page + s.h * g.unit_head + row;
            ptx::bulk_load(&s_ku[us][box << box_shift], g.ku + from, 4u << box_shift, &u_full[us]);
            ptx::bulk_load(&s_vu[us][box << box_shift], g.vu + from, 4u << box_shift, &u_full[us]);
          }
        }
        mine |= 1u << sl;
        parity = (parity & ~(1u << sl)) | (par << sl);
        if (key) {
          u_mine |= 1u << us;
          u_parity = (u_parity & ~(1u << us)) | (u_par << us);
        }
      }
      seq0 += 2u * cnt;
      tile0 += cnt;
    }
    // something gave up: the copies land before the CTA exits
    if (!ok || *abort_flag) {
      for (int sl = 0; sl < RAWS; ++sl)
        if (((mine >> sl) & 1u) && !ptx::mbar_wait_bounded(&raw_full[sl], (parity >> sl) & 1u, WAIT_LIMIT))
          atomicOr(&g_attn8_tile_error, ERR_DRAIN);
      for (int us = 0; us < NU; ++us)
        if (((u_mine >> us) & 1u) && !ptx::mbar_wait_bounded(&u_full[us], (u_parity >> us) & 1u, WAIT_LIMIT))
          atomicOr(&g_attn8_tile_error, ERR_DRAIN);
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer, as for the 16-bit cache
    bool ok = true;
    uint32_t seq0 = 0, q_phase = 0, p_phase = 0;
    uint32_t tile0 = 0;      // tiles of the items before
    const auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!ok) return;
      ok = ptx::mbar_wait_warp(bar, parity, abort_flag, WAIT_LIMIT);
      if (!ok && lane == 0 && !*abort_flag) fail(abort_flag, ERR_CONSUMER);
      ptx::tc_fence_after();
    };
    const uint64_t q_desc = ptx::sw128_kmajor_desc(ptx::smem_u32(sq));
    const uint64_t k_desc = ptx::sw128_kmajor_desc(ptx::smem_u32(ring));
    const uint64_t v_desc = sw128_mn_desc(ptx::smem_u32(ring), HB);
    const uint32_t tm = __shfl_sync(~0u, tmem, 0);
    // a negative scale turns the queries' signs
    const uint32_t s_idesc = idesc<false>(TKT, false) | (a.scale_log2 < 0.f ? 1u << 13 : 0u);
    while (ok && __any_sync(~0u, walk.next(s))) {
      const int cnt = __shfl_sync(~0u, s.t1 - s.t0, 0);
      const auto begin = [&](int i, int x) {        // S of tile i
        const uint32_t nk = seq0 + k_place<C::AHEAD>(i), sk = nk % SLOTS;
        wait(&full[sk], (nk / SLOTS) & 1u);
        if (ok && elect_one()) {
          const uint64_t db = k_desc + sk * (C::SLOT >> 4);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            ptx::mma_f16_ss(tm + C::S_COL + TKT * x, q_desc + ((k >> 2) * (128 * 128 >> 4) + 2 * (k & 3)),
                            db + ((k >> 2) * (HB >> 4) + 2 * (k & 3)), s_idesc, k > 0);
          ptx::mma_commit(&empty[sk]);
          ptx::mma_commit(&s_full[x]);
          if (i == cnt - 1) ptx::mma_commit(&q_empty);   // the item's queries were read
        }
        __syncwarp();
      };
      const auto step = [&](int i, int x) {         // out += P V of tile i
        const uint32_t nv = seq0 + v_place<C::AHEAD>(i, cnt), sv = nv % SLOTS;
        wait(&full[sv], (nv / SLOTS) & 1u);
        wait(&p_full[x], (p_phase >> x) & 1u);
        p_phase ^= 1u << x;
        if (!ok) return;
        const uint64_t dv = v_desc + sv * (C::SLOT >> 4);
        // steps of 16 keys up to the request's last
        const int steps = __shfl_sync(~0u, (min(s.r.len - (s.t0 + i) * TKT, TKT) + 15) >> 4, 0);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < TKT / 16; ++k)
            if (k == 0 || k < steps)
              ptx::mma_f16_ts(tm + C::O_COL, tm + C::S_COL + TKT * x + TKT / 2 + k * 8, dv + k * (2048 >> 4),
                              idesc<false>(D, true), (i > 0 || k > 0) ? 1u : 0u);
          ptx::mma_commit(&o_step[(tile0 + i) & 1u]);
          ptx::mma_commit(&empty[sv]);
        }
        __syncwarp();
      };
      wait(&q_ready, q_phase);
      q_phase ^= 1u;
      // S of tile i + 2 goes to the buffer whose P the MMA before read
      for (int i = 0; i < min(cnt, 2); ++i) begin(i, (tile0 + i) % NS);
      for (int i = 0; i < cnt && ok; ++i) {
        if (i + 2 < cnt) begin(i + 2, (tile0 + i + 2) % NS);
        step(i, (tile0 + i) % NS);
      }
      tile0 += cnt;
      if (ok && elect_one()) ptx::mma_commit(&o_full);
      __syncwarp();
      seq0 += 2u * cnt;
    }
    // every MMA issued has completed once `done` fires
    if (elect_one()) ptx::mma_commit(&done);
    __syncwarp();
    if (!ptx::mbar_wait_bounded(&done, 0, WAIT_LIMIT)) atomicOr(&g_attn8_tile_error, ERR_DRAIN);
  } else if (warp == 2) {
    // ---------------- queries: an item's rows, as soon as the item before
    // needs its own no more (whole tokens with the heads of the group)
    constexpr int HALVES = D / 64;
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
      if (lane == 0) ptx::mbar_arrive_expect_tx(&q_full, static_cast<uint32_t>(stream_rows) * D * 2);
      __syncwarp();
      if (lane < HALVES)
        ptx::tma_load_3d(sq + lane * (128 * 128), &tm_q, &q_full, lane * 64, s.h * a.group,
                         s.r.row0 + s.rt * tokens);
    }
    if (!ptx::mbar_wait_bounded(&q_full, parity, WAIT_LIMIT)) atomicOr(&g_attn8_tile_error, ERR_DRAIN);
  } else if (warp == 3) {
    // ---------------- units: what the softmax and the widening of values take of
    // them
    bool ok = true;
    uint32_t tile0 = 0;
    constexpr int EACH = TKT / 32;
    while (ok && walk.next(s)) {
      const int cnt = s.t1 - s.t0;
      for (int i = 0; i < cnt; ++i) {
        const uint32_t us = (tile0 + i) % NU;
        ok = ptx::mbar_wait_warp(&u_full[us], ((tile0 + i) / NU) & 1u, abort_flag, WAIT_LIMIT);
        if (!ok) {
          if (lane == 0 && !*abort_flag) fail(abort_flag, ERR_CONSUMER);
          break;
        }
        float4 q = make_float4(0.f, INFINITY, 0.f, INFINITY);
        float vu[EACH];
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
          const float ku = s_ku[us][e * 32 + lane];
          vu[e] = s_vu[us][e * 32 + lane];
          s_lu[us][e * 32 + lane] = __log2f(fmaxf(vu[e], kLeastUnit));
          q = make_float4(fmaxf(q.x, ku), fminf(q.y, ku), fmaxf(q.z, vu[e]), fminf(q.w, vu[e]));
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
          q.x = fmaxf(q.x, __shfl_xor_sync(~0u, q.x, d));
          q.y = fminf(q.y, __shfl_xor_sync(~0u, q.y, d));
          q.z = fmaxf(q.z, __shfl_xor_sync(~0u, q.z, d));
          q.w = fminf(q.w, __shfl_xor_sync(~0u, q.w, d));
        }
        if (lane == 0) s_range[us] = q;
        const float by = __int_as_float(max(127 - tile_units(q).e, 1) << 23);
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
          const float f = vu[e] * by;
          const __half hi = __float2half_rn(f), lo = __float2half_rn(f - __half2float(hi));
          const __half2 h2 = __half2half2(hi), l2 = __half2half2(lo);
          s_fold[us][e * 32 + lane] =
              make_uint2(*reinterpret_cast<const uint32_t*>(&h2), *reinterpret_cast<const uint32_t*>(&l2));
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&u_ready[us]);
      }
      tile0 += cnt;
    }
  } else if (warp >= 12) {
    // ---------------- codes to fp16, in the ring's order: 128 threads
    const int t = tid - 384;
    bool ok = true;
    uint32_t seq0 = 0, tile0 = 0, q_phase = 0, item = 0;
    const auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!ok) return;
      ok = ptx::mbar_wait_warp(bar, parity, abort_flag, WAIT_LIMIT);
      if (!ok && lane == 0 && !*abort_flag) fail(abort_flag, ERR_CONSUMER);
    };
    while (ok && walk.next(s)) {
      const int cnt = s.t1 - s.t0;
      wait(&q_full, q_phase);
      q_phase ^= 1u;
      if (!ok) break;
      if (BF16 && t < stream_rows) {
        // a thread has a row: its largest exponent, then 2^13 over that (in two
        // factors, as it may pass 2^127); a row with an infinity or NaN stays
        const auto at = [&](int c) {
          return reinterpret_cast<uint4*>(sq + (c >> 3) * (128 * 128) + t * 128 + (((c & 7) ^ (t & 7)) << 4));
        };
        uint32_t top = 0;
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          const uint4 w = *at(c);
          const uint32_t m = 0x7F807F80u;
          top = __vmaxu2(top, __vmaxu2(__vmaxu2(w.x & m, w.y & m), __vmaxu2(w.z & m, w.w & m)));
        }
        top = max(top & 0xFFFFu, top >> 16);
        const int up = top == 0x7F80u ? 0 : 140 - max(static_cast<int>(top >> 7), 1);
        const float f0 = __int_as_float((127 + up / 2) << 23), f1 = __int_as_float((127 + up - up / 2) << 23);
#pragma unroll 2
        for (int c = 0; c < D / 8; ++c) {
          uint4 w = *at(c);
          uint32_t* x = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[e] = pack2<false>(__uint_as_float(x[e] << 16) * f0 * f1, __uint_as_float(x[e] & 0xFFFF0000u) * f0 * f1);
          *at(c) = w;
        }
        s_scale[item & 3][t] = __int_as_float((127 - up / 2) << 23) * __int_as_float((127 - (up - up / 2)) << 23);
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&q_ready);
      int ik = 0, iv = 0;
      for (int n = 0; n < 2 * cnt && ok; ++n) {
        const bool key = ik < cnt && k_place<C::AHEAD>(ik) == static_cast<uint32_t>(n);
        const int i = key ? ik++ : iv++;
        const uint32_t nn = seq0 + n, sl = nn % SLOTS, rs = nn % RAWS;
        const uint32_t us = (tile0 + i) % NU;
        if (!key) wait(&u_ready[us], ((tile0 + i) / NU) & 1u);
        wait(&raw_full[rs], (nn / RAWS) & 1u);
        wait(&empty[sl], ((nn / SLOTS) & 1u) ^ 1u);
        if (!ok) break;
        // a thread has the same 16-code chunk of every 128 / CH-th row, so that all
        // its places are constants apart.  A chunk becomes two 8-value chunks of
        // a 64-column part; where two lanes of eight would meet in a bank, one
        // takes its halves the other way round.
        constexpr int CH = D / 16, STEP = 128 / CH, ROWS = TKT / STEP;
        const int c = t % CH, r0 = t / CH;
        const bool turn = D >= 128 && (c & 4) != 0;
        const uint8_t* from = codes + rs * C::RAW + (c >> 3) * (TKT * C::ROWB) + chunk_at<C::ROWB>(r0, c & 7);
        uint8_t* row = ring + sl * C::SLOT + (c >> 2) * HB + r0 * 128;
        uint8_t* to0 = row + ((((c & 3) * 2 + (turn ? 1 : 0)) ^ (r0 & 7)) << 4);
        uint8_t* to1 = row + ((((c & 3) * 2 + (turn ? 0 : 1)) ^ (r0 & 7)) << 4);
        const int k0 = (s.t0 + i) * TKT;
        const bool fold = BF16 && !key && k0 <= s.r.ctx - TKT && tile_units(s_range[us]).fold;
        const int keys = key ? TKT : s.r.len - k0;        // values past the last token count as zero
        const auto turned = [&](uint4 w, uint32_t (&o)[8]) {
          widen<KIND>(turn ? w.z : w.x, o[0], o[1]);
          widen<KIND>(turn ? w.w : w.y, o[2], o[3]);
          widen<KIND>(turn ? w.x : w.z, o[4], o[5]);
          widen<KIND>(turn ? w.y : w.w, o[6], o[7]);
        };
        const auto store = [&](int p, const uint32_t (&o)[8]) {
          *reinterpret_cast<uint4*>(to0 + p * STEP * 128) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(to1 + p * STEP * 128) = make_uint4(o[4], o[5], o[6], o[7]);
        };
        const auto codes_of = [&](int p) { return *reinterpret_cast<const uint4*>(from + p * STEP * C::ROWB); };
        // loads ahead of the stores, as the compiler does not know that they are
        // apart; one loop for all tiles, so that the kernel's loops fit the
        // instruction cache
        constexpr int AT = 4;
        const uint2 one = make_uint2(0x3C003C00u, 0u);
#pragma unroll 1
        for (int p0 = 0; p0 < ROWS; p0 += AT) {
          uint4 w[AT];
          uint2 f[AT];
#pragma unroll
          for (int p = 0; p < AT; ++p) {
            w[p] = codes_of(p0 + p);
            f[p] = fold ? s_fold[us][r0 + (p0 + p) * STEP] : one;
            if (r0 + (p0 + p) * STEP >= keys) w[p] = make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int p = 0; p < AT; ++p) {
            uint32_t o[8];
            turned(w[p], o);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = ptx::fma_f16x2(o[e], f[p].x, ptx::mul_f16x2(o[e], f[p].y));
            store(p0 + p, o);
          }
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(&full[sl]);
          ptx::mbar_arrive(&raw_empty[rs]);
          if (!key) ptx::mbar_arrive(&u_empty[us]);
        }
      }
      seq0 += 2u * cnt;
      tile0 += cnt;
      ++item;
    }
  } else if (warp >= 4) {
    // ---------------- softmax and output: the warpgroups take the tiles in turn, a
    // thread one row
    const int x = (warp - 4) >> 2;
    const int lrow = (warp & 3) * 32 + lane;           // row of the tile, its lane
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t o_addr = tmem + C::O_COL + lane_addr;
    const int wid = tid - 128;                         // 0 .. 255
    // the maximum is taken of scaled products, so the scale must not be negative
    // (the MMA turns the queries' signs instead) nor zero
    const float scale = fmaxf(fabsf(a.scale_log2), 1e-37f);
    bool ok = true;
    uint32_t o_phase = 0;
    uint32_t tile0 = 0, item = 0;                      // tiles of the items before
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
      const bool has = lrow < rows;
      const bool active = (warp & 3) * 32 < rows;
      const int tok = has ? div_group(a, r0 + lrow) : 0;
      const uint64_t* mw = a.mask != nullptr ? a.mask + (s.r.row0 + int64_t(tok)) * a.mask_words : nullptr;
      const uint64_t word0 = first_word(a, mw);
      float m = -INFINITY, l = 0.f;
      for (int i = (tile0 + x) & 1; i < cnt; i += 2) {
        const int buf = (tile0 + i) % NS;
        const uint32_t us = (tile0 + i) % NU;
        const uint32_t s_addr = tmem + C::S_COL + TKT * buf + lane_addr;
        const int k0 = (s.t0 + i) * TKT;
        const bool edge = k0 > s.r.ctx - TKT;
        uint64_t vis[TKT / 64];
        if (edge && active) {
#pragma unroll
          for (int c = 0; c < TKT / 64; ++c)
            vis[c] = sees64(a, mw, word0, tok, k0 + 64 * c, s.r.ctx, s.r.len);
        }
        wait(&u_ready[us], ((tile0 + i) / NU) & 1u);
        wait(&s_full[buf], ((tile0 + i) / NS) & 1u);
        if (!ok) break;
        if (active) {
          // a row of S is read twice, 16 columns at a time with the next on their
          // way (32 at a time spilled registers)
          constexpr int NC = TKT / 16;
          const float rs = scale * s_scale[item & 3][lrow];
          const float2 rs2 = make_float2(rs, rs);
          uint32_t v[2][16];
          const TileUnits tu = tile_units(s_range[us]);
          const bool fold = BF16 && !edge && tu.fold;
          // the largest score: the last columns stay for the second pass
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          const auto largest = [&](const uint32_t (&x)[16]) {
#pragma unroll
            for (int e = 0; e < 16; e += 2)
              mx[(e >> 1) & 3] = fmaxf(mx[(e >> 1) & 3], fmaxf(__uint_as_float(x[e]), __uint_as_float(x[e + 1])));
          };
          ptx::tmem_ld_32x32b_x16(s_addr, v[0]);
#pragma unroll 1
          for (int c = 0; c < NC; c += 2) {
            tmem_ld_wait_for(v[0]);
            ptx::tmem_ld_32x32b_x16(s_addr + 16 * (c + 1), v[1]);
            largest(v[0]);
            tmem_ld_wait_for(v[1]);
            if (c + 2 < NC) ptx::tmem_ld_32x32b_x16(s_addr + 16 * (c + 2), v[0]);
            largest(v[1]);
          }
          const float most = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * rs;
          float mp = -INFINITY;   // the other warpgroup's, of the tile before
          if (i > 0) {
            wait(&m_ready[warp & 3], (tile0 + i - 1) & 1u);
            mp = *reinterpret_cast<volatile float*>(&s_m[lrow]);
          }
          const float top = (most > 0.f ? most * tu.k_most : most * tu.k_least) + __log2f(fmaxf(tu.v_most, kLeastUnit));
          float mn = mp;
          if (edge || __any_sync(~0u, !(top <= mp + kTop))) {
            // the maximum itself, of what the row sees; tt of scores alone
            float mt = -INFINITY, tt = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < TKT / 16; ++c) {
              uint32_t x[16];
              ptx::tmem_ld_32x32b_x16(s_addr + 16 * c, x);
              tmem_ld_wait_for(x);
              const uint32_t bits = edge ? static_cast<uint32_t>(vis[TKT == 64 ? 0 : c >> 2] >> (16 * (c & 3))) : ~0u;
              const float4* ku = reinterpret_cast<const float4*>(&s_ku[us][16 * c]);
              const float4* lu = reinterpret_cast<const float4*>(&s_lu[us][16 * c]);
#pragma unroll
              for (int e = 0; e < 16; e += 4) {
                const float4 k4 = ku[e >> 2], l4 = lu[e >> 2];
                const float y[4] = {__uint_as_float(x[e]) * rs * k4.x, __uint_as_float(x[e + 1]) * rs * k4.y,
                                    __uint_as_float(x[e + 2]) * rs * k4.z, __uint_as_float(x[e + 3]) * rs * k4.w};
                const float lg[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
                for (int h = 0; h < 4; ++h)
                  if ((bits >> (e + h)) & 1) {
                    tt = fmaxf(tt, y[h]);
                    mt = fmaxf(mt, y[h] + lg[h]);
                  }
              }
            }
            mt -= kRef;
            if (mt > mp + kMove || (mp == -INFINITY && mt != mp)) mn = mt;
            if (fold) mn = fmaxf(mn, tt + static_cast<float>(tu.e) - kTop);
          }
          *reinterpret_cast<volatile float*>(&s_m[lrow]) = mn;
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&m_ready[warp & 3]);
          const float f = mn != m ? ex2(m - mn) : 1.f;      // of this thread's sum
          m = mn;
          const float fo = mn != mp ? ex2(mp - mn) : 1.f;   // of the accumulator
          bool move = i > 0 && __any_sync(~0u, fo != 1.f);
          if (move) {
            wait(&o_step[(tile0 + i - 1) & 1u], ((tile0 + i - 1) >> 1) & 1u);
            move = ok;
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
          // folded: what the values were divided by comes with the probabilities
          const float ms = (m == -INFINITY ? 0.f : m) - (fold ? static_cast<float>(tu.e) : 0.f);
          const float2 ms2 = make_float2(-ms, -ms);
          float2 sum[2] = {};
          // from the last columns, which are there, down: P goes over the upper
          // half of S, behind what is still to be read
          if (BF16 ? fold : !edge) {
            const auto step = [&](const uint32_t (&x)[16], int c) {
              const float4* ku = reinterpret_cast<const float4*>(&s_ku[us][16 * c]);
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 16; e += 4) {
                const float4 k4 = ku[e >> 2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const int j = e + 2 * h;
                  const float2 y = fma2(mul2(make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), rs2),
                                        h ? make_float2(k4.z, k4.w) : make_float2(k4.x, k4.y), ms2);
                  float2 p = make_float2(ex2(y.x), ex2(y.y));
                  sum[h] = add2(sum[h], p);
                  if constexpr (!BF16) p = mul2(p, *reinterpret_cast<const float2*>(&s_vu[us][16 * c + j]));
                  w[j >> 1] = pack2<false>(p.x, p.y);
                }
              }
              tmem_st_x8(s_addr + TKT / 2 + 8 * c, w);
            };
#pragma unroll 1
            for (int c = NC - 1; c > 0; c -= 2) {
              tmem_ld_wait_for(v[1]);
              ptx::tmem_ld_32x32b_x16(s_addr + 16 * (c - 1), v[0]);
              step(v[1], c);
              tmem_ld_wait_for(v[0]);
              if (c > 1) ptx::tmem_ld_32x32b_x16(s_addr + 16 * (c - 2), v[1]);
              step(v[0], c - 1);
            }
          } else {
            // short code rather than reads ahead: longer code slows the other loops, and
            // the wide trees above take 97 us, not 94, when all of their tiles come here
            // (a zero-valued token in each page)
#pragma unroll 1
            for (int c = NC - 1; c >= 0; --c) {
              ptx::tmem_ld_32x32b_x16(s_addr + 16 * c, v[0]);
              tmem_ld_wait_for(v[0]);
              const uint32_t bits = edge ? static_cast<uint32_t>(vis[TKT == 64 ? 0 : c >> 2] >> (16 * (c & 3))) : ~0u;
              uint32_t w[8];
#pragma unroll
              for (int j = 0; j < 16; j += 2) {
                const float2 ku = *reinterpret_cast<const float2*>(&s_ku[us][16 * c + j]);
                const float2 vu = *reinterpret_cast<const float2*>(&s_vu[us][16 * c + j]);
                const float2 y = fma2(mul2(make_float2(__uint_as_float(v[0][j]), __uint_as_float(v[0][j + 1])), rs2), ku, ms2);
                float2 p = make_float2(ex2(y.x), ex2(y.y));
                float2 pv = mul2(p, vu);
                if (!((bits >> j) & 1)) p.x = pv.x = 0.f;
                if (!((bits >> (j + 1)) & 1)) p.y = pv.y = 0.f;
                sum[(j >> 1) & 1] = add2(sum[(j >> 1) & 1], p);
                w[j >> 1] = pack2<false>(pv.x, pv.y);
              }
              tmem_st_x8(s_addr + TKT / 2 + 8 * c, w);
            }
          }
          const float2 all = add2(sum[0], sum[1]);
          l = l * f + (all.x + all.y) * (fold ? ex2(-static_cast<float>(tu.e)) : 1.f);
          ptx::tmem_st_wait();
        } else if (lane == 0) {
          ptx::mbar_arrive(&m_ready[warp & 3]);    // its phases count tiles, whoever is active
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(&p_full[buf]);
          ptx::mbar_arrive(&u_empty[us]);
        }
      }
      // ---- the item's part is complete
      wait(&o_full, o_phase);
      o_phase ^= 1u;
      tile0 += cnt;
      ++item;
      s_ml[x][lrow] = make_float2(m, l);
      ptx::named_sync(1, 256);
      const bool whole = s.t0 == 0 && s.t1 == s.r.tiles;
      const int64_t slot = 2 * int64_t(blockIdx.x) + (s.t0 == 0 ? 1 : 0);
      if (ok && active) {
        const float2 y = s_ml[x ^ 1][lrow];          // the sums of both warpgroups' tiles
        const float mm = fmaxf(m, y.x);
        l = l * (mm == -INFINITY ? 0.f : ex2(m - mm)) + y.y * (mm == -INFINITY ? 0.f : ex2(y.x - mm));
        m = mm;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t at = (int64_t(s.r.row0) + tok) * a.Hq + s.h * a.group + (r0 + lrow - tok * a.group);
        // this warpgroup's half of the columns, which refer to the larger maximum already
        constexpr int HALF = D / 2;
        const int col0 = x * HALF;
#pragma unroll 1
        for (int c = 0; c < HALF / 16; ++c) {
          uint32_t u[16];
          ptx::tmem_ld_32x32b_x16(o_addr + col0 + 16 * c, u);
          tmem_ld_wait_for(u);
          if (!has) continue;
          float o[16];
          const float fo = whole ? inv : 1.f;
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __uint_as_float(u[e]) * fo;
          const int d = col0 + 16 * c;
          if (whole) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
              *reinterpret_cast<uint4*>(a.out + at * D + d + 8 * e) =
                  make_uint4(pack2<BF16>(o[8 * e], o[8 * e + 1]), pack2<BF16>(o[8 * e + 2], o[8 * e + 3]),
                             pack2<BF16>(o[8 * e + 4], o[8 * e + 5]), pack2<BF16>(o[8 * e + 6], o[8 * e + 7]));
          } else {
            float* po = a.part_o + ((slot * (D / 4) + d / 4) * RT + lrow) * 4;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<float4*>(po + 4 * RT * e) =
                  make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
        if (has && x == 0) {
          if (!whole)
            a.part_ml[slot * RT + lrow] = make_float2(m, l);
          else if (a.lse != nullptr)
            a.lse[at] = l == 0.f ? -INFINITY : lse_of<BF16>(m, l);
        }
      }
      if (!whole && s.t0 == 0 && wid == 0) {
        const int first = static_cast<int>(blockIdx.x);
        a.items[first] = Item{first, cta_of(piece, s.end - 1) - first, s.r.row0, r0, rows, s.h};
      }
      ptx::tc_fence_before();
      ptx::named_sync(1, 256);   // accumulators and s_ml are free again
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 2) ptx::tmem_dealloc(tmem, 512);
}

template <bool BF16, int KIND, int D>
cudaError_t launch_tile8(const TreeAttn8Call& call, Args8 g, cudaStream_t st) {
  using C = Tile8<D>;
  static std::atomic<unsigned long long> attr_done{0};
  cudaError_t e = once_per_device(attr_done, [] {
    return cudaFuncSetAttribute(attn8_tile_kernel<BF16, KIND, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(C::SMEM));
  });
  if (e != cudaSuccess) return e;
  const int grid = std::min(kv_sm_count(), MAX_GRID8);
  const int box = static_cast<int>(std::min<int64_t>(call.cache.page_size, C::TKT));
  const int tokens = 128 / g.a.group;
  CUtensorMap tk, tv, tq;
  if (!make_map8(&tk, call.cache, call.cache.k, box) || !make_map8(&tv, call.cache, call.cache.v, box) ||
      !make_query_map(&tq, call.q, BF16, D, call.Hq, call.T, call.q_head_stride, call.q_token_stride, tokens,
                      g.a.group))
    return cudaErrorInvalidValue;
  const Ws w = ws_layout(grid, C::RT, D);
  uint8_t* ws = static_cast<uint8_t*>(call.ws);
  g.a.part_o = reinterpret_cast<float*>(ws + w.o);
  g.a.part_ml = reinterpret_cast<float2*>(ws + w.ml);
  g.a.arrived = reinterpret_cast<int*>(ws);
  g.a.items = reinterpret_cast<Item*>(ws + w.items);
  g.a.tile_rows = tokens * g.a.group;
  e = launch(attn8_tile_kernel<BF16, KIND, D>, dim3(grid), dim3(THREADS), C::SMEM, st, tk, tv, tq, g);
  if (e != cudaSuccess) return e;
  return launch(combine_kernel<BF16, D>, dim3(4 * kv_sm_count()), dim3(JOIN_THREADS), 0, st, g.a, C::RT, grid);
}

template <bool BF16, int KIND>
cudaError_t launch_kind(const TreeAttn8Call& call, const Args8& g, cudaStream_t st) {
  if (call.cache.dim == 64) return launch_tile8<BF16, KIND, 64>(call, g, st);
  if (call.cache.dim == 128) return launch_tile8<BF16, KIND, 128>(call, g, st);
  return launch_tile8<BF16, KIND, 256>(call, g, st);
}

}  // namespace

cudaError_t launch_attn8_tile(const TreeAttn8Call& call, const Args8& g, cudaStream_t st) {
  if (call.dtype == TERN_KV_BF16)
    return call.cache.dtype == TERN_KV_I8 ? launch_kind<true, I8>(call, g, st) : launch_kind<true, E4M3>(call, g, st);
  return call.cache.dtype == TERN_KV_I8 ? launch_kind<false, I8>(call, g, st) : launch_kind<false, E4M3>(call, g, st);
}

cudaError_t attn8_tile_read_clear_error(unsigned int* err) {
  cudaError_t e = cudaMemcpyFromSymbol(err, g_attn8_tile_error, sizeof(unsigned int));
  if (e != cudaSuccess || *err == 0) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_attn8_tile_error, &zero, sizeof(unsigned int));
}

}  // namespace tern
