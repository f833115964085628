// Attention of drafted tokens over the paged cache.
//
// For a row (new token with a query head) over the keys j that it sees:
//   t_j = scale log2(e) q . k_j,  m = max t_j,  l = sum 2^(t_j - m),
//   out = sum 2^(t_j - m) v_j / l,  lse = (m + log2 l) ln 2,
// kept over the tiles of a piece as (m, l, unnormalised out) in 32 bits and
// rescaled where m grows.  The probabilities are rounded to the cache's type
// for the second product, as its values are; l sums them unrounded.
//
// attn_rows_kernel: 16 rows an item, tiles of 64 keys.  A producer warp
// copies each page's part of a tile with TMA into a ring; four warps take 16
// keys of a tile each and keep their own (m, l, out) of all 16 rows, so that
// no warp waits for another inside an item; they join at its end.  The
// products are mma.sync m16n8k16.
#include <algorithm>

#include "attn_dev.cuh"

namespace tern {

__device__ unsigned int g_attn_error;

namespace {

using namespace attn;

constexpr uint32_t WAIT_LIMIT = 1u << 18;   // polls of a bounded wait, about a second
enum : unsigned int { ERR_PRODUCER = 1u, ERR_CONSUMER = 2u, ERR_DRAIN = 4u };

__device__ __forceinline__ void fail(volatile int* abort_flag, unsigned int code) {
  *abort_flag = 1;
  atomicOr(&g_attn_error, code);
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t c0, int32_t c1, int32_t c2, int32_t c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(ptx::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(ptx::smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2),
      "r"(c3)
      : "memory");
}

// ------------------------------------------------------------------ rows kernel

constexpr int RT = 16;             // rows of an item
constexpr int TK = 64;             // keys of a tile
constexpr int NW = 4;              // consumer warps
constexpr int THREADS = (NW + 1) * 32;

template <int D>
struct Rows {
  static constexpr int STAGE = 2 * TK * D * 2;            // keys and values of a tile
  static constexpr int STAGES = D == 64 ? 6 : 3;
  static constexpr int CTAS = D == 256 ? 1 : 2;           // per SM
  static constexpr int MERGE = RT * D * 4;
  static constexpr size_t SMEM = size_t(STAGES) * STAGE + MERGE + 1024 + 1024;
};

// One tile's copies, spread over the producer warp: box i of `boxes` covers
// box_rows keys of one page; D / 64 halves of 128 bytes a key (the swizzled
// row), keys then values.
template <int D, int TKEYS>
__device__ __forceinline__ void load_tile(const CUtensorMap* tk, const CUtensorMap* tv,
                                          uint8_t* stage, uint64_t* bar, int page, int boxes,
                                          int box_shift, int row, int h, int lane) {
  constexpr int HALVES = D / 64;
  constexpr int HB = TKEYS * 128;
  for (int i0 = 0; i0 < boxes * HALVES; i0 += 32) {
    const int i = i0 + lane;
    const int box = i / HALVES, half = i % HALVES;
    const int pg = __shfl_sync(~0u, page, box & 31);
    if (i < boxes * HALVES) {
      uint8_t* dst = stage + half * HB + (box << box_shift) * 128;
      tma_load_4d(dst, tk, bar, half * 64, row, h, pg);
      tma_load_4d(dst + HALVES * HB, tv, bar, half * 64, row, h, pg);
    }
  }
}

template <bool BF16, int D>
__global__ void __launch_bounds__(THREADS, Rows<D>::CTAS)
    attn_rows_kernel(const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const Args a) {
  using C = Rows<D>;
  constexpr int HALVES = D / 64;
  constexpr int HB = TK * 128;
  constexpr int KS = D / 16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  float* merge = reinterpret_cast<float*>(ring + C::STAGES * C::STAGE);
  __shared__ uint64_t full[C::STAGES], empty[C::STAGES];
  __shared__ int64_t scratch[THREADS / 32 + 3];
  __shared__ float2 s_ml[NW][RT];
  __shared__ unsigned int s_bad[8];     // new tokens with a non-finite value, by index
  __shared__ int s_any_bad;
  __shared__ int s_abort;
  volatile int* abort_flag = &s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], NW);
    }
    s_abort = 0;
    s_any_bad = 0;
    for (int i = 0; i < 8; ++i) s_bad[i] = 0;
    ptx::mbar_fence_init();
    ptx::prefetch_tmap(&tm_k);
    ptx::prefetch_tmap(&tm_v);
  }
  pdl_wait();
  pdl_launch_dependents();
  const Piece piece = find_piece<TK, RT, THREADS>(a, scratch);   // synchronises the CTA
  if (tid == 0) a.join[blockIdx.x].follow = 0;
  if (piece.lo >= piece.hi) return;
  Walk<TK, RT> walk(a, piece);
  Seg s;

  if (warp == NW) {
    // ---------------- producer
    int st = 0;
    uint32_t phase = 0;
    long issued = 0;
    bool ok = true;
    const int page_rows = 1 << a.page_shift;
    const int box_shift = min(a.page_shift, 6);      // rows of a box: a page, or the tile
    const int per_tile = TK >> box_shift;
    while (ok && walk.next(s)) {
      const int32_t* row = a.table + int64_t(s.b) * a.table_stride;
      // lane i: page of box i of a tile, read one tile ahead
      const auto page_at = [&](int t) {
        const int64_t p = (int64_t(t) * TK + (int64_t(lane) << box_shift)) >> a.page_shift;
        int pg = -1;
        if (lane < per_tile && (int64_t(t) * TK + (int64_t(lane) << box_shift)) < s.r.len)
          pg = row[p];
        return pg < 0 || pg >= a.pages ? a.pages : pg;   // out of range: zeros are copied
      };
      int page = page_at(s.t0);
      for (int t = s.t0; t < s.t1; ++t) {
        const int k0 = t * TK;
        const int keys = min(TK, s.r.len - k0);
        const int boxes = keys > 0 ? (keys + (1 << box_shift) - 1) >> box_shift : 0;
        const int ahead = t + 1 < s.t1 ? page_at(t + 1) : 0;
        ok = ptx::mbar_wait_warp(&empty[st], phase ^ 1u, abort_flag, WAIT_LIMIT);
        if (!ok) {
          if (lane == 0 && !*abort_flag) fail(abort_flag, ERR_PRODUCER);
          break;
        }
        if (lane == 0)
          ptx::mbar_arrive_expect_tx(&full[st],
                                     static_cast<uint32_t>(boxes << box_shift) * D * 4u);
        __syncwarp();
        load_tile<D, TK>(&tm_k, &tm_v, ring + st * C::STAGE, &full[st], page, boxes, box_shift,
                         k0 & (page_rows - 1), s.h, lane);
        page = ahead;
        ++issued;
        if (++st == C::STAGES) {
          st = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) {   // let the copies in flight land before the CTA exits
      const long back = issued < C::STAGES ? issued : C::STAGES;
      for (long i = 0; i < back; ++i) {
        if (--st < 0) {
          st = C::STAGES - 1;
          phase ^= 1u;
        }
        if (!ptx::mbar_wait_bounded(&full[st], phase, WAIT_LIMIT)) atomicOr(&g_attn_error, ERR_DRAIN);
      }
    }
    return;
  }

  // ---------------- consumers: warp w has keys 16 w .. 16 w + 15 of each tile
  int st = 0;
  uint32_t phase = 0;
  const int row_a = lane >> 2;           // this lane's rows: row_a, row_a + 8
  const uint32_t ring_u = ptx::smem_u32(ring);
  // ldmatrix rows: keys by key (matrices: keys 0-7 d 0-7, keys 0-7 d 8-15, keys 8-15 ...)
  const int k_row = warp * 16 + (lane & 7) + ((lane >> 4) << 3);
  const int k_chunk = (lane >> 3) & 1;
  // values transposed (matrices: keys 0-7 d 0-7, keys 8-15 d 0-7, keys 0-7 d 8-15 ...)
  const int v_row = warp * 16 + (lane & 15);
  const int v_chunk = lane >> 4;
  bool ok = true;
  while (walk.next(s)) {
    const int rows_all = s.r.n * a.group;
    const int r0 = s.rt * RT;
    const int rows = min(RT, rows_all - r0);
    // query fragments, rows past the tile's last are zero
    uint32_t qf[KS][4];
    const uint64_t* mw[2] = {nullptr, nullptr};
    int tok[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = r0 + row_a + 8 * e;
      const bool in = r < rows_all;
      tok[e] = in ? r / a.group : 0;
      const int64_t t = s.r.row0 + tok[e];
      if (a.mask != nullptr) mw[e] = a.mask + t * a.mask_words;
      const uint16_t* q = a.q + t * a.q_token +
                          int64_t(s.h * a.group + (in ? r % a.group : 0)) * a.q_head + (lane & 3) * 2;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qf[k][e] = in ? *reinterpret_cast<const uint32_t*>(q + k * 16) : 0u;
        qf[k][e + 2] = in ? *reinterpret_cast<const uint32_t*>(q + k * 16 + 8) : 0u;
      }
    }
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (int t = s.t0; t < s.t1; ++t) {
      // a warp whose wait gave up reads no more tiles, but still meets the
      // others at the barriers below
      if (ok) {
        ok = ptx::mbar_wait_warp(&full[st], phase, abort_flag, WAIT_LIMIT);
        if (!ok && lane == 0 && !*abort_flag) fail(abort_flag, ERR_CONSUMER);
      }
      if (!ok) break;
      const uint32_t kbase = ring_u + st * C::STAGE;
      const uint32_t vbase = kbase + HALVES * HB;
      const int k0 = t * TK + warp * 16;       // this warp's first key
      const bool edge = k0 + 16 > s.r.ctx;     // new tokens, or past the last
      if (edge) {
        // values past the last token count as zero, and so does a non-finite
        // value of a new token here: it is added at the item's end, to the
        // rows that see that token
        uint8_t* vw = ring + st * C::STAGE + HALVES * HB;
        for (int i = lane; i < 16 * (D / 8); i += 32) {
          const int kr = warp * 16 + i / (D / 8), c = i % (D / 8);
          uint4* at = reinterpret_cast<uint4*>(vw + (c >> 3) * HB + kr * 128 +
                                               (((c & 7) ^ (kr & 7)) << 4));
          const int j = t * TK + kr;
          if (j >= s.r.len) {
            *at = make_uint4(0, 0, 0, 0);
          } else if (j >= s.r.ctx) {
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
              const int jj = j - s.r.ctx;
              if (jj < 256) atomicOr(&s_bad[jj >> 5], 1u << (jj & 31));
              s_any_bad = 1;
            }
          }
        }
        ptx::fence_proxy_async_smem();   // before the ring's next copy into this place
        __syncwarp();
      }
      float c[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) c[i][0] = c[i][1] = c[i][2] = c[i][3] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t b[4];
        const int chunk = (k & 3) * 2 + k_chunk;
        ldsm_x4(kbase + (k >> 2) * HB + k_row * 128 + ((chunk ^ (k_row & 7)) << 4), b);
        mma16816<BF16>(c[0], qf[k], b[0], b[1]);
        mma16816<BF16>(c[1], qf[k], b[2], b[3]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) c[i][e] *= a.scale_log2;
      if (edge) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = k0 + i * 8 + (lane & 3) * 2 + (e & 1);
            const bool seen = j < s.r.ctx || (j < s.r.len &&
                              sees(a, mw[e >> 1], tok[e >> 1], j - s.r.ctx, s.r.n));
            if (!seen) c[i][e] = -INFINITY;
          }
      }
      float ms[2], al[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = fmaxf(fmaxf(c[0][2 * e], c[0][2 * e + 1]), fmaxf(c[1][2 * e], c[1][2 * e + 1]));
        x = fmaxf(x, __shfl_xor_sync(~0u, x, 1));
        x = fmaxf(x, __shfl_xor_sync(~0u, x, 2));
        const float mn = fmaxf(m[e], x);
        ms[e] = mn == -INFINITY ? 0.f : mn;
        al[e] = ex2(m[e] - ms[e]);
        m[e] = mn;
      }
      uint32_t p[4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) c[i][e] = ex2(c[i][e] - ms[e >> 1]);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        l[e] = l[e] * al[e] + ((c[0][2 * e] + c[0][2 * e + 1]) + (c[1][2 * e] + c[1][2 * e + 1]));
      p[0] = pack2<BF16>(c[0][0], c[0][1]);
      p[1] = pack2<BF16>(c[0][2], c[0][3]);
      p[2] = pack2<BF16>(c[1][0], c[1][1]);
      p[3] = pack2<BF16>(c[1][2], c[1][3]);
      if (__any_sync(~0u, al[0] != 1.f || al[1] != 1.f)) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][0] *= al[0];
          o[i][1] *= al[0];
          o[i][2] *= al[1];
          o[i][3] *= al[1];
        }
      }
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        uint32_t b[4];
        const int chunk = (i & 3) * 2 + v_chunk;
        ldsm_x4_t(vbase + (i >> 2) * HB + v_row * 128 + ((chunk ^ (v_row & 7)) << 4), b);
        mma16816<BF16>(o[2 * i], p, b[0], b[1]);
        mma16816<BF16>(o[2 * i + 1], p, b[2], b[3]);
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&empty[st]);
      if (++st == C::STAGES) {
        st = 0;
        phase ^= 1u;
      }
    }

    // ---- join the four warps: factors from every warp's (m, l), then the
    // outputs added in the order of the warps
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(~0u, l[e], 1);
      l[e] += __shfl_xor_sync(~0u, l[e], 2);
      if ((lane & 3) == 0) s_ml[warp][row_a + 8 * e] = make_float2(m[e], l[e]);
    }
    ptx::named_sync(1, NW * 32);
    float f[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < NW; ++w) mm = fmaxf(mm, s_ml[w][row_a + 8 * e].x);
      f[e] = mm == -INFINITY ? 0.f : ex2(m[e] - mm);
    }
    for (int w = 0; w < NW; ++w) {
      if (w == warp) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float2* at = reinterpret_cast<float2*>(merge + (row_a + 8 * e) * D + i * 8 + (lane & 3) * 2);
            float2 x = make_float2(o[i][2 * e] * f[e], o[i][2 * e + 1] * f[e]);
            if (w > 0) {
              x.x += at->x;
              x.y += at->y;
            }
            *at = x;
          }
      }
      ptx::named_sync(1, NW * 32);
    }
    // ---- write: thread -> 4 consecutive values of a row
    const bool whole = s.t0 == 0 && s.t1 == s.r.tiles;
    const int64_t slot = 2 * int64_t(blockIdx.x) + (s.t0 == 0 ? 1 : 0);
    const bool any_bad = *reinterpret_cast<volatile int*>(&s_any_bad) != 0;
    for (int i = tid; i < rows * (D / 4); i += NW * 32) {
      const int r = i / (D / 4), d = (i % (D / 4)) * 4;
      float4 x = *reinterpret_cast<const float4*>(merge + r * D + d);
      const int token = (r0 + r) / a.group, head = s.h * a.group + (r0 + r) % a.group;
      if (any_bad) {
        const uint64_t* mr = a.mask != nullptr ? a.mask + (s.r.row0 + int64_t(token)) * a.mask_words : nullptr;
        for (int j = 0; j < min(s.r.n, 256); ++j) {
          if (!((s_bad[j >> 5] >> (j & 31)) & 1) || !sees(a, mr, token, j, s.r.n)) continue;
          const int64_t pos = int64_t(s.r.ctx) + j;
          const int pg = a.table[int64_t(s.b) * a.table_stride + (pos >> a.page_shift)];
          if (pg < 0 || pg >= a.pages) continue;
          const uint16_t* v = a.v + int64_t(pg) * a.page_stride +
                              (pos & ((1 << a.page_shift) - 1)) * a.token_stride +
                              int64_t(s.h) * a.head_stride + d;
          float* xf = reinterpret_cast<float*>(&x);
          for (int e = 0; e < 4; ++e)
            if (nonfinite2<BF16>(v[e]) & 1) xf[e] += widen<BF16>(v[e]);
        }
      }
      float mm = -INFINITY, ll = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) mm = fmaxf(mm, s_ml[w][r].x);
#pragma unroll
      for (int w = 0; w < NW; ++w)
        ll += s_ml[w][r].y * (mm == -INFINITY ? 0.f : ex2(s_ml[w][r].x - mm));
      if (whole) {
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        const int64_t at = (int64_t(s.r.row0) + token) * a.Hq + head;
        *reinterpret_cast<uint2*>(a.out + at * D + d) =
            make_uint2(pack2<BF16>(x.x * inv, x.y * inv), pack2<BF16>(x.z * inv, x.w * inv));
        if (d == 0 && a.lse != nullptr)
          a.lse[at] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
      } else {
        *reinterpret_cast<float4*>(a.part_o + (slot * RT + r) * D + d) = x;
        if (d == 0) a.part_ml[slot * RT + r] = make_float2(mm, ll);
      }
    }
    if (!whole && s.t0 == 0 && tid == 0) {
      Join* j = a.join + blockIdx.x;
      j->row0 = s.r.row0;
      j->r0 = r0;
      j->rows = rows;
      j->head = s.h;
      j->follow = cta_of(piece, s.end - 1) - static_cast<int>(blockIdx.x);
    }
    ptx::named_sync(1, NW * 32);   // s_ml, merge and s_bad are free again
    if (any_bad) {
      if (tid < 8) s_bad[tid] = 0;
      if (tid == 0) s_any_bad = 0;
      ptx::named_sync(1, NW * 32);
    }
  }
}

// ------------------------------------------------------------------ join
//
// One warp a row: its pieces' (m, l) give the factors, then the pieces'
// outputs are added in the order of the keys.
constexpr int JOIN_WARPS = 4;

template <bool BF16, int D>
__global__ void __launch_bounds__(JOIN_WARPS * 32) combine_kernel(const Args a, int rt) {
  pdl_wait();
  pdl_launch_dependents();
  const Join j = a.join[blockIdx.x];
  const int r = blockIdx.y * JOIN_WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (j.follow == 0 || r >= j.rows) return;
  const int64_t c = blockIdx.x;
  // piece i: slot 1 of CTA c, then slot 0 of CTA c + i
  const auto slot_of = [&](int i) { return 2 * (c + i) + (i == 0 ? 1 : 0); };
  float mm = -INFINITY;
  for (int i = lane; i <= j.follow; i += 32) mm = fmaxf(mm, a.part_ml[slot_of(i) * rt + r].x);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mm = fmaxf(mm, __shfl_xor_sync(~0u, mm, d));
  constexpr int V = D / 32;
  float x[V] = {};
  float ll = 0.f;
#pragma unroll 4
  for (int i = 0; i <= j.follow; ++i) {
    const int64_t at = slot_of(i) * rt + r;
    const float2 ml = a.part_ml[at];
    const float f = mm == -INFINITY ? 0.f : ex2(ml.x - mm);
    ll += ml.y * f;
    const float* o = a.part_o + at * D + lane * V;
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      const float2 v = *reinterpret_cast<const float2*>(o + e);
      x[e] += v.x * f;
      x[e + 1] += v.y * f;
    }
  }
  const float inv = ll == 0.f ? 0.f : 1.f / ll;
  const int token = (j.r0 + r) / a.group, head = j.head * a.group + (j.r0 + r) % a.group;
  const int64_t at = (int64_t(j.row0) + token) * a.Hq + head;
#pragma unroll
  for (int e = 0; e < V; e += 2)
    *reinterpret_cast<uint32_t*>(a.out + at * D + lane * V + e) =
        pack2<BF16>(x[e] * inv, x[e + 1] * inv);
  if (lane == 0 && a.lse != nullptr)
    a.lse[at] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
}

// ------------------------------------------------------------------ host

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static std::atomic<EncodeTiledFn> fn{nullptr};
  EncodeTiledFn f = fn.load(std::memory_order_acquire);
  if (f == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
      f = reinterpret_cast<EncodeTiledFn>(p);
      fn.store(f, std::memory_order_release);
    }
  }
  return f;
}

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

struct Ws {
  size_t o, ml, join, bytes;
};
Ws ws_layout(int64_t grid, int64_t rt, int64_t D) {
  Ws w;
  w.o = 0;
  w.ml = w.o + static_cast<size_t>(2 * grid * rt * D) * sizeof(float);
  w.join = w.ml + static_cast<size_t>(2 * grid * rt) * sizeof(float2);
  w.bytes = w.join + static_cast<size_t>(grid) * sizeof(Join);
  return w;
}

int rows_grid(int64_t D) { return kv_sm_count() * (D == 256 ? 1 : 2); }

template <bool BF16, int D>
cudaError_t launch_rows(const TreeAttnCall& call, Args a, cudaStream_t st) {
  using C = Rows<D>;
  static std::atomic<unsigned long long> attr_done{0};
  cudaError_t e = once_per_device(attr_done, [] {
    return cudaFuncSetAttribute(attn_rows_kernel<BF16, D>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(C::SMEM));
  });
  if (e != cudaSuccess) return e;
  const int box = static_cast<int>(std::min<int64_t>(call.cache.page_size, TK));
  CUtensorMap tk, tv;
  if (!make_map(&tk, call.cache, call.cache.k, box) || !make_map(&tv, call.cache, call.cache.v, box))
    return cudaErrorInvalidValue;
  const int grid = rows_grid(D);
  const Ws w = ws_layout(grid, RT, D);
  uint8_t* ws = static_cast<uint8_t*>(call.ws);
  a.part_o = reinterpret_cast<float*>(ws + w.o);
  a.part_ml = reinterpret_cast<float2*>(ws + w.ml);
  a.join = reinterpret_cast<Join*>(ws + w.join);
  e = launch(attn_rows_kernel<BF16, D>, dim3(grid), dim3(THREADS), C::SMEM, st, tk, tv, a);
  if (e != cudaSuccess) return e;
  return launch(combine_kernel<BF16, D>, dim3(grid, RT / JOIN_WARPS), dim3(JOIN_WARPS * 32), 0, st,
                a, RT);
}

}  // namespace

size_t tree_attention_workspace_bytes(int64_t, int64_t, int64_t, int64_t D) {
  return ws_layout(rows_grid(D), RT, D).bytes;
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
  a.scale_log2 = call.scale * 1.4426950408889634f;
  const bool bf = c.dtype == TERN_KV_BF16;
  if (c.dim == 64) return bf ? launch_rows<true, 64>(call, a, st) : launch_rows<false, 64>(call, a, st);
  if (c.dim == 128)
    return bf ? launch_rows<true, 128>(call, a, st) : launch_rows<false, 128>(call, a, st);
  return bf ? launch_rows<true, 256>(call, a, st) : launch_rows<false, 256>(call, a, st);
}

cudaError_t attn_read_clear_error(unsigned int* err) {
  cudaError_t e = cudaMemcpyFromSymbol(err, g_attn_error, sizeof(unsigned int));
  if (e != cudaSuccess || *err == 0) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_attn_error, &zero, sizeof(unsigned int));
}

}  // namespace tern
