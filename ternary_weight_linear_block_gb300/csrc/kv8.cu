// Rows on their way into a cache (tern_kv_rotate_write): norms of queries and
// keys for each head, rotary positions, and the keys and values written as
// 16-bit values or quantised to 8 bits; and the 8-bit cache's rows read back
// (tern_kv8_read) and moved (tern_kv8_commit).
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kv_internal.cuh"
#include "tern_internal.cuh"

namespace tern {
namespace {

enum Kind { SAME = 0, I8 = 1, E4M3 = 2 };

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack16<BF16>(x[0], x[1]), pack16<BF16>(x[2], x[3]), pack16<BF16>(x[4], x[5]),
                    pack16<BF16>(x[6], x[7]));
}

// ------------------------------------------------------------------ rotate and write
//
// A lane has two chunks of 8 elements of a head (16 bytes each), D / 16 lanes a
// head, so a warp takes 32 / (D / 16) heads at a time.  The chunks are those whose
// elements turn together, so a rotation needs no other lane; where rows are only
// quantised they are neighbours, so their codes are stored as one.  A lane's
// places in the head, and with them the cosines and sines of a token, stay the
// same for all of a token's heads.  A unit is UNROLL such steps of one token and
// of one kind (queries, keys or values), whose loads are on their way together; a
// warp takes a.per units in a row.
//
// One read and one write of everything, so memory bounds it; with a rotation and a
// norm the instructions of both beside it.  Measured: 185 us for the rows of 16-bit
// keys and values that would take 172 at the copy rate (0.93), 263 for rotated and
// normalised queries and keys that would take 191 (0.73); 206 and 321 with one
// chunk a lane, twice the lanes in a sum and partners from other lanes.  CTAs of 128
// threads an SM (turning, writing): 5, 9; 6, 11: 265, 184; 7, 12: 268, 184; CTAs of
// 256 and steps: 3, 5 and 2: 271 (spills), 184; 4, 6 and 1: 300, 191; 2, 4 and 2: 299,
// 192; 2, 4 and 3: 286, 194; 2, 3 and 4: 281, 209.  A call of few rows is a launch
// and two dependent reads, 4 us.
//
// The angle of pair j is position * turns[j] in 64-bit integers, turns of 2^-64:
// the product wraps where the angle does, so that its top 32 bits are the angle
// at any position, to 2^-32 of a turn; as a float, which has 24 bits, to 2^-26.
//
// Bound: rows read once and written once.

constexpr int ROT_THREADS = 128;
constexpr int UNROLL = 2;
constexpr float kSmallest = 0x1p-100f;   // rows below are stored as zeros

struct RotArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* q_out;
  uint8_t* ck;
  uint8_t* cv;
  float* ks;
  float* vs;
  const int64_t* slots;
  const int32_t* positions;
  const uint64_t* turns;
  const int32_t* axis;
  const void* q_norm;
  const void* k_norm;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head;
  int64_t position_stride;
  int64_t page_stride, token_stride, head_stride;     // elements of the cache
  int64_t scale_page, scale_head;
  int64_t T, n_slots, units;
  int Hq, H, uq, uk;                                  // units of a token's queries, and keys
  int per, page_shift, rot, axes;
  int neighbours, norm_f32;
  float eps;
};

// The largest magnitude of a lane's 8 elements, as bits of a float: of 32-bit
// values, and of 16-bit ones as they were read (their bits compare likewise).
__device__ __forceinline__ uint32_t top_of(const float (&x)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  return top;
}
template <bool BF16>
__device__ __forceinline__ uint32_t top_of(const uint4& w) {
  const uint32_t m = 0x7FFF7FFFu;
  const uint32_t top = __vmaxu2(__vmaxu2(w.x & m, w.y & m), __vmaxu2(w.z & m, w.w & m));
  const uint16_t one = static_cast<uint16_t>(max(top & 0xFFFFu, top >> 16));
  if constexpr (BF16) return static_cast<uint32_t>(one) << 16;
  else return __float_as_uint(__half2float(*reinterpret_cast<const __half*>(&one)));
}

template <int LPH>
__device__ __forceinline__ float sum_over(float x) {
#pragma unroll
  for (int d = LPH / 2; d > 0; d >>= 1) x += __shfl_xor_sync(~0u, x, d);
  return x;
}

// A row's unit and what its elements are multiplied by, from a lane's largest
// magnitude.  The magnitudes' bits compare as the magnitudes do, infinities and
// NaN above all others.  0: the row is stored as zeros.
template <int KIND, int LPH>
__device__ __forceinline__ float unit_of(uint32_t top, float& unit) {
#pragma unroll
  for (int d = LPH / 2; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(~0u, top, d));
  const float most = __uint_as_float(top);
  constexpr float kLargest = KIND == I8 ? 127.f : 448.f;
  const bool whole = top < 0x7F800000u, some = whole && most >= kSmallest;
  unit = some ? __fdiv_rn(most, kLargest) : whole ? 0.f : __uint_as_float(0x7FC00000u);
  return some ? __fdiv_rn(kLargest, most) : 0.f;
}
// The codes of 8 elements.
template <int KIND>
__device__ __forceinline__ uint2 codes_of(const float (&x)[8], float f) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float* y = x + 4 * h;
    if constexpr (KIND == I8) {
      // rounded to a whole number in the last bits of the sum with 3 2^22
      uint32_t c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = __float_as_uint(__fadd_rn(__fmul_rn(y[i], f), 12582912.f));
      w[h] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    } else {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(y[0], f), __fmul_rn(y[1], f)),
                                                   __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(y[2], f), __fmul_rn(y[3], f)),
                                                   __NV_SATFINITE, __NV_E4M3);
      w[h] = lo | hi << 16;
    }
  }
  return f > 0.f ? make_uint2(w[0], w[1]) : make_uint2(0, 0);
}

__device__ __forceinline__ void turn_neighbours(float (&x)[8], const float* cs, const float* sn) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float b = x[2 * j];
    x[2 * j] = b * cs[j] - x[2 * j + 1] * sn[j];
    x[2 * j + 1] = x[2 * j + 1] * cs[j] + b * sn[j];
  }
}

// TURN: queries, norms or a rotation; without them the rows are only written.
template <bool BF16, int D, int KIND, bool TURN>
__global__ void __launch_bounds__(ROT_THREADS, (TURN ? 5 : 9)) rotate_kernel(const __grid_constant__ RotArgs a) {
  constexpr int LPH = D / 16, HPW = 32 / LPH;
  const int lane = threadIdx.x & 31;
  const int sub = lane % LPH, part = lane / LPH;
  // a lane's two chunks of 8 elements
  const int pairs = TURN && !a.neighbours ? a.rot / 16 : 0;     // lanes whose chunks turn together
  const bool together = sub < pairs;
  int c0 = sub, c1 = sub + LPH;
  if (!TURN && KIND != SAME) {
    c0 = 2 * sub;
    c1 = c0 + 1;
  } else if (together) {
    c1 = sub + pairs;
  } else {
    c0 = sub + pairs;
    c1 = c0 + LPH - pairs;
  }
  const int e0 = c0 * 8, e1 = c1 * 8;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t w = (int64_t(blockIdx.x) * ROT_THREADS + threadIdx.x) >> 5;
  const int64_t first = w * a.per;
  if (first >= a.units) return;
  const int n = static_cast<int>(min(int64_t(a.per), a.units - first));
  const int upt = a.uq + 2 * a.uk;
  int64_t t = first / upt;
  int i = static_cast<int>(first - t * upt);
  float cs[8], sn[8];         // of `together`: of both chunks; of neighbours: four pairs of each
  int64_t at = -1;            // the token that cs, sn and to are of
  int64_t to = 0, to_scale = 0;
  bool known = false;
  float wt[16];
  int wt_of = -1;             // whose norm wt has

#pragma unroll 1
  for (int u = 0; u < n; ++u) {
    const int kind = TURN && i < a.uq ? 0 : i < a.uq + a.uk ? 1 : 2;      // queries, keys, values
    const int h0 = (kind == 0 ? i : kind == 1 ? i - a.uq : i - a.uq - a.uk) * (UNROLL * HPW);
    const int heads = kind == 0 ? a.Hq : a.H;
    const uint16_t* src = kind == 0 ? a.q + t * a.q_token : kind == 1 ? a.k + t * a.k_token
                                                                     : a.v + t * a.v_token;
    const int64_t head = kind == 0 ? a.q_head : kind == 1 ? a.k_head : a.v_head;
    uint4 in[UNROLL][2];
#pragma unroll
    for (int s = 0; s < UNROLL; ++s) {
      const int h = h0 + s * HPW + part;
      if (h < heads) {
        in[s][0] = *reinterpret_cast<const uint4*>(src + h * head + e0);
        in[s][1] = *reinterpret_cast<const uint4*>(src + h * head + e1);
      } else {
        in[s][0] = in[s][1] = make_uint4(0, 0, 0, 0);
      }
    }
    if (t != at) {
      at = t;
      const int64_t slot = a.slots[t];
      known = slot >= 0 && slot < a.n_slots;
      const int64_t page = known ? slot >> a.page_shift : 0;
      const int64_t row = known ? slot & ((int64_t(1) << a.page_shift) - 1) : 0;
      to = page * a.page_stride + row * a.token_stride;
      to_scale = page * a.scale_page + row;
      if (TURN && kind != 2 && (together || a.neighbours)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int f = a.neighbours ? (j < 4 ? e0 / 2 + j : e1 / 2 + j - 4) : e0 + j;
          if (2 * f >= a.rot) continue;
          int ax = a.axis != nullptr ? __ldg(a.axis + f) : 0;
          if (ax < 0 || ax >= a.axes) ax = 0;
          const int32_t p = __ldg(a.positions + ax * a.position_stride + t);
          const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(p)) * __ldg(a.turns + f);
          // halves of a turn, -1 to 1
          const float x = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
          sincospif(x, &sn[j], &cs[j]);
        }
      }
    }
    const void* norm = !TURN || kind == 2 ? nullptr : kind == 0 ? a.q_norm : a.k_norm;
    if (norm != nullptr && wt_of != kind) {
      wt_of = kind;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int e = c == 0 ? e0 : e1;
        float (&y)[8] = *reinterpret_cast<float (*)[8]>(wt + 8 * c);
        if (a.norm_f32) {
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = __ldg(static_cast<const float*>(norm) + e + j);
        } else {
          unpack8<BF16>(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(norm) + e)), y);
        }
      }
    }
#pragma unroll
    for (int s = 0; s < UNROLL; ++s) {
      const int h = h0 + s * HPW + part;
      if (h0 + s * HPW >= heads) break;                     // the same for the whole warp
      if (KIND == SAME && kind == 2) {
        if (known && h < heads) {
          uint16_t* row = reinterpret_cast<uint16_t*>(a.cv) + to + h * a.head_stride;
          *reinterpret_cast<uint4*>(row + e0) = in[s][0];
          *reinterpret_cast<uint4*>(row + e1) = in[s][1];
        }
        continue;
      }
      float x[8], y[8];
      unpack8<BF16>(in[s][0], x);
      unpack8<BF16>(in[s][1], y);
      if (norm != nullptr) {
        float sq = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) sq = fmaf(y[j], y[j], fmaf(x[j], x[j], sq));
        sq = sum_over<LPH>(sq);
        const float r = rsqrtf(sq * (1.f / D) + a.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[j] = x[j] * r * wt[j];
          y[j] = y[j] * r * wt[8 + j];
        }
      }
      if (TURN && kind != 2) {
        if (together) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float b = x[j];
            x[j] = b * cs[j] - y[j] * sn[j];
            y[j] = y[j] * cs[j] + b * sn[j];
          }
        } else if (a.neighbours) {
          if (e0 < a.rot) turn_neighbours(x, cs, sn);
          if (e1 < a.rot) turn_neighbours(y, cs + 4, sn + 4);
        }
      }
      if (kind == 0) {
        if (h < heads) {
          uint16_t* row = a.q_out + (t * a.Hq + h) * D;
          *reinterpret_cast<uint4*>(row + e0) = pack8<BF16>(x);
          *reinterpret_cast<uint4*>(row + e1) = pack8<BF16>(y);
        }
      } else if constexpr (KIND == SAME) {
        if (known && h < heads) {
          uint16_t* row = reinterpret_cast<uint16_t*>(a.ck) + to + h * a.head_stride;
          *reinterpret_cast<uint4*>(row + e0) = pack8<BF16>(x);
          *reinterpret_cast<uint4*>(row + e1) = pack8<BF16>(y);
        }
      } else {
        float unit;
        const uint32_t top = TURN && kind == 1 ? max(top_of(x), top_of(y))
                                               : max(top_of<BF16>(in[s][0]), top_of<BF16>(in[s][1]));
        const float f = unit_of<KIND, LPH>(top, unit);
        const uint2 lo = codes_of<KIND>(x, f), hi = codes_of<KIND>(y, f);
        if (known && h < heads) {
          uint8_t* row = (kind == 1 ? a.ck : a.cv) + to + h * a.head_stride;
          if constexpr (!TURN) {
            *reinterpret_cast<uint4*>(row + e0) = make_uint4(lo.x, lo.y, hi.x, hi.y);
          } else {
            *reinterpret_cast<uint2*>(row + e0) = lo;
            *reinterpret_cast<uint2*>(row + e1) = hi;
          }
          if (sub == 0) (kind == 1 ? a.ks : a.vs)[to_scale + h * a.scale_head] = unit;
        }
      }
    }
    if (++i == upt) {
      i = 0;
      ++t;
    }
  }
}

// ------------------------------------------------------------------ read
//
// A thread turns 16 codes into 32 bytes.  Bound: codes read, values written.

constexpr int READ_THREADS = 256;

struct ReadArgs {
  const uint8_t* ck;
  const uint8_t* cv;
  const float* ks;
  const float* vs;
  uint16_t* k;
  uint16_t* v;
  const int64_t* slots;
  int64_t page_stride, token_stride, head_stride, scale_page, scale_head;
  int64_t T, n_slots;
  int H, chunks;                    // 16-code chunks of a token
  int dim_shift, page_shift;        // log2 of the chunks of a head
};

template <int KIND>
__device__ __forceinline__ void widen4(uint32_t w, float (&x)[4]) {
  if constexpr (KIND == I8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * i)), __NV_E4M3);
      const float2 f = __half22float2(__half2(h));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

// code * unit, rounded once.  Memory bounds it: half of the bytes that it writes
// are read, 16 of codes a thread, for which one unit is enough.
template <bool BF16, int KIND>
__global__ void __launch_bounds__(READ_THREADS) read_kernel(const __grid_constant__ ReadArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t total = 2 * a.T * a.chunks;
  const int64_t step = int64_t(gridDim.x) * READ_THREADS;
  for (int64_t p = int64_t(blockIdx.x) * READ_THREADS + threadIdx.x; p < total; p += step) {
    // a token's keys, then its values
    const int64_t t = p / (2 * a.chunks);
    int c = static_cast<int>(p - t * (2 * a.chunks));
    const bool vals = c >= a.chunks;
    if (vals) c -= a.chunks;
    const int64_t slot = a.slots[t];
    uint4 out[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (slot >= 0 && slot < a.n_slots) {
      const int64_t page = slot >> a.page_shift, row = slot & ((int64_t(1) << a.page_shift) - 1);
      const int64_t h = c >> a.dim_shift;
      const int d = (c & ((1 << a.dim_shift) - 1)) * 16;
      const uint4 w = *reinterpret_cast<const uint4*>((vals ? a.cv : a.ck) + page * a.page_stride +
                                                      row * a.token_stride + h * a.head_stride + d);
      const float unit = (vals ? a.vs : a.ks)[page * a.scale_page + h * a.scale_head + row];
      const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x[4];
        widen4<KIND>(ws[i], x);
        o[2 * i] = pack16<BF16>(x[0] * unit, x[1] * unit);
        o[2 * i + 1] = pack16<BF16>(x[2] * unit, x[3] * unit);
      }
      out[0] = make_uint4(o[0], o[1], o[2], o[3]);
      out[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
    uint4* to = reinterpret_cast<uint4*>((vals ? a.v : a.k) + (t * a.chunks + c) * 16);
    to[0] = out[0];
    to[1] = out[1];
  }
}

// ------------------------------------------------------------------ commit
//
// As for 16-bit caches: a thread owns one column of a request's rows (16
// codes, or one head's unit) and moves it for the whole path, which increases,
// so that a row is written only after it was read.

constexpr int MAX_PATH = 256;
constexpr int MOVE_THREADS = 256;
constexpr int MOVE_LAYERS = 32;   // layers of one launch: their pointers are kernel arguments

struct MoveArgs {
  uint8_t* code[2 * MOVE_LAYERS];     // keys, values of each layer
  float* scale[2 * MOVE_LAYERS];
  const int32_t* table;
  const int32_t* ctx_len;
  const int32_t* path;
  const int32_t* path_len;
  int32_t* ctx_out;
  int64_t table_stride, path_stride;
  int64_t page_stride, token_stride, head_stride, scale_page, scale_head, pages;
  int width, path_width, chunks, heads, dim_shift, page_shift;
};

template <class V>
__device__ __forceinline__ void move_column(V* x, const int64_t* from, const int64_t* to, int count) {
  constexpr int U = 4;
  for (int j0 = 0; j0 < count; j0 += U) {
    V r[U];
    bool move[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      move[i] = j0 + i < count && from[j0 + i] != to[j0 + i];
      if (move[i]) r[i] = *reinterpret_cast<const V*>(reinterpret_cast<const uint8_t*>(x) + from[j0 + i]);
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (move[i]) *reinterpret_cast<V*>(reinterpret_cast<uint8_t*>(x) + to[j0 + i]) = r[i];
  }
}

// The path moves towards the start of its tokens, so a thread that has a column of
// bytes of every row may move them in the path's order, four reads ahead of
// their writes; no thread needs another's.  Three dependent reads (path, table,
// row) are its time for one step.
__global__ void __launch_bounds__(MOVE_THREADS) move_kernel(const __grid_constant__ MoveArgs a) {
  // byte offsets of the path's rows: of codes, and of units
  __shared__ int64_t s_from[2][MAX_PATH], s_to[2][MAX_PATH];
  __shared__ int s_count;
  const int b = blockIdx.y, tid = threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const int ctx = a.ctx_len[b];
  const int len = ctx < 0 ? 0 : min(max(a.path_len[b], 0), a.path_width);
  if (tid == 0) s_count = len;
  __syncthreads();
  const int64_t mask = (int64_t(1) << a.page_shift) - 1;
  const auto page_of = [&](int64_t p) -> int64_t {
    const int64_t at = p >> a.page_shift;
    if (at >= a.width) return -1;
    const int64_t page = a.table[b * a.table_stride + at];
    return page < 0 || page >= a.pages ? -1 : page;
  };
  for (int j = tid; j < len; j += MOVE_THREADS) {
    const int p = a.path[b * a.path_stride + j];
    const int prev = j > 0 ? a.path[b * a.path_stride + j - 1] : -1;
    const int64_t fp = int64_t(ctx) + p, tp = int64_t(ctx) + j;
    int64_t from = -1, to = -1;
    if (p >= 0 && p > prev) {
      from = page_of(fp);
      to = page_of(tp);
    }
    if (from < 0 || to < 0) {
      atomicMin(&s_count, j);
      from = to = 0;
    }
    s_from[0][j] = from * a.page_stride + (fp & mask) * a.token_stride;
    s_to[0][j] = to * a.page_stride + (tp & mask) * a.token_stride;
    s_from[1][j] = (from * a.scale_page + (fp & mask)) * 4;
    s_to[1][j] = (to * a.scale_page + (tp & mask)) * 4;
  }
  __syncthreads();
  const int count = s_count;
  if (blockIdx.x == 0 && blockIdx.z == 0 && tid == 0 && a.ctx_out != nullptr) a.ctx_out[b] = ctx + count;
  int c = blockIdx.x * MOVE_THREADS + tid;
  if (c < a.chunks) {
    const int64_t col = int64_t(c >> a.dim_shift) * a.head_stride + (c & ((1 << a.dim_shift) - 1)) * 16;
    move_column(reinterpret_cast<uint4*>(a.code[blockIdx.z] + col), s_from[0], s_to[0], count);
  } else if (c - a.chunks < a.heads) {
    c -= a.chunks;
    move_column(a.scale[blockIdx.z] + c * a.scale_head, s_from[1], s_to[1], count);
  }
}

int log2_of(int64_t v) {
  int s = 0;
  while ((int64_t(1) << s) < v) ++s;
  return s;
}

template <bool BF16, int D>
cudaError_t launch_rotate_dim(int kind, const RotArgs& a, unsigned blocks, cudaStream_t st) {
  const dim3 g(blocks), b(ROT_THREADS);
  const bool turn = a.Hq > 0 || a.rot > 0 || a.k_norm != nullptr;
  if (kind == SAME) return launch(rotate_kernel<BF16, D, SAME, true>, g, b, 0, st, a);
  if (kind == I8)
    return turn ? launch(rotate_kernel<BF16, D, I8, true>, g, b, 0, st, a)
                : launch(rotate_kernel<BF16, D, I8, false>, g, b, 0, st, a);
  return turn ? launch(rotate_kernel<BF16, D, E4M3, true>, g, b, 0, st, a)
              : launch(rotate_kernel<BF16, D, E4M3, false>, g, b, 0, st, a);
}

template <bool BF16>
cudaError_t launch_rotate_type(int kind, int64_t dim, const RotArgs& a, unsigned blocks, cudaStream_t st) {
  if (dim == 64) return launch_rotate_dim<BF16, 64>(kind, a, blocks, st);
  if (dim == 128) return launch_rotate_dim<BF16, 128>(kind, a, blocks, st);
  return launch_rotate_dim<BF16, 256>(kind, a, blocks, st);
}

}  // namespace

cudaError_t launch_kv_rotate_write(const tern_kv_cache* c, const tern_kv_cache8* c8,
                                   const tern_kv_rows& r, cudaStream_t st) {
  RotArgs a{};
  a.q = static_cast<const uint16_t*>(r.q);
  a.k = static_cast<const uint16_t*>(r.k);
  a.v = static_cast<const uint16_t*>(r.v);
  a.q_out = static_cast<uint16_t*>(r.q_out);
  a.slots = r.slots;
  a.positions = r.positions;
  a.turns = r.turns;
  a.axis = r.axis;
  a.q_norm = r.q_norm;
  a.k_norm = r.k_norm;
  a.q_token = r.q_token_stride;
  a.q_head = r.q_head_stride;
  a.k_token = r.k_token_stride;
  a.k_head = r.k_head_stride;
  a.v_token = r.v_token_stride;
  a.v_head = r.v_head_stride;
  a.position_stride = r.position_stride;
  a.T = r.T;
  a.Hq = static_cast<int>(r.Hq);
  a.rot = static_cast<int>(r.rot);
  a.axes = static_cast<int>(r.axes);
  a.neighbours = r.neighbours;
  a.norm_f32 = r.norm_f32;
  a.eps = r.eps;
  int64_t dim, page_size, pages;
  int kind = SAME;
  if (c != nullptr) {
    a.ck = static_cast<uint8_t*>(c->k);
    a.cv = static_cast<uint8_t*>(c->v);
    a.H = static_cast<int>(c->heads);
    a.page_stride = c->page_stride;
    a.token_stride = c->token_stride;
    a.head_stride = c->head_stride;
    dim = c->dim, page_size = c->page_size, pages = c->pages;
  } else {
    kind = c8->dtype == TERN_KV_I8 ? I8 : E4M3;
    a.ck = static_cast<uint8_t*>(c8->k);
    a.cv = static_cast<uint8_t*>(c8->v);
    a.ks = c8->k_scale;
    a.vs = c8->v_scale;
    a.H = static_cast<int>(c8->heads);
    a.page_stride = c8->page_stride;
    a.token_stride = c8->token_stride;
    a.head_stride = c8->head_stride;
    a.scale_page = c8->scale_page_stride;
    a.scale_head = c8->scale_head_stride;
    dim = c8->dim, page_size = c8->page_size, pages = c8->pages;
  }
  a.page_shift = log2_of(page_size);
  a.n_slots = pages * page_size;
  const int step = static_cast<int>(UNROLL * 512 / dim);        // heads of a unit
  a.uq = (a.Hq + step - 1) / step;
  a.uk = (a.H + step - 1) / step;
  const int upt = a.uq + 2 * a.uk;
  a.units = a.T * upt;
  // a token's units share its cosines and sines; few tokens spread over all SMs
  const int64_t room = int64_t(kv_sm_count()) * 32;
  a.per = static_cast<int>(std::min<int64_t>(upt, std::max<int64_t>(1, a.units / room)));
  const int64_t warps = (a.units + a.per - 1) / a.per;
  const unsigned blocks = static_cast<unsigned>((warps + ROT_THREADS / 32 - 1) / (ROT_THREADS / 32));
  return r.dtype == TERN_KV_BF16 ? launch_rotate_type<true>(kind, dim, a, blocks, st)
                                 : launch_rotate_type<false>(kind, dim, a, blocks, st);
}

cudaError_t launch_kv8_read(const tern_kv_cache8& c, const int64_t* slots, int64_t T, void* k, void* v,
                            int dtype, cudaStream_t st) {
  ReadArgs a{static_cast<const uint8_t*>(c.k), static_cast<const uint8_t*>(c.v), c.k_scale, c.v_scale,
             static_cast<uint16_t*>(k), static_cast<uint16_t*>(v), slots, c.page_stride, c.token_stride,
             c.head_stride, c.scale_page_stride, c.scale_head_stride, T, c.pages * c.page_size,
             static_cast<int>(c.heads), static_cast<int>(c.heads * c.dim / 16), log2_of(c.dim / 16),
             log2_of(c.page_size)};
  const int64_t total = 2 * T * a.chunks;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>((total + READ_THREADS - 1) / READ_THREADS,
                                                          int64_t(kv_sm_count()) * 64)));
  const dim3 block(READ_THREADS);
  const bool bf = dtype == TERN_KV_BF16;
  if (c.dtype == TERN_KV_I8)
    return bf ? launch(read_kernel<true, I8>, grid, block, 0, st, a)
              : launch(read_kernel<false, I8>, grid, block, 0, st, a);
  return bf ? launch(read_kernel<true, E4M3>, grid, block, 0, st, a)
            : launch(read_kernel<false, E4M3>, grid, block, 0, st, a);
}

cudaError_t launch_kv8_commit(const tern_kv_cache8* caches, int64_t layers, const int32_t* table,
                              int64_t table_stride, int64_t table_width, const int32_t* ctx_len,
                              const int32_t* path, int64_t path_width, const int32_t* path_len,
                              int32_t* ctx_out, int64_t B, cudaStream_t st) {
  const tern_kv_cache8& c = caches[0];
  const int chunks = static_cast<int>(c.heads * c.dim / 16);
  for (int64_t l0 = 0; l0 < layers; l0 += MOVE_LAYERS) {
    const int n = static_cast<int>(std::min<int64_t>(layers - l0, MOVE_LAYERS));
    MoveArgs a{};
    for (int l = 0; l < n; ++l) {
      const tern_kv_cache8& x = caches[l0 + l];
      a.code[2 * l] = static_cast<uint8_t*>(x.k);
      a.code[2 * l + 1] = static_cast<uint8_t*>(x.v);
      a.scale[2 * l] = x.k_scale;
      a.scale[2 * l + 1] = x.v_scale;
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
    a.scale_page = c.scale_page_stride;
    a.scale_head = c.scale_head_stride;
    a.pages = c.pages;
    a.width = static_cast<int>(table_width);
    a.path_width = static_cast<int>(path_width);
    a.chunks = chunks;
    a.heads = static_cast<int>(c.heads);
    a.dim_shift = log2_of(c.dim / 16);
    a.page_shift = log2_of(c.page_size);
    const dim3 grid(static_cast<unsigned>((chunks + a.heads + MOVE_THREADS - 1) / MOVE_THREADS),
                    static_cast<unsigned>(B), static_cast<unsigned>(2 * n));
    const cudaError_t e = launch(move_kernel, grid, dim3(MOVE_THREADS), 0, st, a);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace tern
