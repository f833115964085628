// Tokens from logits (tern_sample), and the path of a tree of drafts that
// agrees with them (tern_tree_accept).
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv_internal.cuh"
#include "sm100_ptx.cuh"
#include "tern_internal.cuh"

namespace tern {
namespace {

// ------------------------------------------------------------------ sample
//
// The filters keep a prefix of the tokens in the order of their logits (of
// equal ones the lower index first), so all that has to be found is its last
// logit and how many of that logit's tokens are in.  A cluster of CTAs has a
// row, each a stretch of its indices.
//
//  1. The largest logit, and of every thread's elements the largest.
//  2. Few survivors: a bound that at least `aim` of the threads' largest
//     reach, so that about as many tokens do, is found from a histogram of
//     these alone.  The tokens from it on are gathered in the first CTA, sorted,
//     and their weights summed in that order: top-k and top-p fall out where
//     the prefix ends inside the list.  The kept tokens are sorted by index
//     and the drawn one is found in their running sum.
//  3. Otherwise the border is searched by histograms of counts and weights
//     (narrow), in steps of the logit and then of its bits until a single
//     logit is left; of bf16 logits, which have few values, by one histogram of
//     counts (Places).  The draw is a pass over the row: every warp sums the kept
//     weights of its own stretch, and the one where the sum passes u times the
//     whole looks for the token.
//
// Weights are whole numbers of 2^-45 of the largest, so sums are exact and in
// any order the same.
//
// A row is read two (few survivors) to five times, from L2 after the first, and every
// step that a cluster takes together costs it a few us; the vocabulary is too
// short for either memory (18 us for 250 rows of 250007 in bf16) or arithmetic to
// bound it.  Those take 128 us with all kinds of filters (689 with the search by
// histograms for all rows, 259 with the list, 207 with places), 97 with top_k
// alone.  fp16 and fp32 have no places, so their search takes three to five passes, and a
// weight about 45 instructions: 257 and 265 with filters of all kinds, 525 and 530 with
// top_p alone.  4 rows of 131072: 15 us, of which the launch of the clusters and 12 joint steps are
// most.

constexpr int NT = 512;              // threads, and places of the list
constexpr int WARPS = NT / 32;
constexpr int BINS = 1024;
constexpr int MAX_CL = 8;
constexpr uint64_t ONE = uint64_t(1) << 45;
constexpr float kReach = 46.f;       // weights below 2^-46 count as none

// 2^(i / 32) in whole numbers of 2^-31.
__constant__ uint32_t kRoots[32] = {
    2147483648u, 2194507417u, 2242560872u, 2291666561u, 2341847524u, 2393127307u, 2445529972u, 2499080105u,
    2553802834u, 2609723834u, 2666869345u, 2725266179u, 2784941738u, 2845924021u, 2908241642u, 2971923842u,
    3037000500u, 3103502151u, 3171459999u, 3240905930u, 3311872529u, 3384393094u, 3458501653u, 3534232978u,
    3611622603u, 3690706840u, 3771522796u, 3854108391u, 3938502376u, 4024744348u, 4112874773u, 4202935003u};

struct SampleArgs {
  const uint8_t* logits;
  const float* u;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int32_t* token;
  int64_t row_stride;      // elements
  int vocab;
};

// What the search for the border has found.
struct Border {
  uint32_t key;            // of the last kept logit
  uint32_t ties;           // its tokens that are kept
  uint64_t above_mass;     // of the tokens above it
  uint32_t above;          // their number
  bool found;              // no: everything from `key` on is kept
};

struct Shared {
  uint32_t count[BINS];
  uint64_t mass[BINS];
  uint64_t list[NT];       // key << 32 | ~index, largest first
  uint64_t sum[NT];
  uint64_t warp_mass[WARPS];
  uint32_t warp_ties[WARPS];
  uint64_t scan[2][WARPS];
  float warp_max[WARPS];
  uint2 table[32];         // 2^(i / 32) as a whole number of 2^-31 and as a float
  float cta_max;
  float c, c_lo;           // log2(e) / temperature
  double span;             // how far below the largest a logit counts
  uint32_t n;              // entries of the list
  int32_t done;            // the list was enough
  // narrow: the interval of keys, what is above it and in all, the goal
  uint32_t lo, hi, above, all, in_bin;
  int32_t found;
  uint64_t above_mass, all_mass, want;
};

// Order-preserving whole number of a float (not NaN).
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);     // one zero
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// floor(f n) for 0 <= f < 1; `more` says that something was cut off.
__device__ __forceinline__ uint64_t part_of(uint64_t n, float f, bool& more) {
  const uint32_t b = __float_as_uint(f);
  const uint32_t e = b >> 23;
  const uint64_t m = (b & 0x7FFFFFu) | (e > 0 ? 0x800000u : 0u);
  const int shift = 150 - static_cast<int>(e > 0 ? e : 1);     // f = m 2^-shift, 24 <= shift <= 149
  const uint64_t lo = n * m, hi = __umul64hi(n, m);
  if (shift >= 128) {
    more = (lo | hi) != 0;
    return 0;
  }
  if (shift >= 64) {
    const int s = shift - 64;
    more = lo != 0 || (hi & ((uint64_t(1) << s) - 1)) != 0;
    return hi >> s;
  }
  more = (lo & ((uint64_t(1) << shift) - 1)) != 0;
  return (lo >> shift) | (hi << (64 - shift));
}
// The least whole number that is not below f n, and at least 1.
__device__ __forceinline__ uint64_t goal_of(uint64_t n, float f) {
  bool more;
  const uint64_t x = part_of(n, f, more);
  return max(x + (more ? 1 : 0), uint64_t(1));
}

// exp((x - most) / temperature) as 2^z, in whole numbers of 2^-45.
//
// z is a product of 32-bit numbers kept as a sum of two, 2^z a power of two
// times 2^(i / 32) from the table times 2^r, |r| < 1/64, by four terms of its
// series: within 2^-29 before the last bit.
struct Weigh {
  float most, c, c_lo;       // log2(e) / temperature in two parts
  const uint2* table;
  __device__ __forceinline__ uint64_t at(float x) const {
    if (x == most) return ONE;
    const float d = x - most;
    const float z = d * c;
    if (!(z > -kReach)) return 0;
    // with what is lost in d: 2^-25 of the largest, of logits of any type that are far
    // smaller, which the temperature turns into 2^-21 of a weight
    const float b = d - x;                // what of -most is in d
    const float lo = fmaf(d, c, -z) + d * c_lo + ((x - (d - b)) - (most + b)) * c;
    const float m = fmaf(z, 32.f, 12582912.f);
    const int j = __float_as_int(m) - 0x4B400000;
    const float r = fmaf(m - 12582912.f, -0.03125f, z) + lo;
    const float q = r * (0.693147181f + r * (0.240226507f + r * (0.0555041087f + r * 0.00961812911f)));
    const uint2 t = table[j & 31];
    const uint32_t w = t.x + static_cast<uint32_t>(__float2int_rn(__uint_as_float(t.y) * q));
    return (static_cast<uint64_t>(w) << 14) >> -(j >> 5);
  }
};

// The same for bf16's middle place, which few logits have: out of line, as the loops
// that may need it are unrolled over a slot's elements (250 x 250007 with all kinds of
// filters 128 us, in line 150).
static __device__ __noinline__ uint64_t weigh_rare(const Weigh& w, float x) { return w.at(x); }

template <int DT>
struct Elt {
  static constexpr int BYTES = DT == TERN_LOGITS_F32 ? 4 : 2;
  static constexpr int E = 16 / BYTES;       // elements of a 16-byte slot
};

// A row in slots of 16 aligned bytes; its first element is element `off` of slot 0.
struct Row {
  const uint8_t* at;
  int off, vocab;
};

// A slot as it is; what is not the row's is -infinity.
template <int DT>
__device__ __forceinline__ uint4 load_slot(const Row& r, int slot) {
  constexpr int E = Elt<DT>::E;
  const int i0 = slot * E - r.off;
  if (i0 >= 0 && i0 + E <= r.vocab)
    return __ldg(reinterpret_cast<const uint4*>(r.at + int64_t(i0) * Elt<DT>::BYTES));
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == TERN_LOGITS_F32) {
      u[i] = i0 + i >= 0 && i0 + i < r.vocab ? __ldg(reinterpret_cast<const uint32_t*>(r.at) + i0 + i) : 0xFF800000u;
    } else {
      u[i] = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = i0 + 2 * i + h;
        const uint32_t w = at >= 0 && at < r.vocab ? __ldg(reinterpret_cast<const uint16_t*>(r.at) + at)
                                                   : DT == TERN_LOGITS_BF16 ? 0xFF80u : 0xFC00u;
        u[i] |= w << (16 * h);
      }
    }
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// f(slot, w) for slots first, first + step, .. below end; four reads are on their
// way together (one at a time kept a pass at 20 bytes a ns and SM, half of what
// memory gives).
template <int DT, class F>
__device__ __forceinline__ void for_slots(const Row& r, int first, int end, int step, const F& f) {
  constexpr int U = 4;
  for (int at = first; at < end; at += U * step) {
    uint4 w[U];
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (at + j * step < end) w[j] = load_slot<DT>(r, at + j * step);
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (at + j * step < end) f(at + j * step, w[j]);
  }
  __syncwarp();
}

// Its elements, NaN as -infinity.
template <int DT>
__device__ __forceinline__ void unpack(const uint4& w, float (&x)[Elt<DT>::E]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == TERN_LOGITS_F32) {
      x[i] = __uint_as_float(u[i]);
    } else if constexpr (DT == TERN_LOGITS_BF16) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
#pragma unroll
  for (int i = 0; i < Elt<DT>::E; ++i) x[i] = fmaxf(x[i], -INFINITY);
}

// The largest of them (16-bit ones compared two at a time); NaN only where all are.
template <int DT>
__device__ __forceinline__ float largest(const uint4& w) {
  if constexpr (DT == TERN_LOGITS_F32) {
    return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
  } else if constexpr (DT == TERN_LOGITS_BF16) {
    const __nv_bfloat162* v = reinterpret_cast<const __nv_bfloat162*>(&w);
    const float2 f = __bfloat1622float2(__hmax2(__hmax2(v[0], v[1]), __hmax2(v[2], v[3])));
    return fmaxf(f.x, f.y);
  } else {
    const __half2* v = reinterpret_cast<const __half2*>(&w);
    const float2 f = __half22float2(__hmax2(__hmax2(v[0], v[1]), __hmax2(v[2], v[3])));
    return fmaxf(f.x, f.y);
  }
}

template <int CL>
__device__ __forceinline__ void sync_all() {
  if constexpr (CL == 1) {
    __syncthreads();
  } else {
    __syncwarp();
    ptx::cluster_sync();
  }
}

// `p` of this CTA's shared memory, in CTA `rank`'s.
template <int CL, class V>
__device__ __forceinline__ V* in_cta(V* p, uint32_t rank) {
  if constexpr (CL == 1) {
    return p;
  } else {
    uint64_t a;
    asm("mapa.u64 %0, %1, %2;" : "=l"(a) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
    return reinterpret_cast<V*>(a);
  }
}

// Running sums over the CTA's threads of two numbers, without the own ones; in
// all_a and all_b the whole.  Synchronises.
__device__ __forceinline__ void scan_cta(Shared& s, uint64_t& a, uint64_t& b, uint64_t& all_a, uint64_t& all_b) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint64_t a0 = a, b0 = b;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t x = __shfl_up_sync(~0u, a, d), y = __shfl_up_sync(~0u, b, d);
    if (lane >= d) {
      a += x;
      b += y;
    }
  }
  __syncthreads();
  if (lane == 31) {
    s.scan[0][warp] = a;
    s.scan[1][warp] = b;
  }
  __syncthreads();
  a -= a0;
  b -= b0;
  all_a = all_b = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    const uint64_t x = s.scan[0][w], y = s.scan[1][w];
    if (w < warp) {
      a += x;
      b += y;
    }
    all_a += x;
    all_b += y;
  }
}

// Sorts one value a thread, the largest first, over the first n (a power of
// two, 32 at least) threads.
template <class V>
__device__ __forceinline__ V sort_cta(V* buf, V x, int n) {
  const int tid = threadIdx.x;
  for (int size = 2; size <= n; size <<= 1) {
    for (int d = size >> 1; d > 0; d >>= 1) {
      V y;
      if (d >= 32) {
        __syncthreads();
        buf[tid] = x;
        __syncthreads();
        y = buf[tid ^ d];
      } else {
        y = __shfl_xor_sync(~0u, x, d);
      }
      const bool larger = ((tid & d) == 0) == ((tid & size) == 0);
      if (tid < n) x = larger == (x > y) ? x : y;
    }
  }
  return x;
}

// Bin of a logit: linear in it from the largest down.  Does not grow with x.
__device__ __forceinline__ int linear_bin(float x, float most, float step) {
  return x == most ? 0 : static_cast<int>(fminf((most - x) * step, static_cast<float>(BINS - 1)));
}

// The lowest key from lo to hi (which has one) whose bin is `bin` or less.
__device__ __noinline__ uint32_t lowest_key(uint32_t lo, uint32_t hi, float most, float step, int bin) {
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo) / 2;
    if (linear_bin(of_key(mid), most, step) <= bin) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// bf16 logits have few values: a place for each of magnitude 2^-14 to 2^7 in
// their order, from the largest down, and one in the middle for all that are
// smaller.  Weights are then looked up, and a histogram of the places says all
// that a border needs, unless it is in the middle.
struct Places {
  static constexpr int HALF = 2688, LOW = 0x3880;      // 2^-14 as the upper 16 bits
  static constexpr int COUNT = 2 * HALF + 1;
  static constexpr float MOST = 128.f;
  uint64_t weight[COUNT + 7];
  uint32_t count[COUNT + 7];
  static __device__ __forceinline__ int of(float x) {
    const uint32_t b = __float_as_uint(x);
    const int mag = max(static_cast<int>((b >> 16) & 0x7FFFu) - (LOW - 1), 0);
    return HALF + (static_cast<int>(b) < 0 ? mag : -mag);
  }
  static __device__ __forceinline__ float value(int place) {     // (not of the middle)
    const uint32_t mag = static_cast<uint32_t>(abs(place - HALF) + (LOW - 1));
    return __uint_as_float((mag << 16) | (place > HALF ? 0x80000000u : 0u));
  }
};

// *sum += w in shared memory, as two 32-bit additions, the upper one only where there
// is something to add: of the bulk of a row's weights seldom (250 rows of 250007 in
// fp32 by top_p 526 us, with 64-bit additions 592).
__device__ __forceinline__ void add_shared(uint64_t* sum, uint64_t w) {
  uint32_t* half = reinterpret_cast<uint32_t*>(sum);      // (little-endian)
  const uint32_t lo = static_cast<uint32_t>(w);
  const uint32_t old = atomicAdd(half, lo);
  const uint32_t up = static_cast<uint32_t>(w >> 32) + (old + lo < lo ? 1u : 0u);
  if (up != 0) atomicAdd(half + 1, up);
}

template <int DT, int CL>
struct Sampler {
  static constexpr int E = Elt<DT>::E;
  Shared& s;
  const Row& row;
  const Weigh& weigh;
  int begin, end;          // this CTA's slots
  uint32_t rank;
  int tid, lane, warp;
  uint32_t top_key;

  // A warp's own stretch of the slots.
  __device__ __forceinline__ void stretch(int& lo, int& hi) const {
    const int each = (end - begin + WARPS * 32 - 1) / (WARPS * 32) * 32;
    lo = min(begin + warp * each, end);
    hi = min(lo + each, end);
  }

  // The border in the keys [lo, hi], hi the largest logit's: where from the top
  // the tokens number `want` (by_count), or weigh `want`; want = 0: a share `p` of
  // the weight of all.  Every thread has the result.
  __device__ Border narrow(uint32_t lo, uint32_t hi, bool by_count, bool masses, uint64_t want, float p) {
    Border b{lo, ~0u, 0, 0, false};
    uint64_t above_mass = 0;
    uint32_t above = 0;
    const float most = weigh.most, low = of_key(lo);
    const float step = (BINS - 1) / (most - low);
    bool linear = most - low < INFINITY && step < INFINITY;
    while (true) {
      int shift = 0;
      while (((hi - lo) >> shift) >= BINS) ++shift;
      for (int i = tid; i < BINS; i += NT) {
        s.count[i] = 0;
        s.mass[i] = 0;
      }
      __syncthreads();
      int w0, w1;
      stretch(w0, w1);
      const float floor = of_key(lo);
      for_slots<DT>(row, w0 + lane, w1, 32, [&](int, const uint4& w) {
        if (!(largest<DT>(w) >= floor)) return;
        float x[E];
        unpack<DT>(w, x);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint32_t key = key_of(x[e]);
          if (key >= lo && key <= hi) {
            const int bin = linear ? linear_bin(x[e], most, step) : (hi - key) >> shift;
            atomicAdd(&s.count[bin], 1u);
            if (masses) add_shared(&s.mass[bin], weigh.at(x[e]));
          }
        }
      });
      sync_all<CL>();
      if (rank == 0) {
        constexpr int PER = BINS / NT;
        uint64_t cnt[PER], mass[PER], c = 0, m = 0, all_c, all_m;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          cnt[i] = mass[i] = 0;
          for (int r = 0; r < CL; ++r) {
            cnt[i] += in_cta<CL>(s.count, r)[tid * PER + i];
            if (masses) mass[i] += in_cta<CL>(s.mass, r)[tid * PER + i];
          }
          c += cnt[i];
          m += mass[i];
        }
        if (tid == 0) s.found = 0;
        scan_cta(s, c, m, all_c, all_m);
        if (want == 0) want = goal_of(all_m, p);          // once: the weight of all is known now
        if (tid == 0) {
          s.want = want;
          s.all = static_cast<uint32_t>(above + all_c);
          s.all_mass = above_mass + all_m;
        }
        uint64_t acc_c = above + c, acc_m = above_mass + m;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const uint64_t before = by_count ? acc_c : acc_m, here = by_count ? cnt[i] : mass[i];
          if (before < want && before + here >= want) {
            const int bin = tid * PER + i;
            s.found = 1;
            s.above = static_cast<uint32_t>(acc_c);
            s.above_mass = acc_m;
            s.in_bin = static_cast<uint32_t>(cnt[i]);
            if (linear) {
              s.lo = lowest_key(lo, hi, most, step, bin);
              s.hi = bin == 0 ? hi : lowest_key(lo, hi, most, step, bin - 1) - 1;
            } else {
              s.hi = hi - (static_cast<uint32_t>(bin) << shift);
              const uint32_t width = (1u << shift) - 1;
              s.lo = s.hi - lo > width ? s.hi - width : lo;
            }
          }
          acc_c += cnt[i];
          acc_m += mass[i];
        }
      }
      sync_all<CL>();
      const Shared& first = *in_cta<CL>(&s, 0);
      const bool found = first.found != 0;
      const uint32_t in_bin = first.in_bin, all = first.all;
      const uint64_t all_mass = first.all_mass;
      want = first.want;
      if (found) {
        lo = first.lo;
        hi = first.hi;
        above = first.above;
        above_mass = first.above_mass;
      }
      sync_all<CL>();
      if (!found) {            // fewer than wanted: all are kept
        b.above = all;
        b.above_mass = all_mass;
        return b;
      }
      linear = false;
      if (lo == hi) {
        b.key = lo;
        b.found = true;
        b.above = above;
        b.above_mass = above_mass;
        if (by_count) {
          b.ties = static_cast<uint32_t>(want - above);
        } else {
          const uint64_t each = max(weigh.at(of_key(lo)), uint64_t(1));
          b.ties = static_cast<uint32_t>(min((want - above_mass + each - 1) / each, static_cast<uint64_t>(in_bin)));
        }
        return b;
      }
    }
  }

  // This warp's weight above `last` and its tokens of that logit, in slots [w0, w1).
  template <class Weight>
  __device__ __forceinline__ void add_up(int w0, int w1, float last, const Weight& weight) {
    uint64_t mass = 0;
    uint32_t ties = 0;
    for_slots<DT>(row, w0 + lane, w1, 32, [&](int, const uint4& w) {
      if (!(largest<DT>(w) >= last)) return;
      float x[E];
      unpack<DT>(w, x);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (x[e] > last) mass += weight(x[e]);
        ties += x[e] == last ? 1 : 0;
      }
    });
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      mass += __shfl_xor_sync(~0u, mass, d);
      ties += __shfl_xor_sync(~0u, ties, d);
    }
    if (lane == 0) {
      s.warp_mass[warp] = mass;
      s.warp_ties[warp] = ties;
    }
  }

  // Of N warps' sums, where with what is before the kept weight passes `at`; what
  // is before becomes what is before that warp.  For every warp alike.
  template <int N>
  __device__ __forceinline__ int passes(const uint64_t (&m)[(N + 31) / 32], const uint32_t (&t)[(N + 31) / 32],
                                        uint64_t each, uint32_t ties, uint64_t at, uint64_t& mass_before,
                                        uint32_t& ties_before) const {
    int found = -1;
#pragma unroll
    for (int i = 0; i < (N + 31) / 32; ++i) {
      uint64_t up = m[i];
      uint32_t t_up = t[i];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint64_t y = __shfl_up_sync(~0u, up, d);
        const uint32_t z = __shfl_up_sync(~0u, t_up, d);
        if (lane >= d) {
          up += y;
          t_up += z;
        }
      }
      const uint32_t past =
          __ballot_sync(~0u, mass_before + up + each * min(ties, ties_before + t_up) > at);
      const int l = past != 0 ? __ffs(past) - 1 : 31;
      const uint64_t here = __shfl_sync(~0u, past != 0 ? up - m[i] : up, l);
      const uint32_t t_here = __shfl_sync(~0u, past != 0 ? t_up - t[i] : t_up, l);
      if (found < 0) {
        mass_before += here;
        ties_before += t_here;
        if (past != 0) found = i * 32 + l;
      }
    }
    return found;
  }

  // The token of the tokens from logit `key` on, of that logit itself the
  // first `ties`, at u of their weight.  The warps add up their stretches; the
  // CTA that has the one where the sum passes divides it among its warps once
  // more, and the warp where it passes then looks at 32 slots at a time.
  template <class Weight>
  __device__ void draw(uint32_t key, uint32_t ties, float u, int32_t* token, const Weight& weight) {
    const float last = of_key(key);
    const uint64_t each = weight(last);
    int w0, w1;
    stretch(w0, w1);
    add_up(w0, w1, last, weight);
    sync_all<CL>();
    constexpr int N = CL * WARPS, PER = (N + 31) / 32;
    uint64_t m[PER], all = 0;
    uint32_t t[PER], ties_all = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int w = i * 32 + lane;
      m[i] = t[i] = 0;
      if (w < N) {
        const Shared& o = *in_cta<CL>(&s, w / WARPS);
        m[i] = o.warp_mass[w % WARPS];
        t[i] = o.warp_ties[w % WARPS];
      }
      all += m[i];
      ties_all += t[i];
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      all += __shfl_xor_sync(~0u, all, d);
      ties_all += __shfl_xor_sync(~0u, ties_all, d);
    }
    bool more;
    const uint64_t at_u = part_of(all + each * min(ties, ties_all), u, more);
    uint64_t before = 0;
    uint32_t ties_before = 0;
    const int owner = passes<N>(m, t, each, ties, at_u, before, ties_before);
    sync_all<CL>();                     // every CTA has read the sums
    if (owner < 0 || owner / WARPS != static_cast<int>(rank)) return;
    const int per_warp = (end - begin + WARPS * 32 - 1) / (WARPS * 32) * 32;
    w0 = min(begin + owner % WARPS * per_warp, end);
    w1 = min(w0 + per_warp, end);
    const int part = (w1 - w0 + WARPS - 1) / WARPS;
    const int p0 = min(w0 + warp * part, w1), p1 = min(p0 + part, w1);
    add_up(p0, p1, last, weight);
    __syncthreads();
    uint64_t mm[1] = {lane < WARPS ? s.warp_mass[lane] : 0};
    uint32_t tt[1] = {lane < WARPS ? s.warp_ties[lane] : 0};
    if (passes<WARPS>(mm, tt, each, ties, at_u, before, ties_before) != warp) return;
    for (int at = p0; at < p1; at += 32) {
      float x[E];
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = -INFINITY;
      const bool in = at + lane < p1;
      if (in) unpack<DT>(load_slot<DT>(row, at + lane), x);
      uint64_t mass[1] = {0};
      uint32_t of_last[1] = {0};
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (x[e] > last) mass[0] += weight(x[e]);
        of_last[0] += in && x[e] == last ? 1 : 0;
      }
      const int l = passes<32>(mass, of_last, each, ties, at_u, before, ties_before);
      if (l < 0) continue;
      if (lane == l) {
        int hit = -1;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (x[e] > last) before += weight(x[e]);
          else if (in && x[e] == last) ++ties_before;
          if (hit < 0 && before + each * min(ties, ties_before) > at_u) hit = e;
        }
        *token = (at + lane) * E - row.off + hit;
      }
      return;
    }
  }

  __device__ void draw(uint32_t key, uint32_t ties, float u, int32_t* token) {
    draw(key, ties, u, token, [this](float x) { return weigh.at(x); });
  }

  // The list: the n tokens from some logit on; `all`: no others count.  Whether
  // the prefix ends inside it; then also the token.  For the first CTA.
  __device__ bool from_list(int n, bool all, int k, float p, uint64_t row_mass, float u, int32_t* token) {
    int size = 32;
    while (size < n) size <<= 1;
    const uint64_t x = sort_cta(s.sum, tid < n ? s.list[tid] : uint64_t(0), size);
    const uint32_t key = static_cast<uint32_t>(x >> 32), index = ~static_cast<uint32_t>(x);
    const uint64_t w = tid < n ? weigh.at(of_key(key)) : 0;
    uint64_t before = w, none = 0, sum, z;
    scan_cta(s, before, none, sum, z);
    int kept = n;
    bool closed = all;         // what top-k and min-p leave is in the list
    if (k > 0 && k <= n) {
      kept = k;
      closed = true;
    }
    if (!closed && k > 0) return false;
    if (p < 1.f) {
      uint64_t whole = row_mass;
      if (closed) {
        if (tid == kept - 1) s.want = before + w;
        __syncthreads();
        whole = s.want;
      }
      const uint64_t want = goal_of(whole, p);
      if (!closed && sum < want) return false;
      kept = max(__syncthreads_count(tid < kept && before < want), 1);
    }
    // by index, with the weights behind
    __syncthreads();
    s.list[tid] = w;
    const uint32_t y = sort_cta(reinterpret_cast<uint32_t*>(s.sum),
                                tid < kept ? ~(index << 9 | static_cast<uint32_t>(tid)) : 0u, size);
    __syncthreads();
    const uint32_t place = ~y;
    const uint64_t own = tid < kept ? s.list[place & 511] : 0;
    uint64_t up = own;
    none = 0;
    scan_cta(s, up, none, sum, z);
    bool more;
    const uint64_t at_u = part_of(sum, u, more);
    if (tid < kept && up <= at_u && at_u < up + own) *token = static_cast<int32_t>(place >> 9);
    return true;
  }
};

// The border by places: bf16 logits below 128 of which those above `cut` count.
// false: it is among the values of the middle place.  Every thread has the result.
template <int CL>
__device__ bool places_border(Shared& s, Places& t, const Row& row, const Weigh& weigh, int begin, int end,
                              uint32_t rank, float cut, int k, float p, Border& b) {
  constexpr int DT = TERN_LOGITS_BF16, E = Elt<DT>::E;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint64_t middle = 0;
  for_slots<DT>(row, begin + tid, end, NT, [&](int, const uint4& w) {
    if (!(largest<DT>(w) >= cut)) return;
    float x[E];
    unpack<DT>(w, x);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (x[e] >= cut) {
        const int place = Places::of(x[e]);
        atomicAdd(&t.count[place], 1u);
        if (place == Places::HALF) middle += weigh_rare(weigh, x[e]);
      }
    }
  });
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) middle += __shfl_xor_sync(~0u, middle, d);
  if (lane == 0) s.warp_mass[warp] = middle;
  sync_all<CL>();
  if (rank == 0) {
    constexpr int PER = (Places::COUNT + NT - 1) / NT;
    const int first = tid * PER;
    uint32_t cnt[PER];
    uint64_t c = 0, m = 0, all_c, all_m, mid = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      cnt[i] = 0;
      if (first + i < Places::COUNT)
        for (int r = 0; r < CL; ++r) cnt[i] += in_cta<CL>(t.count, r)[first + i];
      if (first + i == Places::HALF)
        for (int r = 0; r < CL; ++r)
          for (int w = 0; w < WARPS; ++w) mid += in_cta<CL>(s.warp_mass, r)[w];
      c += cnt[i];
    }
    const auto mass = [&](int i) {
      return first + i == Places::HALF ? mid : first + i < Places::COUNT ? cnt[i] * t.weight[first + i] : uint64_t(0);
    };
#pragma unroll
    for (int i = 0; i < PER; ++i) m += mass(i);
    if (tid == 0) s.found = 0;
    scan_cta(s, c, m, all_c, all_m);
    // top-k: the place where the count reaches it, and the weight of what it leaves
    if (tid == 0) s.all_mass = all_m;
    __syncthreads();
    uint64_t acc = c, acc_m = m;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (k > 0 && acc < k && acc + cnt[i] >= k) {
        const uint32_t ties = static_cast<uint32_t>(k - acc);
        s.found = first + i == Places::HALF ? -1 : 1;
        s.hi = first + i;
        s.in_bin = ties;
        if (first + i != Places::HALF) s.all_mass = acc_m + ties * t.weight[first + i];
      }
      acc += cnt[i];
      acc_m += mass(i);
    }
    __syncthreads();
    const int found = s.found;
    const uint32_t k_place = s.hi, k_ties = s.in_bin;
    __syncthreads();
    if (p < 1.f && found >= 0) {
      const uint64_t want = goal_of(s.all_mass, p);
      acc_m = m;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const uint64_t here = mass(i);
        if (acc_m < want && acc_m + here >= want) {
          const int place = first + i;
          s.found = place == Places::HALF ? -1 : 1;
          const uint64_t each = max(t.weight[place], uint64_t(1));
          uint32_t ties = static_cast<uint32_t>(min((want - acc_m + each - 1) / each, static_cast<uint64_t>(cnt[i])));
          if (found == 1 && k_place == place) ties = min(ties, k_ties);
          s.lo = place;
          s.above = ties;
        }
        acc_m += here;
      }
    } else if (tid == 0) {
      s.lo = k_place;
      s.above = k_ties;
    }
  }
  sync_all<CL>();
  const Shared& from = *in_cta<CL>(&s, 0);
  const int found = from.found;
  b.found = found > 0;
  b.key = key_of(found > 0 ? Places::value(from.lo) : cut);
  b.ties = found > 0 ? from.above : ~0u;
  sync_all<CL>();
  return found >= 0;
}

template <int DT, int CL>
__global__ void __launch_bounds__(NT, 2) sample_kernel(const __grid_constant__ SampleArgs a) {
  constexpr int E = Elt<DT>::E;
  __shared__ Shared s;
  extern __shared__ __align__(16) uint8_t dynamic[];
  Places& places = *reinterpret_cast<Places*>(dynamic);      // bf16
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = CL == 1 ? 0 : ptx::cluster_ctarank();
  const int64_t r = blockIdx.x / CL;
  if (tid < 32) s.table[tid] = make_uint2(kRoots[tid], __float_as_uint(static_cast<float>(kRoots[tid])));
  if (tid == 0) {
    s.n = 0;
    s.done = 0;
  }
  for (int i = tid; i < BINS; i += NT) s.count[i] = 0;
  pdl_wait();
  pdl_launch_dependents();
  Row row;
  row.at = a.logits + r * a.row_stride * Elt<DT>::BYTES;
  row.off = static_cast<int>((reinterpret_cast<uintptr_t>(row.at) & 15) / Elt<DT>::BYTES);
  row.vocab = a.vocab;
  const int slots = (row.off + a.vocab + E - 1) / E;
  const int each = (slots + CL - 1) / CL;
  const int begin = min(static_cast<int>(rank) * each, slots), end = min(begin + each, slots);
  const float temperature = a.temperature != nullptr ? a.temperature[r] : 1.f;
  int k = a.top_k != nullptr ? a.top_k[r] : 0;
  float p = a.top_p != nullptr ? a.top_p[r] : 1.f;
  const float min_p = a.min_p != nullptr ? fminf(a.min_p[r], 1.f) : 0.f;
  float u = a.u[r];
  u = u > 0.f ? fminf(u, 0x1.fffffep-1f) : 0.f;
  if (k >= a.vocab || k < 0) k = 0;
  p = p < 1.f ? fmaxf(p, 0.f) : 1.f;                // (a NaN: 1)

  // 64-bit arithmetic is slow here: one warp's, while the others wait for the row
  if (warp == WARPS - 1) {
    const double c = 1.4426950408889634 / static_cast<double>(temperature);
    double span = -static_cast<double>(kReach) / c;                 // with a weight, and min-p's
    if (min_p > 0.f) span = fmax(span, log(static_cast<double>(min_p)) * static_cast<double>(temperature));
    const float c_hi = static_cast<float>(c), c_lo = static_cast<float>(c - static_cast<double>(c_hi));
    s.c = c_hi;
    s.c_lo = fabsf(c_lo) < INFINITY ? c_lo : 0.f;
    s.span = span;
  }

  // the largest
  float mine = -INFINITY;
  for_slots<DT>(row, begin + tid, end, NT, [&](int, const uint4& w) { mine = fmaxf(mine, largest<DT>(w)); });
  float most = mine;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, d));
  if (lane == 0) s.warp_max[warp] = most;
  __syncthreads();
  most = s.warp_max[0];
#pragma unroll
  for (int w = 1; w < WARPS; ++w) most = fmaxf(most, s.warp_max[w]);
  if constexpr (CL > 1) {
    if (tid == 0) s.cta_max = most;
    sync_all<CL>();
    for (int i = 0; i < CL; ++i) most = fmaxf(most, *in_cta<CL>(&s.cta_max, i));
  }

  const Weigh weigh{most, s.c, s.c_lo, s.table};
  Sampler<DT, CL> sampler{s, row, weigh, begin, end, rank, tid, lane, warp, key_of(most)};
  if (most == -INFINITY) {
    if (rank == 0 && tid == 0) a.token[r] = -1;
    if constexpr (CL > 1) sync_all<CL>();      // others still read this CTA's largest
    return;
  }
  if (!(temperature > 0.f) || k == 1 || p == 0.f) {
    sampler.draw(key_of(most), 1, 0.f, a.token + r);
    if constexpr (CL > 1) sync_all<CL>();
    return;
  }
  // the lowest logit that counts
  const double low = static_cast<double>(most) + s.span;
  const float cut = fminf(low == low ? __double2float_ru(low) : most, most);
  const uint32_t cut_key = key_of(cut);
  const int aim = max(k, 160);
  const bool list = aim <= 384;
  // a bf16 row whose survivors may be many: by places
  if constexpr (DT == TERN_LOGITS_BF16) {
    if (most < Places::MOST && cut > -Places::MOST && !(k > 0 && list)) {
      for (int i = tid; i < Places::COUNT; i += NT) {
        const float x = Places::value(i);
        places.weight[i] = i != Places::HALF && x <= most && x >= cut ? weigh.at(x) : 0;
        places.count[i] = 0;
      }
      __syncthreads();
      Border b{cut_key, ~0u, 0, 0, false};
      if ((k == 0 && p >= 1.f) || places_border<CL>(s, places, row, weigh, begin, end, rank, cut, k, p, b)) {
        sampler.draw(b.key, b.ties, u, a.token + r, [&](float x) {
          const int place = Places::of(x);
          return place == Places::HALF ? weigh_rare(weigh, x) : places.weight[place];
        });
        if constexpr (CL > 1) sync_all<CL>();
        return;
      }
    }
  }
  if (k == 0 && p >= 1.f) {
    sampler.draw(cut_key, ~0u, u, a.token + r);
    if constexpr (CL > 1) sync_all<CL>();
    return;
  }

  // a bound that `aim` of the threads' largest reach
  uint32_t bound = cut_key;
  const float step = (BINS - 1) / (most - cut);
  if (list && most - cut < INFINITY && step < INFINITY) {
    if (mine >= cut) atomicAdd(&s.count[linear_bin(mine, most, step)], 1u);
    sync_all<CL>();
    if (rank == 0) {
      constexpr int PER = BINS / NT;
      uint64_t cnt[PER], sum = 0, none = 0, all, z;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        cnt[i] = 0;
        for (int q = 0; q < CL; ++q) cnt[i] += in_cta<CL>(s.count, q)[tid * PER + i];
        sum += cnt[i];
      }
      if (tid == 0) s.lo = cut_key;
      scan_cta(s, sum, none, all, z);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (sum < aim && sum + cnt[i] >= aim)
          s.lo = lowest_key(cut_key, key_of(most), most, step, tid * PER + i);
        sum += cnt[i];
      }
    }
    sync_all<CL>();
    bound = in_cta<CL>(&s, 0)->lo;
  }
  if (list) {
    // gather; where a share of all of the row's weight is asked for, add that up too
    const bool all = bound <= cut_key;
    const bool sums = p < 1.f && k == 0 && !all;
    const float from = of_key(bound);
    uint64_t mass = 0;
    Shared& first = *in_cta<CL>(&s, 0);
    for_slots<DT>(row, begin + tid, end, NT, [&](int at, const uint4& w) {
      if (!(largest<DT>(w) >= (sums ? cut : from))) return;
      float x[E];
      unpack<DT>(w, x);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (sums && x[e] >= cut) mass += weigh.at(x[e]);
        const int index = at * E - row.off + e;
        if (x[e] >= from && index >= 0 && index < a.vocab) {
          const uint32_t i = atomicAdd(&first.n, 1u);
          if (i < NT) first.list[i] = static_cast<uint64_t>(key_of(x[e])) << 32 | ~static_cast<uint32_t>(index);
        }
      }
    });
    if (sums) {
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) mass += __shfl_xor_sync(~0u, mass, d);
      if (lane == 0) s.warp_mass[warp] = mass;
    }
    sync_all<CL>();
    if (rank == 0) {
      const int n = static_cast<int>(min(s.n, static_cast<uint32_t>(NT + 1)));
      uint64_t row_mass = 0;
      if (sums)
        for (int q = 0; q < CL; ++q)
          for (int w = 0; w < WARPS; ++w) row_mass += in_cta<CL>(s.warp_mass, q)[w];
      if (n <= NT) {
        const bool ok = sampler.from_list(n, all, k, p, row_mass, u, a.token + r);
        if (tid == 0) s.done = ok ? 1 : 0;
      }
    }
    sync_all<CL>();
    const bool done = first.done != 0;
    if constexpr (CL > 1) sync_all<CL>();
    if (done) return;
  }

  // the border by histograms
  const uint32_t top = key_of(most);
  Border b{cut_key, ~0u, 0, 0, false};
  uint64_t want = 0;
  uint32_t k_key = cut_key, k_ties = ~0u;
  if (k > 0) {
    b = sampler.narrow(cut_key, top, true, p < 1.f, static_cast<uint64_t>(k), 0.f);
    if (b.found) {
      k_key = b.key;
      k_ties = b.ties;
    }
    if (p < 1.f)
      want = goal_of(b.found ? b.above_mass + b.ties * weigh.at(of_key(b.key)) : b.above_mass, p);
  }
  if (p < 1.f) {
    const Border q = sampler.narrow(k_key, top, false, true, want, p);
    if (q.found) {
      b = q;
      if (q.key == k_key) b.ties = min(q.ties, k_ties);
    }
  }
  sampler.draw(b.key, b.found ? b.ties : ~0u, u, a.token + r);
  if constexpr (CL > 1) sync_all<CL>();
}

// ------------------------------------------------------------------ accept
//
// A warp a request.  A path goes up, so 32 rows at a time are looked at once:
// the first that fits the path's last row is the next, and its target is in
// the lane that has it.  Bound: the launch and two dependent reads.

constexpr int ACCEPT_THREADS = 128;

struct AcceptArgs {
  const int32_t* tokens;
  const int32_t* target;
  const int32_t* parent;
  const int32_t* row_start;
  int32_t* path;
  int32_t* path_len;
  int32_t* next;
  int64_t T;
  int B, width;
};

// A warp has a request: its lanes look among 32 drafts at a time for the child with
// the wanted token.  A chain of dependent reads, 2.2 us for one step's requests,
// launch included (2.8 for 1000).
__global__ void __launch_bounds__(ACCEPT_THREADS) accept_kernel(const __grid_constant__ AcceptArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int b = (blockIdx.x * ACCEPT_THREADS + threadIdx.x) >> 5;
  if (b >= a.B) return;
  const int64_t s0 = a.row_start[b], s1 = a.row_start[b + 1];
  const bool ok = s0 >= 0 && s1 >= s0 && s1 <= a.T;
  const int n = ok ? static_cast<int>(min(s1 - s0, int64_t(a.width))) : 0;
  int32_t* path = a.path + int64_t(b) * a.width;
  int len = 0, cur = -1, want = -1;
  for (int base = 0; base < n; base += 32) {
    const int j = base + lane;
    const bool in = j < n;
    const int token = in ? a.tokens[s0 + j] : 0;
    const int parent = in && j > 0 ? a.parent[s0 + j] : -1;
    const int target = in ? a.target[s0 + j] : 0;
    if (base == 0) {
      cur = 0;
      want = __shfl_sync(~0u, target, 0);
      if (lane == 0) path[0] = 0;
      len = 1;
    }
    while (true) {
      const uint32_t fits = __ballot_sync(~0u, in && j > cur && parent == cur && token == want);
      if (fits == 0) break;
      const int l = __ffs(fits) - 1;
      cur = base + l;
      want = __shfl_sync(~0u, target, l);
      if (lane == 0) path[len] = cur;
      ++len;
    }
  }
  for (int i = len + lane; i < a.width; i += 32) path[i] = -1;
  if (lane == 0) {
    a.path_len[b] = len;
    a.next[b] = want;
  }
}

template <int DT, int CL>
cudaError_t launch_sample_cl(const SampleArgs& a, int64_t rows, cudaStream_t st) {
  constexpr size_t smem = DT == TERN_LOGITS_BF16 ? sizeof(Places) : 0;
  static std::atomic<unsigned long long> attr_done{0};
  const cudaError_t e = once_per_device(attr_done, [] {
    return cudaFuncSetAttribute(sample_kernel<DT, CL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(smem));
  });
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(rows * CL));
  if constexpr (CL == 1) return launch(sample_kernel<DT, 1>, grid, dim3(NT), smem, st, a);
  else return launch_cluster(sample_kernel<DT, CL>, grid, dim3(NT), smem, st, CL, a);
}

template <int DT>
cudaError_t launch_sample_type(const SampleArgs& a, int64_t rows, cudaStream_t st) {
  // CTAs a row: as many as the GPU holds at once (two an SM), while half of the
  // threads have a slot of their own. Beyond that, up to `most` an SM in turn,
  // while each keeps `least` elements: long rows then end together, although
  // some need more passes than others, but each CTA of a bf16 row also clears and
  // adds up places. us with the CTAs that the GPU holds, then with this rule
  // (mixed filters, top_k alone):
  //   304 x 250007 bf16     222, 93 -> 158, 99      304 x 250007 fp32   668 -> 310
  //   200 x 128256 bf16     121, 60 ->  85, 67      200 x 128256 fp32   349 -> 196
  //   152 x 250007 bf16     106, 53 (4 a row: 107, 82)
  //   152 x  32011 bf16      35, 25 (2 a row: 65, 49)
  constexpr bool PLACES = DT == TERN_LOGITS_BF16;
  constexpr int64_t most = PLACES ? 6 : 12, least = PLACES ? 64000 : 16000;
  const int64_t sms = kv_sm_count();
  int cl = 1;
  while (cl < MAX_CL) {
    const int64_t ctas = rows * (2 * cl), part = a.vocab / (2 * cl);
    if (!(ctas <= 2 * sms && part / Elt<DT>::E >= NT / 2) && !(ctas <= most * sms && part >= least)) break;
    cl *= 2;
  }
  if (cl == 8) return launch_sample_cl<DT, 8>(a, rows, st);
  if (cl == 4) return launch_sample_cl<DT, 4>(a, rows, st);
  if (cl == 2) return launch_sample_cl<DT, 2>(a, rows, st);
  return launch_sample_cl<DT, 1>(a, rows, st);
}

}  // namespace

cudaError_t launch_sample(const void* logits, int64_t row_stride, int64_t rows, int64_t vocab, int dtype,
                          const float* u, const float* temperature, const int32_t* top_k, const float* top_p,
                          const float* min_p, int32_t* token, cudaStream_t st) {
  const SampleArgs a{static_cast<const uint8_t*>(logits), u, temperature, top_k, top_p, min_p, token, row_stride,
                     static_cast<int>(vocab)};
  if (dtype == TERN_LOGITS_BF16) return launch_sample_type<TERN_LOGITS_BF16>(a, rows, st);
  if (dtype == TERN_LOGITS_F16) return launch_sample_type<TERN_LOGITS_F16>(a, rows, st);
  return launch_sample_type<TERN_LOGITS_F32>(a, rows, st);
}

cudaError_t launch_tree_accept(const int32_t* tokens, const int32_t* target, const int32_t* parent,
                               const int32_t* row_start, int64_t B, int64_t T, int64_t path_width, int32_t* path,
                               int32_t* path_len, int32_t* next, cudaStream_t st) {
  const AcceptArgs a{tokens, target, parent, row_start, path, path_len, next, T, static_cast<int>(B),
                     static_cast<int>(path_width)};
  const int64_t blocks = (B + ACCEPT_THREADS / 32 - 1) / (ACCEPT_THREADS / 32);
  return launch(accept_kernel, dim3(static_cast<unsigned>(blocks)), dim3(ACCEPT_THREADS), 0, st, a);
}

}  // namespace tern
