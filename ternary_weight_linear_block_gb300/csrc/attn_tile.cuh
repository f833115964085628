// Code shared by the tcgen05 attention kernels, of 16-bit and 8-bit caches: the
// order of tiles in the ring, descriptors, loads from and stores to tensor
// memory, and the kernel that joins their pieces.
#pragma once

#include "attn_dev.cuh"

namespace tern {
namespace attn {

// Places of the keys and values of an item's i-th tile of cnt in the ring's
// order, the keys AHEAD tiles before the values.
template <int AHEAD>
__device__ __forceinline__ uint32_t k_place(int i) {
  return i <= AHEAD ? i : 2 * i - AHEAD;
}
template <int AHEAD>
__device__ __forceinline__ uint32_t v_place(int i, int cnt) {
  return 2 * i + 1 + AHEAD - max(0, i - (cnt - 1 - AHEAD));
}

// Descriptor of V [keys][64 columns] as the MN-major B operand: 8 keys of 128
// bytes make an atom of the 128-byte swizzle, atoms 1024 bytes apart along
// the keys (stride byte offset), the next 64 columns `lbo` bytes on.
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t addr, uint32_t lbo) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(lbo >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}
template <bool BF16>
__host__ __device__ constexpr uint32_t idesc(int n, bool b_mn) {
  return (1u << 4) | ((BF16 ? 1u : 0u) << 7) | ((BF16 ? 1u : 0u) << 10) |
         ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// Wait for this thread's loads from tensor memory; what was loaded into v
// cannot be used before it.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                   "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                   "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]),
                   "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                   "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                   "+r"(v[30]), "+r"(v[31])
               :
               : "memory");
}

__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                 "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                 "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
               :
               : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n.reg .pred p;\n"
      "elect.sync _|p, 0xffffffff;\n"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(p));
  return p != 0;
}

// Two 32-bit operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(x)), "l"(reinterpret_cast<uint64_t&>(y)),
        "l"(reinterpret_cast<uint64_t&>(z)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(x)), "l"(reinterpret_cast<uint64_t&>(y)));
  return d;
}

// Scores that a row does not see.
__device__ __forceinline__ void mask_out(uint32_t (&v)[32], uint32_t vis) {
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (!((vis >> e) & 1)) v[e] = 0xFF800000u;
}

// ------------------------------------------------------------------ join
//
// The items that several CTAs of the tile kernel share, a thread for each
// (row, 4 columns) place, rows first as the pieces are stored.  Hundreds of
// pieces (one long context on one key head) would be read one after another
// that way, so from JOIN_GROUPS pieces on a place has that many threads, each
// with a running sum over every JOIN_GROUPS-th piece, which are added in
// order.  The blocks share the passes of all items (each adds up for itself
// where they lie), because a few items with many pieces and many with few
// would otherwise leave most blocks without work.  Bound by the launch and
// three round trips to L2, with many rows by L2's rate.  Joined by the last
// CTA to arrive, as the rows kernel does, these items cost more: a context of
// 131001 keys 111 us against 94, 512 rows a key head 198 against 170.
constexpr int JOIN_THREADS = 256, JOIN_GROUPS = 8;
static_assert(JOIN_THREADS == 1 << 8 && JOIN_THREADS / JOIN_GROUPS == 1 << 5, "passes");
// Room for the arrival counters of this many CTAs (two an SM).
constexpr int MAX_GRID = TERN_TREE_ATTENTION_ZERO_BYTES / (3 * sizeof(int));

template <bool BF16, int D>
__global__ void __launch_bounds__(JOIN_THREADS) combine_kernel(const Args a, int rt, int ctas) {
  __shared__ float4 s_o[JOIN_THREADS];
  __shared__ float2 s_ml[JOIN_THREADS];
  __shared__ Item s_item[MAX_GRID];
  __shared__ int s_first[MAX_GRID];         // passes before each CTA's item
  __shared__ int s_warp[JOIN_THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31;
  pdl_wait();
  pdl_launch_dependents();
  int total = 0;
  for (int base = 0; base < ctas; base += JOIN_THREADS) {
    int n = 0;
    if (base + tid < ctas) {
      const Item it = a.items[base + tid];
      s_item[base + tid] = it;
      const int shift = it.follow + 1 < JOIN_GROUPS ? 8 : 5;      // log2 of a pass's places
      if (it.follow > 0) n = (it.rows * (D / 4) + (1 << shift) - 1) >> shift;
    }
    int x = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(~0u, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) s_warp[tid >> 5] = x;
    __syncthreads();
    int below = total;
    for (int w = 0; w < JOIN_THREADS / 32; ++w) {
      if (w < (tid >> 5)) below += s_warp[w];
      total += s_warp[w];
    }
    if (base + tid < ctas) s_first[base + tid] = below + x - n;
    __syncthreads();
  }
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    int lo = 0, hi = ctas;                   // the last CTA with s_first <= u has pass u
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_first[mid] <= u) lo = mid; else hi = mid;
    }
    const Item it = s_item[lo];
    const int groups = it.follow + 1 < JOIN_GROUPS ? 1 : JOIN_GROUPS;
    const int shift = groups == 1 ? 8 : 5, width = 1 << shift;
    const int p = tid & (width - 1), g = tid >> shift;
    const int place = (u - s_first[lo]) * width + p;
    const bool in = place < it.rows * (D / 4);
    const int d4 = place / it.rows, r = place - d4 * it.rows;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in) {
      // piece i: slot 1 of CTA `first`, then slot 0 of CTA first + i
#pragma unroll 4
      for (int i = g; i <= it.follow; i += groups) {
        const int64_t slot = 2 * (int64_t(it.first) + i) + (i == 0 ? 1 : 0);
        add_piece(m, l, o, a.part_ml[slot * rt + r],
                  *reinterpret_cast<const float4*>(a.part_o + ((slot * (D / 4) + d4) * rt + r) * 4));
      }
    }
    if (groups > 1) {
      s_o[tid] = o;
      s_ml[tid] = make_float2(m, l);
      __syncthreads();
      if (g == 0)
        for (int i = 1; i < JOIN_GROUPS; ++i)
          add_piece(m, l, o, s_ml[i * width + p], s_o[i * width + p]);
    }
    if (g == 0 && in) write_joined<BF16, D>(a, it, r, d4, m, l, o);
    if (groups > 1) __syncthreads();
  }
}

// The queries as [T][Hq][dim]: boxes of `tokens` tokens, the group's heads and 64
// values (128 bytes, swizzled).
inline bool make_query_map(CUtensorMap* map, const void* q, bool bf16, int64_t dim, int64_t Hq, int64_t T,
                           int64_t head_stride, int64_t token_stride, int tokens, int group) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(Hq),
                              static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_stride) * 2,
                                 static_cast<cuuint64_t>(token_stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(tokens)};
  const cuuint32_t estr[3] = {1, 1, 1};
  const auto type = bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return enc(map, type, 3, const_cast<void*>(q), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace attn
}  // namespace tern
