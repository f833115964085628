// Code shared by the attention kernels over the 8-bit cache: arguments, codes to
// fp16, how a tile of codes lies in shared memory.
#pragma once

#include "attn_dev.cuh"

namespace tern {
namespace attn {

// Room for the arrival counters of this many CTAs.
constexpr int MAX_GRID8 = TERN_TREE_ATTENTION_ZERO_BYTES / (3 * sizeof(int));

enum Kind { I8 = 1, E4M3 = 2 };

// Values' units below this count as this in the reference of a row's exponents, as
// a unit of 0 would leave none.  So a key's 2^(t_j - m) is below 2^106 whatever its
// unit is, and sums over millions of such keys stay below 2^128 (2^-100 let some
// thousands pass it).  What is rounded to fp16 then has 2^-25 of 2^-9 left at the
// smallest unit that is written, 2^-107, and all its bits from 2^-90 on.
constexpr float kLeastUnit = 0x1p-90f;

struct Args8 {
  Args a;
  const float* ku;
  const float* vu;
  int64_t unit_page, unit_head;
};

// Four codes to two pairs of fp16: (0, 1) and (2, 3).
template <int KIND>
__device__ __forceinline__ void widen(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (KIND == I8) {
    // 1024 + (code + 128) has the byte in its last bits
    w ^= 0x80808080u;
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));     // 1152
    const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), bias);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), bias);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  } else {
    asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\n"
        "cvt.rn.f16x2.e4m3x2 %0, a;\ncvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(lo), "=r"(hi) : "r"(w));
  }
}

// Where 16-byte chunk c of row r of a tile's part is (the copies' swizzle).
template <int ROWB>
__device__ __forceinline__ int chunk_at(int r, int c) {
  return ROWB == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// The cache as [pages][heads][rows][dim]: boxes of `rows` rows of one page and
// head, up to 128 codes wide (swizzled).
inline bool make_map8(CUtensorMap* map, const tern_kv_cache8& c, void* base, int rows) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.dim), static_cast<cuuint64_t>(c.page_size),
                              static_cast<cuuint64_t>(c.heads), static_cast<cuuint64_t>(c.pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.token_stride),
                                 static_cast<cuuint64_t>(c.head_stride),
                                 static_cast<cuuint64_t>(c.page_stride)};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(std::min<int64_t>(c.dim, 128)),
                             static_cast<cuuint32_t>(rows), 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, base, dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             c.dim == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace attn

// The tile kernel's calls (attn8_tile.cu).
cudaError_t launch_attn8_tile(const TreeAttn8Call& call, const attn::Args8& g, cudaStream_t st);
cudaError_t attn8_tile_read_clear_error(unsigned int* err);

}  // namespace tern
