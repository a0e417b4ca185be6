// Shared pieces of the operators around the expert layer (include/moe_block.h):
// host-side argument checks, row element types, wave reductions.
#pragma once

#include "route.h"
#include "moe_block.h"

namespace moe {

// Argument checks shared with the expert layer's entry points (api.hip).
int validate_dims(const moe_dims* d);
int validate_route_out(const moe_route_out* r, bool for_route);
int32_t max_blocks_of(const moe_dims& d);

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int launched(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ELAUNCH; }
inline bool elem_ok(int type) { return type == MOE_ELEM_F32 || type == MOE_ELEM_BF16 || type == MOE_ELEM_F16; }
inline int elem_bytes(int type) { return type == MOE_ELEM_F32 ? 4 : 2; }

// Entry b of a block map of *n entries; false past its end.  The length is
// waited for first, so that entries behind the map are never read; loading the
// two together was no faster (gate/up of one token 8.0 us, of 16 33.2, either
// way: the length lands under the division that finds b).
__host__ __device__ inline bool map_entry(const int4* blocks, const int32_t* n, int b, int4& e) {
  if (b >= *n) return false;
  e = blocks[b];
  return true;
}

// Launches of more workgroups than x takes (a launch holds fewer than 2^32
// threads in x): rows of kGridX of them along y.  Workgroups of the last row
// past the count find no work.
constexpr unsigned kGridX = 1u << 20;
inline dim3 grid_of(unsigned groups) {
  return dim3(groups < kGridX ? groups : kGridX, (groups + kGridX - 1) / kGridX);
}
__device__ __forceinline__ unsigned workgroup() { return blockIdx.y * kGridX + blockIdx.x; }

// ---------------------------------------------------------------------------
// Row elements.  Elem<TYPE>::V elements make one 16-byte access.
// ---------------------------------------------------------------------------
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

template <int TYPE>
struct Elem;

template <>
struct Elem<MOE_ELEM_F32> {
  static constexpr int V = 4;
  static __device__ __forceinline__ void unpack(uint4 r, float* v) {
    v[0] = __uint_as_float(r.x);
    v[1] = __uint_as_float(r.y);
    v[2] = __uint_as_float(r.z);
    v[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* v) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
  }
};

template <>
struct Elem<MOE_ELEM_BF16> {
  static constexpr int V = 8;
  static __device__ __forceinline__ void unpack(uint4 r, float* v) {
    const uint32_t p[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(p[i] << 16);
      v[2 * i + 1] = __uint_as_float(p[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* v) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
  }
};

// Two float32 -> packed half pair (low half = a), each rounded to nearest even.
__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
  const f16x2 r = {static_cast<_Float16>(a), static_cast<_Float16>(b)};
  return __builtin_bit_cast(uint32_t, r);
}

template <>
struct Elem<MOE_ELEM_F16> {
  static constexpr int V = 8;
  static __device__ __forceinline__ void unpack(uint4 r, float* v) {
    const uint32_t p[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f16x2 h = __builtin_bit_cast(f16x2, p[i]);
      v[2 * i] = static_cast<float>(h[0]);
      v[2 * i + 1] = static_cast<float>(h[1]);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* v) {
    return make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]),
                      pack_f16x2(v[6], v[7]));
  }
};

// ---------------------------------------------------------------------------
// Streaming accesses: NT marks data that is not used again before it would be
// evicted anyway, so that it does not push out what is.  An array larger than
// the L2s together (8 x 4 MB) leaves them before a later kernel reads it; one
// larger than a quarter of the 256 MB last-level cache does not stay there
// next to the other arrays of a step.
// ---------------------------------------------------------------------------
constexpr size_t kStreamStore = 32u << 20;
constexpr size_t kStreamLoad = 64u << 20;

template <bool NT>
__device__ __forceinline__ uint4 load16(const uint4* p) {
  if (!NT) return *p;
  const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  return make_uint4(v[0], v[1], v[2], v[3]);
}
template <bool NT>
__device__ __forceinline__ void store16(uint4* p, uint4 v) {
  if (!NT)
    *p = v;
  else
    __builtin_nontemporal_store(u32x4{v.x, v.y, v.z, v.w}, reinterpret_cast<u32x4*>(p));
}

// ---------------------------------------------------------------------------
// Reductions over a wave of 64, every lane gets the result: four steps inside
// the 16-lane DPP rows (pairs, quads, halves of eight, the row), then the rows
// against each other with the two swap instructions.  The order is fixed.
// ---------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, false));
}
constexpr int kDppXor1 = 0xB1;         // quad_perm(1,0,3,2)
constexpr int kDppXor2 = 0x4E;         // quad_perm(2,3,0,1)
constexpr int kDppHalfMirror = 0x141;  // lane i of eight <- lane 7 - i
constexpr int kDppMirror = 0x140;      // lane i of sixteen <- lane 15 - i

__device__ __forceinline__ float wave_sum(float x) {
  x += __uint_as_float(dpp<kDppXor1>(__float_as_uint(x)));
  x += __uint_as_float(dpp<kDppXor2>(__float_as_uint(x)));
  x += __uint_as_float(dpp<kDppHalfMirror>(__float_as_uint(x)));
  x += __uint_as_float(dpp<kDppMirror>(__float_as_uint(x)));
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  x = max(x, dpp<kDppXor1>(x));
  x = max(x, dpp<kDppXor2>(x));
  x = max(x, dpp<kDppHalfMirror>(x));
  x = max(x, dpp<kDppMirror>(x));
  const auto a = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  x = max(static_cast<uint32_t>(a[0]), static_cast<uint32_t>(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return max(static_cast<uint32_t>(b[0]), static_cast<uint32_t>(b[1]));
}

}  // namespace moe
