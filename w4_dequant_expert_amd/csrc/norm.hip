// Residual addition with its root-mean-square norm, with an 8-bit output, and
// the gradient (include/moe_block.h).
//
// Forward, per row of H elements:  s = x + r,  rho = 1 / sqrt(mean(s^2) + eps),
// y = s rho w;  a = max|y|, yq = rint(127 y / a), ys = a / 127.
// Backward, with xh = s rho and g = dy w:
//   dx = rho (g - xh mean(g xh)) + dsum = rho g - s rho^3 mean(g s) + dsum,
//   dw = sum over rows of dy xh.
//
// Both are bound by memory: about ten operations an element against 8 bytes
// (two bfloat16 rows read, two written).  A row therefore stays in registers
// from its one read to its writes; the sums (s^2, g s) and the maximum need
// the whole row, so they are reduced across the row's lanes in between.  All
// arithmetic is float32; each output is rounded once.
//
// A row belongs to NW waves (1, 4 or 16) with C chunks of eight elements per
// lane: one wave has no barrier and no LDS, several waves shorten the row's
// latency and hold longer rows.
#include "block.h"

namespace moe {
namespace {

constexpr int kMaxNormH = 16384;

// Eight elements of a row, raw.
template <int TYPE>
struct Raw8 {
  uint4 q[8 / Elem<TYPE>::V];
};

template <int TYPE, bool NT>
__device__ __forceinline__ Raw8<TYPE> load8(const void* base, size_t chunk) {
  constexpr int n = 8 / Elem<TYPE>::V;
  Raw8<TYPE> r;
#pragma unroll
  for (int i = 0; i < n; ++i) r.q[i] = load16<NT>(static_cast<const uint4*>(base) + chunk * n + i);
  return r;
}

template <int TYPE>
__device__ __forceinline__ void unpack8(const Raw8<TYPE>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8 / Elem<TYPE>::V; ++i) Elem<TYPE>::unpack(r.q[i], v + i * Elem<TYPE>::V);
}

template <int TYPE, bool NT>
__device__ __forceinline__ void store8(void* base, size_t chunk, const float (&v)[8]) {
  constexpr int n = 8 / Elem<TYPE>::V;
#pragma unroll
  for (int i = 0; i < n; ++i)
    store16<NT>(static_cast<uint4*>(base) + chunk * n + i, Elem<TYPE>::pack(v + i * Elem<TYPE>::V));
}

__device__ __forceinline__ void load_weight8(const float* w, int chunk, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(w)[chunk * 2];
  const float4 b = reinterpret_cast<const float4*>(w)[chunk * 2 + 1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Sum or maximum over a row's NW waves; `red` holds NW words of its own for
// each use between two barriers.
template <int NW>
__device__ __forceinline__ float row_sum(float x, float* red, int wave) {
  x = wave_sum(x);
  if (NW == 1) return x;
  if ((threadIdx.x & 63) == 0) red[wave] = x;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < NW; ++i) t += red[i];
  return t;
}

template <int NW>
__device__ __forceinline__ uint32_t row_max(uint32_t x, uint32_t* red, int wave) {
  x = wave_max(x);
  if (NW == 1) return x;
  if ((threadIdx.x & 63) == 0) red[wave] = x;
  __syncthreads();
  uint32_t t = 0;
#pragma unroll
  for (int i = 0; i < NW; ++i) t = max(t, red[i]);
  return t;
}

// One row's 8-bit scale from the bits of its largest |y|.  As unsigned
// integers the bits of |y| order like the values, with infinities and NaNs on
// top, so the maximum also tells a row that holds one of them: its scale is
// NaN and its codes 0.  Rows smaller than 2^-100 are scaled up (exactly) first, so
// that 127 / a stays finite; a row of zeros gives scale 0 and codes 0.
struct RowScale {
  float up, inv, scale;
  bool bad;
};
__device__ __forceinline__ RowScale row_scale(uint32_t abits) {
  const float a = __uint_as_float(abits);
  RowScale r;
  r.bad = abits >= 0x7F800000u;
  r.up = a < 0x1p-100f ? 0x1p100f : 1.0f;
  r.inv = (a > 0.0f && !r.bad) ? 127.0f / (a * r.up) : 0.0f;
  r.scale = r.bad ? __uint_as_float(0x7FC00000u) : a / 127.0f;
  return r;
}

__device__ __forceinline__ uint32_t quant4(const float* y, const RowScale& r) {
  uint32_t o = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // |y| <= a, so the product rounds to at most 127
    const int q = r.bad ? 0 : static_cast<int>(__builtin_rintf(y[i] * r.up * r.inv));
    o |= (static_cast<uint32_t>(q) & 0xFFu) << (8 * i);
  }
  return o;
}

// NORM false: the 8-bit form of x alone (y = x).
template <int TYPE, int NW, int C, bool NORM, bool NT>
__global__ __launch_bounds__(NW == 1 ? 256 : 64 * NW) void add_rmsnorm_kernel(
    int T, int H, float eps, const void* x, const void* res, const float* __restrict__ weight,
    void* sum, void* y, int8_t* __restrict__ yq, float* __restrict__ ys) {
  __shared__ float red_s[NW];
  __shared__ uint32_t red_m[NW];
  const int wave = uniform(threadIdx.x >> 6);
  const int group = static_cast<int>(workgroup());
  const int row = NW == 1 ? group * 4 + wave : group;
  if (row >= T) return;  // whole waves (NW = 1) or whole workgroups
  const int li = NW == 1 ? (threadIdx.x & 63) : threadIdx.x;
  const int chunks = H / 8;
  const size_t base = static_cast<size_t>(row) * chunks;
  float v[C][8], w[C][8];
  {
    Raw8<TYPE> a[C], b[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = li + i * 64 * NW;
      if (c < chunks) {
        a[i] = load8<TYPE, NT>(x, base + c);
        if (NORM && res) b[i] = load8<TYPE, NT>(res, base + c);
      }
    }
    if (NORM) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int c = li + i * 64 * NW;
        if (c < chunks) load_weight8(weight, c, w[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = li + i * 64 * NW;
      if (c < chunks) {
        unpack8<TYPE>(a[i], v[i]);
        if (NORM && res) {
          float u[8];
          unpack8<TYPE>(b[i], u);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] += u[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
      }
    }
  }
  uint32_t abits = 0;
  if (NORM) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(v[i][e], v[i][e], ss);
    if (sum) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int c = li + i * 64 * NW;
        if (c < chunks) store8<TYPE, NT>(sum, base + c, v[i]);
      }
    }
    ss = row_sum<NW>(ss, red_s, wave);
    const float rho = 1.0f / __builtin_sqrtf(ss / static_cast<float>(H) + eps);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = li + i * 64 * NW;
      if (c < chunks) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = v[i][e] * rho * w[i][e];
        if (y) store8<TYPE, NT>(y, base + c, v[i]);
      }
    }
    if (!yq) return;
  }
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) abits = max(abits, __float_as_uint(v[i][e]) & 0x7FFFFFFFu);
  const RowScale r = row_scale(row_max<NW>(abits, red_m, wave));
  if (li == 0) ys[row] = r.scale;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = li + i * 64 * NW;
    if (c < chunks) {
      uint2 o;
      o.x = quant4(v[i], r);
      o.y = quant4(v[i] + 4, r);
      reinterpret_cast<uint2*>(yq)[base + c] = o;
    }
  }
}

// Gradient.  Workgroups walk the rows with a fixed stride, so each lane keeps
// its columns' share of dw in registers over all its rows; at the end the
// waves of a workgroup that hold the same columns are added through LDS in a
// fixed tree and the workgroup writes one row of partial sums.  A second
// kernel adds those.  Nothing is added by atomics, so dw has the same bits in
// every run.
constexpr int kBwdWaves = 8;  // waves per workgroup where a wave holds a row

template <int NW>
constexpr int bwd_threads() { return NW == 1 ? 64 * kBwdWaves : 64 * NW; }

template <int TYPE, int NW, int C, bool NT>
__global__ __launch_bounds__(bwd_threads<NW>()) void add_rmsnorm_backward_kernel(
    int T, int H, float eps, const void* __restrict__ sum, const float* __restrict__ weight,
    const void* dy, const void* dsum, void* dx, float* __restrict__ part) {
  constexpr int RG = NW == 1 ? kBwdWaves : 1;  // rows a workgroup works on together
  constexpr int kWidth = 64 * C * 8;           // columns a wave covers (NW = 1)
  __shared__ float red[NW == 1 ? 1 : 4 * NW];
  __shared__ float fold[NW == 1 ? (kBwdWaves / 2) * kWidth : 1];
  const int wave = uniform(threadIdx.x >> 6);
  const int li = NW == 1 ? (threadIdx.x & 63) : threadIdx.x;
  const int chunks = H / 8;
  const float invH = 1.0f / static_cast<float>(H);
  float acc[C][8], w[C][8];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = li + i * 64 * NW;
    if (c < chunks) {
      load_weight8(weight, c, w[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[i][e] = 0.0f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[i][e] = 0.0f;
  }
  int parity = 0;
  const int first = NW == 1 ? static_cast<int>(blockIdx.x) * RG + wave : static_cast<int>(blockIdx.x);
  for (int row = first; row < T; row += static_cast<int>(gridDim.x) * RG) {
    const size_t base = static_cast<size_t>(row) * chunks;
    Raw8<TYPE> rs[C], rd[C], rr[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = li + i * 64 * NW;
      if (c < chunks) {
        rs[i] = load8<TYPE, NT>(sum, base + c);
        rd[i] = load8<TYPE, NT>(dy, base + c);
        if (dsum) rr[i] = load8<TYPE, NT>(dsum, base + c);
      } else {
#pragma unroll
        for (int q = 0; q < 8 / Elem<TYPE>::V; ++q) rs[i].q[q] = rd[i].q[q] = make_uint4(0, 0, 0, 0);
      }
    }
    float ss = 0.0f, gs = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float s[8], d[8];
      unpack8<TYPE>(rs[i], s);
      unpack8<TYPE>(rd[i], d);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss = __builtin_fmaf(s[e], s[e], ss);
        gs = __builtin_fmaf(d[e] * w[i][e], s[e], gs);
      }
    }
    ss = wave_sum(ss);
    gs = wave_sum(gs);
    if (NW > 1) {
      // two sets of words in turn: a set is rewritten two rows later, after
      // the barrier of the row between
      float* r = red + parity * 2 * NW;
      parity ^= 1;
      if ((threadIdx.x & 63) == 0) {
        r[wave] = ss;
        r[NW + wave] = gs;
      }
      __syncthreads();
      ss = gs = 0.0f;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        ss += r[i];
        gs += r[NW + i];
      }
    }
    const float rho = 1.0f / __builtin_sqrtf(ss * invH + eps);
    const float k = gs * invH * rho * rho;  // xh mean(g xh) = s rho k / rho
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = li + i * 64 * NW;
      if (c < chunks) {
        float s[8], d[8], o[8];
        unpack8<TYPE>(rs[i], s);
        unpack8<TYPE>(rd[i], d);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          o[e] = rho * (d[e] * w[i][e] - s[e] * k);
          acc[i][e] = __builtin_fmaf(d[e], s[e] * rho, acc[i][e]);
        }
        if (dsum) {
          float u[8];
          unpack8<TYPE>(rr[i], u);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] += u[e];
        }
        store8<TYPE, NT>(dx, base + c, o);
      }
    }
  }
  if (!part) return;
  if (NW == 1) {
#pragma unroll
    for (int half = kBwdWaves / 2; half >= 1; half /= 2) {
      if (wave >= half && wave < 2 * half) {
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            fold[((wave - half) * C * 8 + i * 8 + e) * 64 + li] = acc[i][e];
      }
      __syncthreads();
      if (wave < half) {
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[i][e] += fold[(wave * C * 8 + i * 8 + e) * 64 + li];
      }
      __syncthreads();
    }
    if (wave) return;
  }
  float4* out = reinterpret_cast<float4*>(part + static_cast<size_t>(blockIdx.x) * H);
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = li + i * 64 * NW;
    if (c < chunks) {
      out[2 * c] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
      out[2 * c + 1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
    }
  }
}

// dw: the sum of P rows of partial sums, sixteen waves per 64 columns (each
// every sixteenth row), joined through LDS.
__global__ __launch_bounds__(1024) void norm_dweight_kernel(int P, int H, const float* __restrict__ part,
                                                           float* __restrict__ dw) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int c = blockIdx.x * 64 + lane;
  float t = 0.0f;
  if (c < H) {
#pragma unroll 16
    for (int p = wave; p < P; p += 16) t += part[static_cast<size_t>(p) * H + c];
  }
  red[wave][lane] = t;
  __syncthreads();
  if (wave == 0 && c < H) {
    t = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += red[i][lane];
    dw[c] = t;
  }
}

int validate_norm(const moe_norm_dims* d) {
  if (!d) return MOE_EINVAL;
  if (d->T < 0 || d->T > (1 << 24)) return MOE_EINVAL;
  if (d->H <= 0 || d->H % 8 || d->H > kMaxNormH) return MOE_EINVAL;
  if (!elem_ok(d->type)) return MOE_EINVAL;
  if (!(d->eps >= 0.0f) || !(d->eps <= 3.402823466e38f)) return MOE_EINVAL;
  return MOE_OK;
}

// Waves per row: one where the row fits a wave (H <= 2048) and there are rows
// enough to fill the chip, else four (H <= 8192), else sixteen.  At 2048 x 2048
// the forward pass takes the same either way; the gradient of 333 x 2048 takes
// 10.1 us with one wave a row and 8.3 with four, of 4096 x 2048 17.1 with one.
int row_waves(int T, int H) {
  if (H <= 2048 && T >= 2048) return 1;
  return H <= 8192 ? 4 : 16;
}

// Rows that leave the L2s before anyone reads them again go past the caches
// (16384 x 4096 with 8 bits: 109 us -> 99; gradient of 16384 x 2048: 57 -> 53).
bool streamed(const moe_norm_dims& d) {
  return static_cast<size_t>(d.T) * d.H * elem_bytes(d.type) > kStreamStore;
}

template <int TYPE, int NW, int C, bool NORM>
void launch_norm(const moe_norm_dims& d, const void* x, const void* res, const float* weight,
                 void* sum, void* y, int8_t* yq, float* ys, hipStream_t stream) {
  const int rows = NW == 1 ? 4 : 1;
  const unsigned groups = static_cast<unsigned>((d.T + rows - 1) / rows);
  hipLaunchKernelGGL((streamed(d) ? add_rmsnorm_kernel<TYPE, NW, C, NORM, true>
                                  : add_rmsnorm_kernel<TYPE, NW, C, NORM, false>),
                     grid_of(groups),
                     dim3(NW == 1 ? 256 : 64 * NW), 0, stream, d.T, d.H, d.eps, x, res, weight, sum,
                     y, yq, ys);
}

template <int TYPE, bool NORM>
void launch_norm_type(const moe_norm_dims& d, const void* x, const void* res, const float* weight,
                      void* sum, void* y, int8_t* yq, float* ys, hipStream_t s) {
  const int nw = row_waves(d.T, d.H);
  const int c = (d.H / 8 + 64 * nw - 1) / (64 * nw);
#define MOE_NORM(NW, C) launch_norm<TYPE, NW, C, NORM>(d, x, res, weight, sum, y, yq, ys, s)
  if (nw == 1) {
    c == 1 ? MOE_NORM(1, 1) : c == 2 ? MOE_NORM(1, 2) : c == 3 ? MOE_NORM(1, 3) : MOE_NORM(1, 4);
  } else if (nw == 4) {
    c == 1 ? MOE_NORM(4, 1) : c == 2 ? MOE_NORM(4, 2) : c == 3 ? MOE_NORM(4, 3) : MOE_NORM(4, 4);
  } else {
    MOE_NORM(16, 2);
  }
#undef MOE_NORM
}

template <bool NORM>
hipError_t launch_norm_any(const moe_norm_dims& d, const void* x, const void* res,
                           const float* weight, void* sum, void* y, int8_t* yq, float* ys,
                           hipStream_t s) {
  switch (d.type) {
    case MOE_ELEM_F32: launch_norm_type<MOE_ELEM_F32, NORM>(d, x, res, weight, sum, y, yq, ys, s); break;
    case MOE_ELEM_BF16: launch_norm_type<MOE_ELEM_BF16, NORM>(d, x, res, weight, sum, y, yq, ys, s); break;
    default: launch_norm_type<MOE_ELEM_F16, NORM>(d, x, res, weight, sum, y, yq, ys, s); break;
  }
  return hipGetLastError();
}

// Waves per row of the gradient kernel: eight rows or fewer also go one wave
// each, in one workgroup, whose sums are then dw already.
int bwd_waves(int T, int H) { return H <= 2048 && T <= kBwdWaves ? 1 : row_waves(T, H); }

// Workgroups of the gradient kernel: one per CU of eight waves, two of four
// waves once there are rows for both, one of sixteen.  More of them hide more
// latency but leave more partial sums to add.  Measured, us: 16384 x 2048 256
// groups 50.7, 512 53; 333 x 2048 256 8.3, 512 9.5; 2000 x 2048 256 16.2, 512
// 12.8, 1024 14.4; 2048 x 16384 128 69, 256 56, 512 64.
int bwd_groups(const moe_norm_dims& d) {
  const int nw = bwd_waves(d.T, d.H);
  const int rows = nw == 1 ? kBwdWaves : 1;
  const int cap = nw == 4 && d.T >= 1024 ? 512 : 256;
  const int need = (d.T + rows - 1) / rows;
  return need < cap ? need : cap;
}

template <int TYPE>
void launch_bwd_type(const moe_norm_dims& d, const void* sum, const float* weight, const void* dy,
                     const void* dsum, void* dx, float* part, hipStream_t s) {
  const int nw = bwd_waves(d.T, d.H);
  const int c = (d.H / 8 + 64 * nw - 1) / (64 * nw);
  const dim3 grid(static_cast<unsigned>(bwd_groups(d)));
#define MOE_BWD(NW, C)                                                                           \
  hipLaunchKernelGGL((streamed(d) ? add_rmsnorm_backward_kernel<TYPE, NW, C, true>               \
                                  : add_rmsnorm_backward_kernel<TYPE, NW, C, false>),            \
                     grid, dim3(bwd_threads<NW>()), 0, s, d.T, d.H, d.eps, sum, weight, dy, dsum, dx, part)
  if (nw == 1) {
    if (c == 1) MOE_BWD(1, 1); else if (c == 2) MOE_BWD(1, 2); else if (c == 3) MOE_BWD(1, 3); else MOE_BWD(1, 4);
  } else if (nw == 4) {
    if (c == 1) MOE_BWD(4, 1); else if (c == 2) MOE_BWD(4, 2); else if (c == 3) MOE_BWD(4, 3); else MOE_BWD(4, 4);
  } else {
    MOE_BWD(16, 2);
  }
#undef MOE_BWD
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_add_rmsnorm(const moe_norm_dims* d, const void* x, const void* res, const float* weight,
                    void* sum, void* y, int8_t* yq, float* ys, void* stream) {
  int rc = validate_norm(d);
  if (rc || d->T == 0) return rc;
  if (!x || !weight || (!y && !yq) || (yq == nullptr) != (ys == nullptr) || (y && y == sum))
    return MOE_EINVAL;
  if (!aligned(x, 16) || !aligned(res, 16) || !aligned(weight, 16) || !aligned(sum, 16) ||
      !aligned(y, 16) || !aligned(yq, 16) || !aligned(ys, 4))
    return MOE_EALIGN;
  if ((rc = check_device())) return rc;
  (void)hipGetLastError();
  return launched(launch_norm_any<true>(*d, x, res, weight, sum, y, yq, ys,
                                        static_cast<hipStream_t>(stream)));
}

int moe_q8_quantize(const moe_norm_dims* d, const void* x, int8_t* xq, float* xs, void* stream) {
  int rc = validate_norm(d);
  if (rc || d->T == 0) return rc;
  if (!x || !xq || !xs) return MOE_EINVAL;
  if (!aligned(x, 16) || !aligned(xq, 16) || !aligned(xs, 4)) return MOE_EALIGN;
  if ((rc = check_device())) return rc;
  (void)hipGetLastError();
  return launched(launch_norm_any<false>(*d, x, nullptr, nullptr, nullptr, nullptr, xq, xs,
                                         static_cast<hipStream_t>(stream)));
}

size_t moe_add_rmsnorm_backward_ws_bytes(const moe_norm_dims* d) {
  if (validate_norm(d)) return 0;
  return static_cast<size_t>(bwd_groups(*d)) * d->H * sizeof(float);
}

int moe_add_rmsnorm_backward(const moe_norm_dims* d, const void* sum, const float* weight,
                             const void* dy, const void* dsum, void* dx, float* dweight, void* ws,
                             size_t ws_bytes, void* stream) {
  int rc = validate_norm(d);
  if (rc) return rc;
  const size_t need = moe_add_rmsnorm_backward_ws_bytes(d);
  if (d->T > 0 && (!sum || !weight || !dy || !dx || (dweight && !ws))) return MOE_EINVAL;
  if (!aligned(sum, 16) || !aligned(weight, 16) || !aligned(dy, 16) || !aligned(dsum, 16) ||
      !aligned(dx, 16) || !aligned(dweight, 4) || !aligned(ws, 16))
    return MOE_EALIGN;
  if (dweight && ws_bytes < need) return MOE_EWS;
  if (d->T == 0 && !dweight) return MOE_OK;
  if ((rc = check_device())) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  // one workgroup's partial sums are the sums (written in 16-byte pieces)
  const bool direct = dweight && bwd_groups(*d) == 1 && aligned(dweight, 16);
  float* part = direct ? dweight : dweight ? static_cast<float*>(ws) : nullptr;
  (void)hipGetLastError();
  if (d->T > 0) {
    switch (d->type) {
      case MOE_ELEM_F32: launch_bwd_type<MOE_ELEM_F32>(*d, sum, weight, dy, dsum, dx, part, s); break;
      case MOE_ELEM_BF16: launch_bwd_type<MOE_ELEM_BF16>(*d, sum, weight, dy, dsum, dx, part, s); break;
      default: launch_bwd_type<MOE_ELEM_F16>(*d, sum, weight, dy, dsum, dx, part, s); break;
    }
    if ((rc = launched(hipGetLastError()))) return rc;
  }
  if (dweight && !direct) {
    hipLaunchKernelGGL(norm_dweight_kernel, dim3(static_cast<unsigned>((d->H + 63) / 64)), dim3(1024), 0,
                       s, bwd_groups(*d), d->H, part, dweight);
    if ((rc = launched(hipGetLastError()))) return rc;
  }
  return MOE_OK;
}

}  // extern "C"
