// Token rows sorted by expert and back, with the routing weights applied, and
// the gradients of both directions (include/moe_block.h).
//
//   dispatch            rows[pos(t,j)] = x[t], rows[Tk+t] = x[t]
//   its gradient        dx[t] = sum_j drows[pos(t,j)] + drows[Tk+t]
//   combine             y[t] = sum_j w(t,j) rows[pos(t,j)] + rows[Tk+t]
//   its gradient        drows[pos(t,j)] = w(t,j) dy[t], drows[Tk+t] = dy[t],
//                       dw(t,j) = <dy[t], rows[pos(t,j)]>
//
// All of it is bound by memory: at most two operations an element moved.  The
// work is cut by token, never by row of the sorted order: a token's row (or
// its gradient) is then read or written once and its k+1 sorted rows are each
// touched by one workgroup, so there is nothing to add up across workgroups,
// no atomics, and every sorted row is still one contiguous run of whole
// 16-byte accesses.  Slot positions and weights are workgroup-uniform.  Sorted
// rows of large batches are streamed past the caches (kStreamStore, kStreamLoad
// in block.h).  Measured at 8192 tokens of 2048 bfloat16, 8 + 1 rows a token
// (335 MB moved, 604 MB for the combine's gradient, which does not read the
// shared rows), us plain -> streamed: dispatch 68 -> 53, combine 65 -> 57, its
// gradient 123 -> 108, the dispatch's 65 -> 57: 6.3, 5.9, 5.6 and 5.9 TB/s, about
// the rate of a plain streaming read (5.85).
#include "block.h"

namespace moe {
namespace {

constexpr int kRowThreads = 256;
constexpr int kGroup = 8;  // slots whose loads are in flight together

// One token's positions of slots j0 .. j0+7, clamped where out of range.
struct Slots {
  int pos[kGroup];
  bool ok[kGroup];
};
__device__ __forceinline__ Slots load_slots(const int32_t* __restrict__ slot_pos, int t, int k, int S,
                                            int j0, uint32_t* status) {
  Slots s;
#pragma unroll
  for (int u = 0; u < kGroup; ++u) {
    const int p = slot_pos[static_cast<size_t>(t) * k + min(j0 + u, k - 1)];
    s.ok[u] = j0 + u < k && p >= 0 && p < S;
    s.pos[u] = (p >= 0 && p < S) ? p : 0;
    if (j0 + u < k && !s.ok[u]) status_set(status, MOE_STATUS_BAD_INDEX);
  }
  return s;
}

// chunks: 16-byte pieces of a row.  One token and 256 pieces per workgroup.
template <bool NT>
__global__ __launch_bounds__(kRowThreads) void dispatch_rows_kernel(
    int T, int k, int n_shared, int chunks, const int32_t* __restrict__ slot_pos,
    const uint4* __restrict__ x, uint4* __restrict__ rows, uint32_t* __restrict__ status) {
  const int t = blockIdx.x;
  const int c = static_cast<int>(blockIdx.y) * kRowThreads + threadIdx.x;
  if (c >= chunks) return;
  const int S = T * k;
  const uint4 v = x[static_cast<size_t>(t) * chunks + c];
  for (int j0 = 0; j0 < k; j0 += kGroup) {
    const Slots s = load_slots(slot_pos, t, k, S, j0, status);
#pragma unroll
    for (int u = 0; u < kGroup; ++u)
      if (s.ok[u]) store16<NT>(rows + static_cast<size_t>(s.pos[u]) * chunks + c, v);
  }
  if (n_shared) store16<NT>(rows + (static_cast<size_t>(S) + t) * chunks + c, v);
}

// WEIGHTED: the combine; else the gradient of the dispatch (weights of one).
template <int TYPE, bool WEIGHTED, bool NT>
__global__ __launch_bounds__(kRowThreads) void combine_rows_kernel(
    int T, int k, int n_shared, int chunks, const float* __restrict__ topk_w,
    const int32_t* __restrict__ slot_pos, const uint4* __restrict__ rows, uint4* __restrict__ y,
    uint32_t* __restrict__ status) {
  constexpr int V = Elem<TYPE>::V;
  const int t = blockIdx.x;
  const int c = static_cast<int>(blockIdx.y) * kRowThreads + threadIdx.x;
  if (c >= chunks) return;
  const int S = T * k;
  const uint4 vsh = load16<NT>(rows + static_cast<size_t>(n_shared ? S + t : 0) * chunks + c);
  float acc[V];
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.0f;
  for (int j0 = 0; j0 < k; j0 += kGroup) {
    const Slots s = load_slots(slot_pos, t, k, S, j0, status);
    uint4 v[kGroup];
    float w[kGroup];
#pragma unroll
    for (int u = 0; u < kGroup; ++u) {
      v[u] = load16<NT>(rows + static_cast<size_t>(s.pos[u]) * chunks + c);
      w[u] = WEIGHTED ? topk_w[static_cast<size_t>(t) * k + min(j0 + u, k - 1)] : 1.0f;
    }
#pragma unroll
    for (int u = 0; u < kGroup; ++u) {
      if (!s.ok[u]) continue;
      float r[V];
      Elem<TYPE>::unpack(v[u], r);
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] = __builtin_fmaf(w[u], r[e], acc[e]);
    }
  }
  if (n_shared) {
    float r[V];
    Elem<TYPE>::unpack(vsh, r);
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] += r[e];
  }
  y[static_cast<size_t>(t) * chunks + c] = Elem<TYPE>::pack(acc);
}

// One token per workgroup: dy's pieces are scaled into the k+1 rows, and the k
// dot products are summed over the workgroup (lanes, then the four waves).
template <int TYPE, bool NTL, bool NTS>
__global__ __launch_bounds__(kRowThreads) void combine_rows_backward_kernel(
    int T, int k, int n_shared, int chunks, const float* __restrict__ topk_w,
    const int32_t* __restrict__ slot_pos, const uint4* __restrict__ dy, const uint4* rows,
    uint4* drows, float* __restrict__ dw, uint32_t* __restrict__ status) {
  constexpr int V = Elem<TYPE>::V;
  __shared__ float red[kRowThreads / 64][kGroup];
  const int t = blockIdx.x;
  const int S = T * k;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  for (int j0 = 0; j0 < k; j0 += kGroup) {
    const Slots s = load_slots(slot_pos, t, k, S, j0, threadIdx.x == 0 ? status : nullptr);
    float w[kGroup], dot[kGroup];
#pragma unroll
    for (int u = 0; u < kGroup; ++u) {
      w[u] = topk_w[static_cast<size_t>(t) * k + min(j0 + u, k - 1)];
      dot[u] = 0.0f;
    }
    for (int c = threadIdx.x; c < chunks; c += kRowThreads) {
      const uint4 draw = dy[static_cast<size_t>(t) * chunks + c];
      uint4 v[kGroup];
      if (dw) {
#pragma unroll
        for (int u = 0; u < kGroup; ++u) v[u] = load16<NTL>(rows + static_cast<size_t>(s.pos[u]) * chunks + c);
      }
      float d[V];
      Elem<TYPE>::unpack(draw, d);
      if (j0 == 0 && n_shared) store16<NTS>(drows + (static_cast<size_t>(S) + t) * chunks + c, draw);
#pragma unroll
      for (int u = 0; u < kGroup; ++u) {
        if (!s.ok[u]) continue;
        float o[V];
        if (dw) {
          float r[V];
          Elem<TYPE>::unpack(v[u], r);
#pragma unroll
          for (int e = 0; e < V; ++e) dot[u] = __builtin_fmaf(d[e], r[e], dot[u]);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = w[u] * d[e];
        store16<NTS>(drows + static_cast<size_t>(s.pos[u]) * chunks + c, Elem<TYPE>::pack(o));
      }
    }
    if (dw) {
#pragma unroll
      for (int u = 0; u < kGroup; ++u) {
        const float x = wave_sum(dot[u]);
        if (lane == 0) red[wave][u] = x;
      }
      __syncthreads();
      if (threadIdx.x < kGroup && j0 + static_cast<int>(threadIdx.x) < k) {
        float x = 0.0f;
#pragma unroll
        for (int i = 0; i < kRowThreads / 64; ++i) x += red[i][threadIdx.x];
        dw[static_cast<size_t>(t) * k + j0 + threadIdx.x] = x;
      }
      __syncthreads();  // red is written again in the next group of slots
    }
  }
}

int validate_rows(const moe_dims* d, int32_t type, const moe_route_out* r, bool weighted) {
  int rc = validate_dims(d);
  if (rc) return rc;
  if (!elem_ok(type)) return MOE_EINVAL;
  if (d->T == 0) return MOE_OK;
  if (!r || !r->slot_pos || !r->status || (weighted && !r->topk_w)) return MOE_EINVAL;
  if (!aligned(r->slot_pos, 4) || !aligned(r->status, 4) || (weighted && !aligned(r->topk_w, 4)))
    return MOE_EALIGN;
  return MOE_OK;
}

int row_chunks(const moe_dims& d, int type) { return d.H * elem_bytes(type) / 16; }

// Bytes of the sorted rows.
size_t rows_bytes(const moe_dims& d, int type) {
  return static_cast<size_t>(d.T) * (d.k + d.n_shared) * d.H * elem_bytes(type);
}

template <bool WEIGHTED>
int combine_any(const moe_dims& d, int type, const void* rows, const moe_route_out* r, void* y,
                void* stream) {
  const int chunks = row_chunks(d, type);
  const dim3 grid(static_cast<unsigned>(d.T), static_cast<unsigned>((chunks + kRowThreads - 1) / kRowThreads));
  hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  const bool stream_rows = rows_bytes(d, type) > kStreamLoad;
#define MOE_COMBINE(TYPE)                                                                        \
  hipLaunchKernelGGL((stream_rows ? combine_rows_kernel<TYPE, WEIGHTED, true>                    \
                                  : combine_rows_kernel<TYPE, WEIGHTED, false>),                 \
                     grid, dim3(kRowThreads), 0, s, d.T, d.k, d.n_shared, chunks, r->topk_w,     \
                     r->slot_pos, static_cast<const uint4*>(rows), static_cast<uint4*>(y), r->status)
  switch (type) {
    case MOE_ELEM_F32: MOE_COMBINE(MOE_ELEM_F32); break;
    case MOE_ELEM_BF16: MOE_COMBINE(MOE_ELEM_BF16); break;
    default: MOE_COMBINE(MOE_ELEM_F16); break;
  }
#undef MOE_COMBINE
  return launched(hipGetLastError());
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_dispatch_rows(const moe_dims* d, int32_t type, const void* x, const moe_route_out* r,
                      void* rows, void* stream) {
  int rc = validate_rows(d, type, r, false);
  if (rc || d->T == 0) return rc;
  if (!x || !rows) return MOE_EINVAL;
  if (!aligned(x, 16) || !aligned(rows, 16)) return MOE_EALIGN;
  if ((rc = check_device())) return rc;
  const int chunks = row_chunks(*d, type);
  const dim3 grid(static_cast<unsigned>(d->T), static_cast<unsigned>((chunks + kRowThreads - 1) / kRowThreads));
  (void)hipGetLastError();
  hipLaunchKernelGGL((rows_bytes(*d, type) > kStreamStore ? dispatch_rows_kernel<true>
                                                          : dispatch_rows_kernel<false>),
                     grid, dim3(kRowThreads), 0, static_cast<hipStream_t>(stream), d->T, d->k, d->n_shared, chunks, r->slot_pos,
                     static_cast<const uint4*>(x), static_cast<uint4*>(rows), r->status);
  return launched(hipGetLastError());
}

int moe_dispatch_rows_backward(const moe_dims* d, int32_t type, const void* drows,
                               const moe_route_out* r, void* dx, void* stream) {
  int rc = validate_rows(d, type, r, false);
  if (rc || d->T == 0) return rc;
  if (!drows || !dx) return MOE_EINVAL;
  if (!aligned(drows, 16) || !aligned(dx, 16)) return MOE_EALIGN;
  if ((rc = check_device())) return rc;
  return combine_any<false>(*d, type, drows, r, dx, stream);
}

int moe_combine_rows(const moe_dims* d, int32_t type, const void* rows, const moe_route_out* r,
                     void* y, void* stream) {
  int rc = validate_rows(d, type, r, true);
  if (rc || d->T == 0) return rc;
  if (!rows || !y) return MOE_EINVAL;
  if (!aligned(rows, 16) || !aligned(y, 16)) return MOE_EALIGN;
  if ((rc = check_device())) return rc;
  return combine_any<true>(*d, type, rows, r, y, stream);
}

int moe_combine_rows_backward(const moe_dims* d, int32_t type, const void* dy, const void* rows,
                              const moe_route_out* r, void* drows, float* dtopk_w, void* stream) {
  int rc = validate_rows(d, type, r, true);
  if (rc || d->T == 0) return rc;
  if (!dy || !drows || (dtopk_w && !rows)) return MOE_EINVAL;
  if (!aligned(dy, 16) || !aligned(rows, 16) || !aligned(drows, 16) || !aligned(dtopk_w, 4))
    return MOE_EALIGN;
  if ((rc = check_device())) return rc;
  const int chunks = row_chunks(*d, type);
  const dim3 grid(static_cast<unsigned>(d->T));
  hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  const size_t bytes = rows_bytes(*d, type);
#define MOE_COMBINE_BWD(TYPE)                                                                    \
  hipLaunchKernelGGL((bytes > kStreamLoad    ? combine_rows_backward_kernel<TYPE, true, true>    \
                      : bytes > kStreamStore ? combine_rows_backward_kernel<TYPE, false, true>   \
                                             : combine_rows_backward_kernel<TYPE, false, false>), \
                     grid, dim3(kRowThreads), 0, s, d->T, d->k, d->n_shared, chunks, r->topk_w,  \
                     r->slot_pos, static_cast<const uint4*>(dy), static_cast<const uint4*>(rows), \
                     static_cast<uint4*>(drows), dtopk_w, r->status)
  switch (type) {
    case MOE_ELEM_F32: MOE_COMBINE_BWD(MOE_ELEM_F32); break;
    case MOE_ELEM_BF16: MOE_COMBINE_BWD(MOE_ELEM_BF16); break;
    default: MOE_COMBINE_BWD(MOE_ELEM_F16); break;
  }
#undef MOE_COMBINE_BWD
  return launched(hipGetLastError());
}

}  // extern "C"
