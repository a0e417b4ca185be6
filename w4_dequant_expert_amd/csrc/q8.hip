// Matrix products in 8-bit integers with a scale for each token and each
// output channel, dense and grouped by expert (include/moe_block.h):
//   out[m][n] = xs[m] ws[n] sum_k xq[m][k] wq[n][k]
// The sum is exact in int32 (|xq wq| <= 2^14 and K <= 2^16 give at most 2^30),
// so the order of its terms is free: kernels may split K over waves, or read
// the inputs in any order the two operands share, and every kernel here gives
// the same bits.
//
// Two kernels, on v_mfma_i32_16x16x64_i8 (weights as the first operand, so a
// lane ends with four neighbouring output channels of one row):
//   q8_stream_kernel: few rows.  Bound by reading the weights once; every wave
//     streams its share of K straight from memory into the matrix operands,
//     with no LDS and no barrier until the waves' sums are added.
//   q8_tile_kernel: many rows.  Bound by the int8 matrix rate; tiles of both
//     operands go through LDS in steps of 128 inputs.
#include "block.h"

namespace moe {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

struct Q8Args {
  const int8_t* x;
  const float* xs;
  const int8_t* w;          // dense: the matrix; grouped: the routed bank
  const float* ws;
  const int8_t* w_shared;
  const float* ws_shared;
  void* out;
  int rows;                 // rows of the output
  int N, K;                 // rows and inputs of one weight matrix
  int type;                 // output element
  // grouped products only
  const int32_t* blocks;
  const int32_t* n_blocks;
  const int32_t* sorted_slot;
  uint32_t* status;
  int max_blocks, E, T, k, n_shared;
};

// A block of output rows that share one weight matrix.
struct Q8Block {
  const int8_t* w;
  const float* ws;
  int row0, rows;
};

// Block b of the map; false (with the status bit) for an entry out of range.
__device__ __forceinline__ bool q8_block(const Q8Args& a, int b, Q8Block& o) {
  const int4 e = reinterpret_cast<const int4*>(a.blocks)[b];
  const int g = uniform(e.x);
  o.row0 = uniform(e.y);
  o.rows = uniform(e.z);
  const bool shared = g == a.E;
  if (g < 0 || g > a.E || (shared && !a.n_shared) || o.row0 < 0 || o.rows <= 0 ||
      o.rows > a.rows - o.row0) {
    if (threadIdx.x == 0) status_set(a.status, MOE_STATUS_BAD_INDEX);
    return false;
  }
  o.w = shared ? a.w_shared : a.w + static_cast<size_t>(g) * a.N * a.K;
  o.ws = shared ? a.ws_shared : a.ws + static_cast<size_t>(g) * a.N;
  return true;
}

// The input row of an output row: its token where GATHER (-1 for a table entry
// out of range), else the row itself.
template <bool GATHER>
__device__ __forceinline__ int q8_source(const Q8Args& a, int row) {
  if (!GATHER) return row;
  const int S = a.T * a.k;
  if (row >= S) return row - S;
  const int slot = a.sorted_slot[row];
  return (slot >= 0 && slot < S) ? slot / a.k : -1;
}

// The weight row of virtual column v.  SwiGLU pairs sixteen gate rows with
// their sixteen up rows, so that one wave holds both in the same lanes.
template <bool SWIGLU>
__device__ __forceinline__ int q8_weight_row(int v, int N) {
  if (!SWIGLU) return min(v, N - 1);
  const int half = N / 2, r = (v / 32) * 16 + (v & 15);
  return (v & 16) ? min(half + r, N - 1) : min(r, half - 1);
}

__device__ __forceinline__ void store4(void* out, size_t at, int type, const float (&v)[4]) {
  if (type == MOE_ELEM_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    const uint2 o = type == MOE_ELEM_BF16 ? make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]))
                                          : make_uint2(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]));
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = o;
  }
}

// Four neighbouring outputs (columns v .. v+3) of one row from the integer sums.
__device__ __forceinline__ void q8_store(const Q8Args& a, const float* __restrict__ ws, size_t row, int v,
                                         float xs, i32x4 acc) {
  if (v >= a.N) return;
  const float4 s = *reinterpret_cast<const float4*>(ws + v);
  const float o[4] = {static_cast<float>(acc[0]) * xs * s.x, static_cast<float>(acc[1]) * xs * s.y,
                      static_cast<float>(acc[2]) * xs * s.z, static_cast<float>(acc[3]) * xs * s.w};
  store4(a.out, row * a.N + v, a.type, o);
}

// silu(g) u for four neighbouring hidden columns c .. c+3 of one row.
__device__ __forceinline__ void q8_store_swiglu(const Q8Args& a, const float* __restrict__ ws, size_t row,
                                                int c, float xs, i32x4 g, i32x4 u) {
  const int half = a.N / 2;
  if (c >= half) return;
  const float4 sg = *reinterpret_cast<const float4*>(ws + c);
  const float4 su = *reinterpret_cast<const float4*>(ws + half + c);
  const float fg[4] = {sg.x, sg.y, sg.z, sg.w}, fu[4] = {su.x, su.y, su.z, su.w};
  float o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float gv = static_cast<float>(g[i]) * xs * fg[i];
    const float uv = static_cast<float>(u[i]) * xs * fu[i];
    o[i] = gv * __builtin_amdgcn_rcpf(1.0f + __expf(-gv)) * uv;
  }
  store4(a.out, row * half + c, MOE_ELEM_BF16, o);
}

__device__ __forceinline__ i32x4 mfma(uint4 a, uint4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c,
                                               0, 0, 0);
}

// ---------------------------------------------------------------------------
// Few rows.  A workgroup of four waves owns CT*16 columns of a block and takes
// its rows MT*16 at a time; wave w multiplies every fourth unit of 128 inputs.
// Within a unit lane group q = lane/16 holds inputs 32q .. 32q+31 of its
// weight row and of its token row (two 16-byte loads each, so a row's 128
// bytes are read by neighbouring lanes at once); both operands agree on that
// order, which is all the exact sum needs.  The four waves' sums meet in LDS.
// ---------------------------------------------------------------------------
template <int CT, int MT, bool GROUPED, bool GATHER, bool SWIGLU>
__global__ __launch_bounds__(256) void q8_stream_kernel(Q8Args a) {
  static_assert(!SWIGLU || CT % 2 == 0, "gate and up columns come in pairs");
  __shared__ i32x4 part[4][MT * CT][64];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int q = lane >> 4, r16 = lane & 15;
  const int nt = (a.N + CT * 16 - 1) / (CT * 16);
  const int b = blockIdx.x / nt;
  const int v0 = (blockIdx.x % nt) * CT * 16;
  Q8Block blk;
  if (GROUPED) {
    if (b >= min(*a.n_blocks, a.max_blocks) || !q8_block(a, b, blk)) return;
  } else {
    blk.w = a.w;
    blk.ws = a.ws;
    blk.row0 = 0;
    blk.rows = a.rows;
  }
  const int8_t* wp[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c)
    wp[c] = blk.w + static_cast<size_t>(q8_weight_row<SWIGLU>(v0 + c * 16 + r16, a.N)) * a.K;
  const int units = a.K / 128;  // whole units; K mod 128 = 64 leaves half of one
  for (int m0 = 0; m0 < blk.rows; m0 += MT * 16) {
    const int8_t* xp[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int src = q8_source<GATHER>(a, blk.row0 + min(m0 + m * 16 + r16, blk.rows - 1));
      xp[m] = a.x + static_cast<size_t>(max(src, 0)) * a.K;
    }
    i32x4 acc[MT][CT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int c = 0; c < CT; ++c) acc[m][c] = i32x4{0, 0, 0, 0};
    for (int u = wave; u < units; u += 4) {
      const int at = u * 128 + q * 32;
      uint4 wv[CT][2], xv[MT][2];
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        wv[c][0] = *reinterpret_cast<const uint4*>(wp[c] + at);
        wv[c][1] = *reinterpret_cast<const uint4*>(wp[c] + at + 16);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        xv[m][0] = *reinterpret_cast<const uint4*>(xp[m] + at);
        xv[m][1] = *reinterpret_cast<const uint4*>(xp[m] + at + 16);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int c = 0; c < CT; ++c) acc[m][c] = mfma(wv[c][h], xv[m][h], acc[m][c]);
    }
    if ((a.K & 64) && wave == (units & 3)) {
      const int at = units * 128 + q * 16;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const uint4 xv = *reinterpret_cast<const uint4*>(xp[m] + at);
#pragma unroll
        for (int c = 0; c < CT; ++c)
          acc[m][c] = mfma(*reinterpret_cast<const uint4*>(wp[c] + at), xv, acc[m][c]);
      }
    }
    if (m0) __syncthreads();  // the sums of the rows before have been read
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int c = 0; c < CT; ++c) part[wave][m * CT + c][lane] = acc[m][c];
    __syncthreads();
    auto total = [&](int i) {
      return part[0][i][lane] + part[1][i][lane] + part[2][i][lane] + part[3][i][lane];
    };
    constexpr int STEP = SWIGLU ? 2 : 1;
    for (int i = wave * STEP; i < MT * CT; i += 4 * STEP) {
      const int m = m0 + (i / CT) * 16 + r16;
      if (m >= blk.rows) continue;
      const int row = blk.row0 + m;
      const int src = q8_source<GATHER>(a, row);
      if (src < 0) {
        status_set(a.status, MOE_STATUS_BAD_INDEX);
        continue;
      }
      const float xs = a.xs[src];
      const int v = v0 + (i % CT) * 16;
      if (SWIGLU)
        q8_store_swiglu(a, blk.ws, row, v / 2 + 4 * q, xs, total(i), total(i + 1));
      else
        q8_store(a, blk.ws, row, v + 4 * q, xs, total(i));
    }
  }
}

// ---------------------------------------------------------------------------
// Many rows.  WM x WN waves own a tile of up to WM*MT*16 rows and WN*NT*16
// columns; a wave multiplies mt (1..MT, from the block's rows) times NT tiles
// of 16 x 16.  Both operands are copied straight from memory into LDS in steps
// of 128 inputs, into two buffers in turn: the copies of step s+1 are in
// flight while step s is multiplied.  A staged row is 128 bytes with its
// 16-byte pieces XORed by the row (piece c of row r at c ^ (r mod 8)), so the
// sixteen rows of an operand fragment spread over all banks; the copy puts
// lane l's 16 bytes at byte 16 l, so the permutation is made by the address
// each lane reads from.  Rows past the block repeat its last row and columns
// past N the last column; they only reach outputs that are not stored.
//
// Tiles are dealt to the chip's eight XCDs (workgroup i runs on XCD i mod 8)
// in contiguous runs, each run going through groups of four row blocks column
// by column, so that the tiles an XCD works on together share rows and columns
// in its own L2.
// ---------------------------------------------------------------------------
constexpr int kStep = 128;

// This wave's copies have landed and every wave is here (one statement with a
// memory clobber: no LDS access moves across it).
__device__ __forceinline__ void copies_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// What a wave of a tile keeps over the steps.
template <int WCOPY, int XCOPY>
struct TileWave {
  const int8_t* wp[WCOPY];  // this lane's weight row in each of the wave's copies
  const int8_t* xp[XCOPY];  // and its token row
  int xcopies;              // copies of token rows the workgroup makes
  int piece;                // the bytes of a step this lane copies
  int wave, wm, wn, lane;
};

// One pass over K for M tiles of rows per wave, and their outputs.
template <int M, int WM, int WN, int NT, int WCOPY, int XCOPY, bool GATHER, bool SWIGLU>
__device__ __forceinline__ void q8_tile_rows(const Q8Args& a, const Q8Block& blk, int m0, int v0,
                                             const TileWave<WCOPY, XCOPY>& t, uint8_t* buf0,
                                             uint8_t* buf1) {
  constexpr int WAVES = WM * WN, BN = WN * NT * 16;
  const int nk = (a.K + kStep - 1) / kStep;
  const int r16 = t.lane & 15, q = t.lane >> 4;
  // byte of this lane's fragment piece within a 16-row tile: inputs 0..63 and 64..127 of a step
  const int f0 = r16 * kStep + ((q ^ (r16 & 7)) << 4);
  const int f1 = r16 * kStep + (((4 + q) ^ (r16 & 7)) << 4);
  i32x4 acc[M][NT];
#pragma unroll
  for (int i = 0; i < M; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  auto copy = [&](int s, uint8_t* buf) {
    // the last step may hold 64 inputs: its second half repeats the first
    // (read into LDS, never multiplied)
    const int at = s * kStep + t.piece;
    const int k0 = at < a.K ? at : at - 64;
#pragma unroll
    for (int i = 0; i < WCOPY; ++i)
      __builtin_amdgcn_global_load_lds(t.wp[i] + k0, buf + (i * WAVES + t.wave) * 1024, 16, 0, 0);
#pragma unroll
    for (int i = 0; i < XCOPY; ++i)
      if (i * WAVES + t.wave < t.xcopies)
        __builtin_amdgcn_global_load_lds(t.xp[i] + k0, buf + BN * kStep + (i * WAVES + t.wave) * 1024, 16, 0,
                                         0);
  };
  auto half = [&](const uint8_t* buf, int f) {
    uint4 wf[NT], xf[M];
#pragma unroll
    for (int j = 0; j < NT; ++j)
      wf[j] = *reinterpret_cast<const uint4*>(buf + (t.wn * NT + j) * 16 * kStep + f);
#pragma unroll
    for (int i = 0; i < M; ++i)
      xf[i] = *reinterpret_cast<const uint4*>(buf + (BN + (t.wm * M + i) * 16) * kStep + f);
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = mfma(wf[j], xf[i], acc[i][j]);
  };
  auto step = [&](int s, uint8_t* cur, uint8_t* next) {
    copies_barrier();  // step s is in LDS; nobody reads `next` any more
    __builtin_amdgcn_sched_barrier(0);
    if (s + 1 < nk) copy(s + 1, next);
    __builtin_amdgcn_sched_barrier(0);
    half(cur, f0);
    if (s * kStep + 64 < a.K) half(cur, f1);
    __builtin_amdgcn_sched_barrier(0);
  };
  copy(0, buf0);
  for (int s = 0; s < nk; s += 2) {
    step(s, buf0, buf1);
    if (s + 1 < nk) step(s + 1, buf1, buf0);
  }
#pragma unroll
  for (int i = 0; i < M; ++i) {
    const int m = m0 + (t.wm * M + i) * 16 + r16;
    if (m >= blk.rows) continue;
    const int row = blk.row0 + m;
    const int src = q8_source<GATHER>(a, row);
    if (src < 0) {
      status_set(a.status, MOE_STATUS_BAD_INDEX);
      continue;
    }
    const float xs = a.xs[src];
#pragma unroll
    for (int j = 0; j < NT; j += SWIGLU ? 2 : 1) {
      const int v = v0 + (t.wn * NT + j) * 16;
      if (SWIGLU)
        q8_store_swiglu(a, blk.ws, row, v / 2 + 4 * q, xs, acc[i][j], acc[i][j + (SWIGLU ? 1 : 0)]);
      else
        q8_store(a, blk.ws, row, v + 4 * q, xs, acc[i][j]);
    }
  }
}

// q8_tile_rows for mt (1..M) tiles of rows.
template <int M, int WM, int WN, int NT, int WCOPY, int XCOPY, bool GATHER, bool SWIGLU>
__device__ __forceinline__ void q8_tile_pick(int mt, const Q8Args& a, const Q8Block& blk, int m0, int v0,
                                             const TileWave<WCOPY, XCOPY>& t, uint8_t* buf0,
                                             uint8_t* buf1) {
  if constexpr (M > 1) {
    if (mt < M) {
      q8_tile_pick<M - 1, WM, WN, NT, WCOPY, XCOPY, GATHER, SWIGLU>(mt, a, blk, m0, v0, t, buf0, buf1);
      return;
    }
  }
  q8_tile_rows<M, WM, WN, NT, WCOPY, XCOPY, GATHER, SWIGLU>(a, blk, m0, v0, t, buf0, buf1);
}

template <int WM, int WN, int MT, int NT, bool GROUPED, bool GATHER, bool SWIGLU>
__global__ __launch_bounds__(64 * WM * WN) void q8_tile_kernel(Q8Args a) {
  constexpr int WAVES = WM * WN, BM = WM * MT * 16, BN = WN * NT * 16;
  constexpr int WCOPY = BN / 8 / WAVES;  // copies of eight weight rows per wave and step
  constexpr int XCOPY = BM / 8 / WAVES;  // of eight token rows, at most
  static_assert(WCOPY * 8 * WAVES == BN && XCOPY * 8 * WAVES == BM, "whole copies");
  // distinct arrays, so that reads of one do not wait for the copies into the other
  __shared__ __attribute__((aligned(1024))) uint8_t buf0[(BN + BM) * kStep];
  __shared__ __attribute__((aligned(1024))) uint8_t buf1[(BN + BM) * kStep];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int nt = (a.N + BN - 1) / BN;
  const int nb = GROUPED ? min(*a.n_blocks, a.max_blocks) : (a.rows + BM - 1) / BM;
  int b, ni;
  {
    const int total = nb * nt, per = (total + 7) / 8;
    const int i = blockIdx.x >> 3, tile = (blockIdx.x & 7) * per + i;
    if (i >= per || tile >= total) return;
    const int g = tile / (4 * nt), r = tile - g * 4 * nt, gm = min(4, nb - 4 * g);
    b = 4 * g + r % gm;
    ni = r / gm;
  }
  Q8Block blk;
  if (GROUPED) {
    if (!q8_block(a, b, blk)) return;
  } else {
    blk.w = a.w;
    blk.ws = a.ws;
    blk.row0 = b * BM;
    blk.rows = min(BM, a.rows - blk.row0);
  }
  const int v0 = ni * BN;
  TileWave<WCOPY, XCOPY> t;
  t.lane = lane;
  t.wave = wave;
  t.wm = wave / WN;
  t.wn = wave % WN;
  t.piece = ((lane & 7) ^ (lane >> 3)) * 16;
#pragma unroll
  for (int i = 0; i < WCOPY; ++i)
    t.wp[i] = blk.w +
              static_cast<size_t>(q8_weight_row<SWIGLU>(v0 + (i * WAVES + wave) * 8 + (lane >> 3), a.N)) * a.K;
  for (int m0 = 0; m0 < blk.rows; m0 += BM) {
    const int mt = (min(BM, blk.rows - m0) + WM * 16 - 1) / (WM * 16);
    t.xcopies = 2 * WM * mt;
#pragma unroll
    for (int i = 0; i < XCOPY; ++i) {
      const int m = min(m0 + (i * WAVES + wave) * 8 + (lane >> 3), blk.rows - 1);
      t.xp[i] = a.x + static_cast<size_t>(max(q8_source<GATHER>(a, blk.row0 + m), 0)) * a.K;
    }
    q8_tile_pick<MT, WM, WN, NT, WCOPY, XCOPY, GATHER, SWIGLU>(mt, a, blk, m0, v0, t, buf0, buf1);
    __syncthreads();  // the buffers have been read before the next rows' copies
  }
}

int cdiv(int a, int b) { return (a + b - 1) / b; }

template <int CT, int MT, bool GROUPED, bool GATHER, bool SWIGLU>
void launch_stream(const Q8Args& a, int blocks, hipStream_t s) {
  const long long n = static_cast<long long>(blocks) * cdiv(a.N, CT * 16);
  hipLaunchKernelGGL((q8_stream_kernel<CT, MT, GROUPED, GATHER, SWIGLU>), dim3(static_cast<unsigned>(n)),
                     dim3(256), 0, s, a);
}

template <int WM, int WN, int MT, int NT, bool GROUPED, bool GATHER, bool SWIGLU>
void launch_tile(const Q8Args& a, int blocks, hipStream_t s) {
  const long long tiles = static_cast<long long>(blocks) * cdiv(a.N, WN * NT * 16);
  hipLaunchKernelGGL((q8_tile_kernel<WM, WN, MT, NT, GROUPED, GATHER, SWIGLU>),
                     dim3(static_cast<unsigned>((tiles + 7) / 8 * 8)), dim3(64 * WM * WN), 0, s, a);
}

// rows_per_block: rows a block is expected to hold; blocks: the most there can
// be; used: blocks expected to be there.
template <bool GROUPED, bool GATHER, bool SWIGLU>
hipError_t launch_q8(const Q8Args& a, int rows_per_block, int blocks, int used, hipStream_t s) {
  if (rows_per_block <= 32) {
    const bool two = rows_per_block > 16;
    const long long columns = static_cast<long long>(used) * (a.N / 16);
    if (columns >= 4 * 512) {
      two ? launch_stream<4, 2, GROUPED, GATHER, SWIGLU>(a, blocks, s)
          : launch_stream<4, 1, GROUPED, GATHER, SWIGLU>(a, blocks, s);
    } else {
      two ? launch_stream<2, 2, GROUPED, GATHER, SWIGLU>(a, blocks, s)
          : launch_stream<2, 1, GROUPED, GATHER, SWIGLU>(a, blocks, s);
    }
  } else if (GROUPED) {
    if (rows_per_block <= 128)
      launch_tile<2, 2, 4, 4, GROUPED, GATHER, SWIGLU>(a, blocks, s);
    else
      launch_tile<2, 4, 8, 4, GROUPED, GATHER, SWIGLU>(a, blocks, s);
  } else {
    if (static_cast<long long>(cdiv(a.rows, 256)) * cdiv(a.N, 256) >= 256)
      launch_tile<2, 4, 8, 4, GROUPED, GATHER, SWIGLU>(a, cdiv(a.rows, 256), s);
    else
      launch_tile<2, 2, 4, 4, GROUPED, GATHER, SWIGLU>(a, cdiv(a.rows, 128), s);
  }
  return hipGetLastError();
}

// What a grouped call expects of its block map, from the host's side alone:
// the routed slots spread evenly over the experts they can touch.
void expected_blocks(const moe_dims& d, int& rows_per_block, int& used) {
  const long long S = static_cast<long long>(d.T) * d.k;
  const int touched = static_cast<int>(S < d.E ? S : d.E);
  const int avg = static_cast<int>((S + touched - 1) / touched);
  const int cuts = cdiv(avg, d.tile_m_max);
  rows_per_block = cdiv(avg, cuts);
  used = touched * cuts + (d.n_shared ? cdiv(d.T, d.tile_m_max) : 0);
}

int validate_grouped(const moe_dims* d, const moe_route_out* r, const void* xq, const void* xs,
                     const void* out) {
  int rc = validate_dims(d);
  if (rc) return rc;
  if ((rc = validate_route_out(r, false))) return rc;
  if (!xq || !xs || !out) return MOE_EINVAL;
  if (!aligned(xq, 16) || !aligned(xs, 4) || !aligned(out, 16)) return MOE_EALIGN;
  return MOE_OK;
}

int validate_half(const int8_t* w, const float* s) {
  if (!w || !s) return MOE_EINVAL;
  return aligned(w, 16) && aligned(s, 16) ? MOE_OK : MOE_EALIGN;
}

Q8Args grouped_args(const moe_dims& d, const moe_route_out* r, const int8_t* xq, const float* xs,
                    void* out) {
  Q8Args a{};
  a.x = xq;
  a.xs = xs;
  a.out = out;
  a.rows = d.T * (d.k + d.n_shared);
  a.type = MOE_ELEM_BF16;
  a.blocks = r->blocks;
  a.n_blocks = r->n_blocks;
  a.sorted_slot = r->sorted_slot;
  a.status = r->status;
  a.max_blocks = max_blocks_of(d);
  a.E = d.E;
  a.T = d.T;
  a.k = d.k;
  a.n_shared = d.n_shared;
  return a;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_q8_matmul(const moe_q8_dims* d, const int8_t* xq, const float* xs, const int8_t* wq,
                  const float* ws, void* out, void* stream) {
  if (!d || d->M < 0 || d->M > (1 << 24) || d->N <= 0 || d->N % 8 || d->N > (1 << 20) || d->K <= 0 ||
      d->K % 64 || d->K > (1 << 16) || !elem_ok(d->type))
    return MOE_EINVAL;
  if (!xq || !xs || !wq || !ws || !out) return MOE_EINVAL;
  if (!aligned(xq, 16) || !aligned(xs, 4) || !aligned(wq, 16) || !aligned(ws, 16) || !aligned(out, 16))
    return MOE_EALIGN;
  if (d->M == 0) return MOE_OK;
  int rc = check_device();
  if (rc) return rc;
  Q8Args a{};
  a.x = xq;
  a.xs = xs;
  a.w = wq;
  a.ws = ws;
  a.out = out;
  a.rows = d->M;
  a.N = d->N;
  a.K = d->K;
  a.type = d->type;
  (void)hipGetLastError();
  return launched(launch_q8<false, false, false>(a, d->M, 1, 1, static_cast<hipStream_t>(stream)));
}

int moe_q8_gate_up(const moe_dims* d, const int8_t* xq, const float* xs, const moe_route_out* r,
                   const moe_q8_bank* routed, const moe_q8_bank* shared, uint16_t* h, void* stream) {
  int rc = validate_grouped(d, r, xq, xs, h);
  if (rc) return rc;
  if (!routed || (d->n_shared && !shared)) return MOE_EINVAL;
  if ((rc = validate_half(routed->gu, routed->gu_s))) return rc;
  if (d->n_shared && (rc = validate_half(shared->gu, shared->gu_s))) return rc;
  if (d->T == 0) return MOE_OK;
  if ((rc = check_device())) return rc;
  Q8Args a = grouped_args(*d, r, xq, xs, h);
  a.w = routed->gu;
  a.ws = routed->gu_s;
  a.w_shared = d->n_shared ? shared->gu : nullptr;
  a.ws_shared = d->n_shared ? shared->gu_s : nullptr;
  a.N = 2 * d->I;
  a.K = d->H;
  int per, used;
  expected_blocks(*d, per, used);
  (void)hipGetLastError();
  return launched(launch_q8<true, true, true>(a, per, a.max_blocks, used, static_cast<hipStream_t>(stream)));
}

int moe_q8_down(const moe_dims* d, const moe_route_out* r, const moe_q8_bank* routed,
                const moe_q8_bank* shared, const int8_t* hq, const float* hs, uint16_t* y_slots,
                void* stream) {
  int rc = validate_grouped(d, r, hq, hs, y_slots);
  if (rc) return rc;
  if (!routed || (d->n_shared && !shared)) return MOE_EINVAL;
  if ((rc = validate_half(routed->dn, routed->dn_s))) return rc;
  if (d->n_shared && (rc = validate_half(shared->dn, shared->dn_s))) return rc;
  if (d->T == 0) return MOE_OK;
  if ((rc = check_device())) return rc;
  Q8Args a = grouped_args(*d, r, hq, hs, y_slots);
  a.w = routed->dn;
  a.ws = routed->dn_s;
  a.w_shared = d->n_shared ? shared->dn : nullptr;
  a.ws_shared = d->n_shared ? shared->dn_s : nullptr;
  a.N = d->H;
  a.K = d->I;
  int per, used;
  expected_blocks(*d, per, used);
  (void)hipGetLastError();
  return launched(launch_q8<true, false, false>(a, per, a.max_blocks, used, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
