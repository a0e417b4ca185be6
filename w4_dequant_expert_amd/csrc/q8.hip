// Matrix products in 8-bit integers with a scale for each token and each
// output channel, dense and grouped by expert (include/moe_block.h):
//   out[m][n] = xs[m] ws[n] sum_k xq[m][k] wq[n][k]
// The sum is exact in int32 (|xq wq| <= 2^14 and K <= 2^16 give at most 2^30),
// so the order of its terms is free: kernels may split K over waves, or read
// the inputs in any order the two operands share, and every kernel here gives
// the same bits.
//
// Two kernels, on the int8 matrix instructions (weights as the first operand,
// so a lane ends with runs of four neighbouring output channels of one row):
//   q8_stream_kernel: few rows.  Bound by reading the weights once; every wave
//     streams its share of K straight from memory into the matrix operands,
//     with no LDS and no barrier until the waves' sums are added.  One row of
//     2048 times 8192 columns: 5.1 us, 3.3 TB/s.
//   q8_tile_kernel: more rows.  Tiles of both operands go through LDS in steps
//     of 128 inputs.  Bound by the weights' bytes up to some hundred rows a
//     matrix (512 tokens over 256 experts: 5.1 to 5.3 TB/s), then by what the
//     L2s feed the copies: without its copies a step of the largest tile takes
//     1.1 us, the time of its products, with them 1.5.
#include <algorithm>

#include "block.h"

namespace moe {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

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
  int stream_out;           // outputs past the caches (more of them than kStreamStore)
  int stream_w;             // an expert's rows are one block, so its weights are read once
  // grouped products only
  const int32_t* blocks;
  const int32_t* n_blocks;
  const int32_t* sorted_slot;
  uint32_t* status;
  int max_blocks, E, T, k, n_shared, tile_m_max;
};

// A block of output rows that share one weight matrix.
struct Q8Block {
  const int8_t* w;
  const float* ws;
  int row0, rows;
  bool once;  // nobody else reads these weights
};

// Block b < max_blocks of the map; false past its end, and (with the status
// bit) for an entry out of range.  One of more than tile_m_max rows counts as
// such for every kernel, so that which one is chosen never decides it.
__device__ __forceinline__ bool q8_block(const Q8Args& a, int b, Q8Block& o) {
  int4 e;
  if (!map_entry(reinterpret_cast<const int4*>(a.blocks), a.n_blocks, b, e)) return false;
  const int g = uniform(e.x);
  o.row0 = uniform(e.y);
  o.rows = uniform(e.z);
  const bool shared = g == a.E;
  if (g < 0 || g > a.E || (shared && !a.n_shared) || o.row0 < 0 || o.rows <= 0 ||
      o.rows > min(a.tile_m_max, a.rows - o.row0)) {
    if (threadIdx.x == 0) status_set(a.status, MOE_STATUS_BAD_INDEX);
    return false;
  }
  o.w = shared ? a.w_shared : a.w + static_cast<size_t>(g) * a.N * a.K;
  o.ws = shared ? a.ws_shared : a.ws + static_cast<size_t>(g) * a.N;
  o.once = a.stream_w && !shared;
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

// The weight row of virtual column v.  SwiGLU pairs W gate rows (the width of
// a matrix tile) with their W up rows, so that one wave holds both in the same
// lanes.
template <bool SWIGLU, int W>
__device__ __forceinline__ int q8_weight_row(int v, int N) {
  if (!SWIGLU) return min(v, N - 1);
  const int half = N / 2, r = (v / (2 * W)) * W + v % W;
  return (v & W) ? min(half + r, N - 1) : min(r, half - 1);
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

// Four neighbouring outputs of one row from the integer sums; s their channels' scales.
__device__ __forceinline__ void q8_scale(float xs, float4 s, i32x4 acc, float (&o)[4]) {
  const float f[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = static_cast<float>(acc[i]) * xs * f[i];
}

// silu(g) u of four neighbouring hidden columns.
__device__ __forceinline__ void q8_swiglu(float xs, float4 sg, float4 su, i32x4 g, i32x4 u, float (&o)[4]) {
  float gv[4], uv[4];
  q8_scale(xs, sg, g, gv);
  q8_scale(xs, su, u, uv);
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = gv[i] * __builtin_amdgcn_rcpf(1.0f + __expf(-gv[i])) * uv[i];
}

// Scales of columns v .. v+3 (v a multiple of 4, N of 8); past N zeros.
__device__ __forceinline__ float4 load_scales(const float* __restrict__ ws, int v, int N) {
  return v < N ? *reinterpret_cast<const float4*>(ws + v) : make_float4(0.f, 0.f, 0.f, 0.f);
}

__device__ __forceinline__ i32x4 mfma(uint4 a, uint4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c,
                                               0, 0, 0);
}

__device__ __forceinline__ i32x16 mfma32(uint4 a, uint4 b, i32x16 c) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c,
                                               0, 0, 0);
}

// ---------------------------------------------------------------------------
// Few rows.  A workgroup of W waves owns CT*16 columns of a block and takes its
// rows MT*16 at a time; wave w multiplies every W-th unit of 128 inputs.  A load
// covers 64 contiguous bytes of each of sixteen rows.  The waves' sums meet in
// LDS.
// ---------------------------------------------------------------------------
template <int W, int CT, int MT, bool GROUPED, bool GATHER, bool SWIGLU>
__global__ __launch_bounds__(64 * W) void q8_stream_kernel(Q8Args a) {
  static_assert(!SWIGLU || CT % 2 == 0, "gate and up columns come in pairs");
  __shared__ i32x4 part[W][MT * CT][64];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int q = lane >> 4, r16 = lane & 15;
  const int nt = (a.N + CT * 16 - 1) / (CT * 16);
  const int b = blockIdx.x / nt;
  const int v0 = (blockIdx.x % nt) * CT * 16;
  Q8Block blk;
  if (GROUPED) {
    if (!q8_block(a, b, blk)) return;
  } else {
    blk.w = a.w;
    blk.ws = a.ws;
    blk.row0 = 0;
    blk.rows = a.rows;
    blk.once = false;
  }
  const int8_t* wp[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c)
    wp[c] = blk.w + static_cast<size_t>(q8_weight_row<SWIGLU, 16>(v0 + c * 16 + r16, a.N)) * a.K + q * 16;
  const int units = (a.K + 127) / 128;
  for (int m0 = 0; m0 < blk.rows; m0 += MT * 16) {
    const int8_t* xp[MT];
    i32x4 acc[MT][CT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int c = 0; c < CT; ++c) acc[m][c] = i32x4{0, 0, 0, 0};
    for (int u = wave; u < units; u += W) {
      uint4 wv[CT][2], xv[MT][2];
      const int at = u * 128;
      const bool whole = at + 64 < a.K;         // the last unit may hold 64 inputs,
      const int second = whole ? at + 64 : at;  // which are then not multiplied twice
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        wv[c][0] = *reinterpret_cast<const uint4*>(wp[c] + at);
        wv[c][1] = *reinterpret_cast<const uint4*>(wp[c] + second);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (u == wave) {
        // the tokens' addresses wait for the routing tables: behind the first
        // weight loads, which do not
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int src = q8_source<GATHER>(a, blk.row0 + min(m0 + m * 16 + r16, blk.rows - 1));
          xp[m] = a.x + static_cast<size_t>(max(src, 0)) * a.K + q * 16;
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        xv[m][0] = *reinterpret_cast<const uint4*>(xp[m] + at);
        xv[m][1] = *reinterpret_cast<const uint4*>(xp[m] + second);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && !whole) break;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int c = 0; c < CT; ++c) acc[m][c] = mfma(wv[c][h], xv[m][h], acc[m][c]);
      }
    }
    if (m0) __syncthreads();  // the sums of the rows before have been read
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int c = 0; c < CT; ++c) part[wave][m * CT + c][lane] = acc[m][c];
    __syncthreads();
    auto total = [&](int i) {
      i32x4 s = part[0][i][lane];
#pragma unroll
      for (int w = 1; w < W; ++w) s += part[w][i][lane];
      return s;
    };
    constexpr int STEP = SWIGLU ? 2 : 1;
    for (int i = wave * STEP; i < MT * CT; i += W * STEP) {
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
      float o[4];
      if (SWIGLU) {
        const int c = v / 2 + 4 * q, half = a.N / 2;
        if (c >= half) continue;
        q8_swiglu(xs, load_scales(blk.ws, c, half), load_scales(blk.ws + half, c, half), total(i), total(i + 1), o);
        store4(a.out, static_cast<size_t>(row) * half + c, MOE_ELEM_BF16, o);
      } else {
        const int c = v + 4 * q;
        if (c >= a.N) continue;
        q8_scale(xs, load_scales(blk.ws, c, a.N), total(i), o);
        store4(a.out, static_cast<size_t>(row) * a.N + c, a.type, o);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Many rows.  WM x WN waves own a tile of up to WM*MT*32 rows and WN*NT*32
// columns; a wave multiplies M (1..MT, from the block's rows) times NT tiles
// of 32 x 32, by v_mfma_i32_32x32x32_i8: each operand register feeds twice the
// products of the 16 x 16 form.
//
// K goes by in steps of 128 inputs (whole cache lines of both operands)
// through a ring of R LDS buffers, each step in four quarters of 32 inputs.
// The operands of a quarter are read from LDS under the products of the quarter
// before.  The one barrier of a step stands before the products of its last
// quarter, whose operands are in registers by then: behind it the next step is
// in LDS and nobody reads this step's buffer any more, so the copies of step
// s + R start into it and have R - 1 steps to land.
//
// A staged row is 128 bytes, its 16-byte pieces XORed by the row (piece c of
// row r at c ^ (r / 2 mod 8)), so that any sixteen neighbouring rows of a
// fragment cover all 64 banks.  A copy moves eight rows, lane l's 16 bytes
// landing at byte 16 l: the permutation is made by the address each lane reads.
// Rows past the block repeat its last row and columns past N the last column;
// they only reach outputs that are not stored.
//
// Tiles are dealt to the chip's eight XCDs (workgroup i runs on XCD i mod 8, a
// row of the grid being a multiple of 8) in contiguous runs, so that the tiles
// an XCD works on together share rows and columns in its own L2: a dense run
// goes through groups of four row blocks column by column (8192 cubed: groups of
// one 513 us, two 467, four 456, eight 461), a grouped one block by block
// (gate/up of 16384 tokens: 411 us, in groups of four 424), since neighbouring
// blocks mostly have other weights.
// ---------------------------------------------------------------------------
constexpr int kStep = 128;
constexpr int kNonTemporal = 2;  // cache policy of a copy whose data nobody else reads

// At most N of this wave's copies are still in flight, its LDS reads are done
// and every wave is here.  The wait is the builtin, which the compiler's own
// bookkeeping of waits takes into account; the empty statements keep LDS
// accesses from moving across.
template <int N>
__device__ __forceinline__ void copies_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));  // vmcnt(N) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// What a wave of a tile keeps over the steps.
template <int WCOPY, int XCOPY>
struct TileWave {
  const int8_t* wbase[WCOPY];  // first weight row of each of the wave's copies (uniform)
  uint32_t woff[WCOPY];        // this lane's bytes from there
  const int8_t* xp[XCOPY];     // its token row in each
  int piece;                   // the bytes of a step this lane copies
  int wave, wm, wn, lane;
};

// 32 rows of a wave's outputs, from its sums to memory.  A lane holds, of each
// tile of 32 columns, the columns 8g + 4hi .. +3 (g = 0..3) of row lane mod 32:
// they go to LDS as rows, their 16-byte pieces XORed by the row against bank
// conflicts, and come back as whole pieces in row order, so that a store
// covers whole lines.  The wave uses LDS of its own, whose accesses stay in
// order.  ok: this lane's row (lane mod 32) may be stored.
template <int NT, bool SWIGLU, int TYPE>
__device__ __forceinline__ void q8_tile_out(const Q8Args& a, const Q8Block& blk, const i32x16 (&acc)[NT],
                                            const float4 (&sc)[NT][4], float xs, uint8_t* out, int m1, int c0,
                                            int n_out, int lane, bool ok) {
  constexpr int ELEM = TYPE == MOE_ELEM_F32 ? 4 : 2;
  constexpr int COLS = (SWIGLU ? NT / 2 : NT) * 32, PIECES = COLS * ELEM / 16;
  const int r32 = lane & 31, hi = lane >> 5;
  // XOR of a row's pieces: sixteen rows' pieces cover all banks (256 bytes)
  const auto turn = [](int r) { return (r * PIECES / 16) & (PIECES - 1); };
#pragma unroll
  for (int j = 0; j < NT; j += SWIGLU ? 2 : 1) {
    const int cj = SWIGLU ? j / 2 * 32 : j * 32;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int c = cj + 8 * g + 4 * hi;
      const i32x4 s0 = {acc[j][4 * g], acc[j][4 * g + 1], acc[j][4 * g + 2], acc[j][4 * g + 3]};
      float o[4];
      if (SWIGLU) {
        constexpr int P = SWIGLU ? 1 : 0;
        const i32x4 s1 = {acc[j + P][4 * g], acc[j + P][4 * g + 1], acc[j + P][4 * g + 2], acc[j + P][4 * g + 3]};
        q8_swiglu(xs, sc[j][g], sc[j + P][g], s0, s1, o);
      } else {
        q8_scale(xs, sc[j][g], s0, o);
      }
      const int byte = c * ELEM;
      uint8_t* const to = out + r32 * PIECES * 16 + (((byte >> 4) ^ turn(r32)) << 4);
      store4(to + (byte & 15), 0, TYPE, o);
    }
  }
  asm volatile("" ::: "memory");
  const uint64_t stored = __ballot(ok);
#pragma unroll
  for (int it = 0; it < 32 * PIECES / 64; ++it) {
    const int r = (it * 64 + lane) / PIECES, piece = (it * 64 + lane) % PIECES;
    const uint4 v = *reinterpret_cast<const uint4*>(out + r * PIECES * 16 + ((piece ^ turn(r)) << 4));
    const int c = c0 + piece * (16 / ELEM);
    if (m1 + r < blk.rows && c < n_out && ((stored >> r) & 1)) {
      uint4* const to = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) +
                                                 (static_cast<size_t>(blk.row0 + m1 + r) * n_out + c) * ELEM);
      if (a.stream_out)
        store16<true>(to, v);
      else
        store16<false>(to, v);
    }
  }
  asm volatile("" ::: "memory");
}

// One pass over K for M tiles of rows per wave, and their outputs.
template <int M, int WM, int WN, int NT, int R, int WCOPY, int XCOPY, bool GROUPED, bool GATHER, bool SWIGLU>
__device__ __forceinline__ void q8_tile_rows(const Q8Args& a, const Q8Block& blk, int m0, int v0,
                                             const TileWave<WCOPY, XCOPY>& t, uint8_t* b0, uint8_t* b1,
                                             uint8_t* b2, uint8_t* b3) {
  constexpr int WAVES = WM * WN, BN = WN * NT * 32, BM = XCOPY * 8 * WAVES;
  // copies of token rows each wave makes, the same for all (so that the copies
  // in flight are a known number): past the rows they repeat the last row
  constexpr int XC = (WM * M * 4 + WAVES - 1) / WAVES;
  constexpr int COPIES = WCOPY + XC;
  static_assert(XC <= XCOPY && (R - 2) * COPIES < 64, "copies in flight fit the wait's field");
  const int nk = (a.K + kStep - 1) / kStep;
  const int r32 = t.lane & 31, hi = t.lane >> 5;
  i32x16 acc[M][NT];
#pragma unroll
  for (int i = 0; i < M; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;
  // Copy i (0 .. COPIES-1) of step s: the wave's weight rows, then its token
  // rows.  The last step may hold 64 inputs: its second half repeats the first
  // (read into LDS, never multiplied).
  auto copy_one = [&](int s, uint8_t* buf, int i) {
    const int at = s * kStep + t.piece;
    const int k0 = at < a.K ? at : at - 64;
    if (i < WCOPY) {
      uint8_t* const to = buf + (i * WAVES + t.wave) * 1024;
      if (GROUPED && WM * M <= 2 && blk.once)
        __builtin_amdgcn_global_load_lds(t.wbase[i] + (t.woff[i] + static_cast<uint32_t>(k0)), to, 16, 0, kNonTemporal);
      else
        __builtin_amdgcn_global_load_lds(t.wbase[i] + (t.woff[i] + static_cast<uint32_t>(k0)), to, 16, 0, 0);
    } else {
      __builtin_amdgcn_global_load_lds(t.xp[i - WCOPY] + k0, buf + BN * kStep + ((i - WCOPY) * WAVES + t.wave) * 1024,
                                       16, 0, 0);
    }
  };
  auto copy = [&](int s, uint8_t* buf) {
#pragma unroll
    for (int i = 0; i < COPIES; ++i) copy_one(s, buf, i);
  };
  struct Frags {
    uint4 w[NT], x[M];
  };
  // quarter q (inputs 32q .. 32q+31) of a step
  auto read = [&](Frags& f, const uint8_t* buf, int q) {
    const int at = r32 * kStep + (((2 * q + hi) ^ ((r32 >> 1) & 7)) << 4);
#pragma unroll
    for (int j = 0; j < NT; ++j)
      f.w[j] = *reinterpret_cast<const uint4*>(buf + (t.wn * NT + j) * 32 * kStep + at);
#pragma unroll
    for (int i = 0; i < M; ++i)
      f.x[i] = *reinterpret_cast<const uint4*>(buf + (BN + (t.wm * M + i) * 32) * kStep + at);
  };
  // products lo .. hi-1 of the wave's M * NT
  auto multiply = [&](const Frags& f, int lo, int hi) {
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
        if (i * NT + j >= lo && i * NT + j < hi) acc[i][j] = mfma32(f.w[j], f.x[i], acc[i][j]);
  };
  Frags fa, fb;
  // Products lo .. of f with copies c0 .. c1-1 of step s started between them.
  auto spread = [&](const Frags& f, int lo, bool on, int s, uint8_t* buf, int c0, int c1) {
    const int n = c1 - c0, left = M * NT - lo;
#pragma unroll
    for (int c = 0; c < n; ++c) {
      if (on) copy_one(s, buf, c0 + c);
      __builtin_amdgcn_sched_barrier(0);
      multiply(f, lo + left * c / n, lo + left * (c + 1) / n);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (n == 0) multiply(f, lo, M * NT);
    __builtin_amdgcn_sched_barrier(0);
  };
  // One quarter: its products from f, quarter q of buf read into g behind the
  // first of them (so that the wait for f stands ahead of the newer reads).
  auto quarter = [&](const Frags& f, Frags& g, const uint8_t* buf, int q, bool on, int s, uint8_t* to, int c0, int c1) {
    multiply(f, 0, 1);
    __builtin_amdgcn_sched_barrier(0);
    read(g, buf, q);
    __builtin_amdgcn_sched_barrier(0);
    spread(f, 1, on, s, to, c0, c1);
  };
  // With eight waves a step's copies keep the address path busy for about half
  // of the step's products, and a wave that waits there multiplies nothing: two
  // eighths of them are started in the quarter behind the barrier, three in the
  // next step's first quarter and three in its second, between the products
  // (16384x8192x4096: 509 us in one run behind the barrier, 475 spread).
  constexpr bool SPREAD = WAVES >= 8;
  constexpr int C1 = SPREAD ? (COPIES * 2 + 7) / 8 : COPIES, C2 = SPREAD ? (COPIES * 5 + 7) / 8 : COPIES;
  // Step s from its first quarter's operands in fa; leaves the next step's
  // there.  full: the R - 1 steps after it are there.  prev: the buffer that
  // step s - 1 freed, whose copies (of step s + R - 1) go on under this step.
  auto step = [&](int s, bool full, uint8_t* cur, uint8_t* next, uint8_t* prev) {
    const bool on = SPREAD && s > 0 && s + R - 1 < nk;
    quarter(fa, fb, cur, 1, on, s + R - 1, prev, C1, C2);
    if ((s + 1) * kStep <= a.K) {  // else 64 inputs: two quarters
      quarter(fb, fa, cur, 2, on, s + R - 1, prev, C2, COPIES);
      quarter(fa, fb, cur, 3, false, 0, prev, 0, 0);
    }
    if (full || s + R - 1 < nk)
      copies_barrier<(R - 2) * COPIES>();
    else
      copies_barrier<0>();
    __builtin_amdgcn_sched_barrier(0);
    if (!SPREAD && s + R < nk) copy(s + R, cur);
    if (full || s + 1 < nk) read(fa, next, 0);
    __builtin_amdgcn_sched_barrier(0);
    if (SPREAD)
      spread(fb, 0, s + R < nk, s + R, cur, 0, C1);
    else
      multiply(fb, 0, M * NT);
    __builtin_amdgcn_sched_barrier(0);
  };
  uint8_t* const ring[4] = {b0, b1, b2, b3};
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (i < nk) copy(i, ring[i]);
  if (nk >= R)
    copies_barrier<(R - 1) * COPIES>();
  else
    copies_barrier<0>();
  read(fa, b0, 0);
  int s = 0;
  for (; s + 2 * R - 2 < nk; s += R)
#pragma unroll
    for (int i = 0; i < R; ++i) step(s + i, true, ring[i], ring[(i + 1) % R], ring[(i + R - 1) % R]);
  for (; s < nk; s += R)
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (s + i < nk) step(s + i, false, ring[i], ring[(i + 1) % R], ring[(i + R - 1) % R]);
  // Every wave has read its last operands (the last step's barrier): its share
  // of the buffers holds its outputs, 32 rows at a time, on the way to
  // whole-line stores.
  constexpr int kShare = (BN + BM) * kStep / (WAVES / 2);
  uint8_t* const out = (t.wave < WAVES / 2 ? b0 : b1) + (t.wave % (WAVES / 2)) * kShare;
  const int n_out = SWIGLU ? a.N / 2 : a.N;
  const int c0 = (SWIGLU ? v0 / 2 : v0) + t.wn * (SWIGLU ? NT / 2 : NT) * 32;
  // the scales of the wave's columns and rows, loaded together
  float4 sc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int c = c0 + (SWIGLU ? j / 2 : j) * 32 + 8 * g + 4 * hi;
      sc[j][g] = load_scales(blk.ws + (SWIGLU && j % 2 ? n_out : 0), c, n_out);
    }
  int srcs[M];
  float xss[M];
#pragma unroll
  for (int i = 0; i < M; ++i) {
    srcs[i] = q8_source<GATHER>(a, blk.row0 + min(m0 + (t.wm * M + i) * 32 + r32, blk.rows - 1));
    xss[i] = a.xs[max(srcs[i], 0)];
  }
#pragma unroll
  for (int i = 0; i < M; ++i) {
    const int m1 = m0 + (t.wm * M + i) * 32;
    if (m1 >= blk.rows) break;
    const int src = srcs[i];
    if (src < 0) status_set(a.status, MOE_STATUS_BAD_INDEX);
    const float xs = xss[i];
    if constexpr (!GROUPED) {
      static_assert(32 * NT * 32 * 4 <= kShare, "a wave's outputs fit its share");
      if (a.type == MOE_ELEM_F32) {
        q8_tile_out<NT, SWIGLU, MOE_ELEM_F32>(a, blk, acc[i], sc, xs, out, m1, c0, n_out, t.lane, true);
        continue;
      } else if (a.type == MOE_ELEM_F16) {
        q8_tile_out<NT, SWIGLU, MOE_ELEM_F16>(a, blk, acc[i], sc, xs, out, m1, c0, n_out, t.lane, true);
        continue;
      }
    }
    q8_tile_out<NT, SWIGLU, MOE_ELEM_BF16>(a, blk, acc[i], sc, xs, out, m1, c0, n_out, t.lane, !GATHER || src >= 0);
  }
}

// q8_tile_rows for mt (1..M) tiles of rows.
template <int M, int WM, int WN, int NT, int R, int WCOPY, int XCOPY, bool GROUPED, bool GATHER, bool SWIGLU>
__device__ __forceinline__ void q8_tile_pick(int mt, const Q8Args& a, const Q8Block& blk, int m0, int v0,
                                             const TileWave<WCOPY, XCOPY>& t, uint8_t* b0, uint8_t* b1,
                                             uint8_t* b2, uint8_t* b3) {
  if constexpr (M > 1) {
    if (mt < M) {
      q8_tile_pick<M - 1, WM, WN, NT, R, WCOPY, XCOPY, GROUPED, GATHER, SWIGLU>(mt, a, blk, m0, v0, t, b0, b1, b2, b3);
      return;
    }
  }
  q8_tile_rows<M, WM, WN, NT, R, WCOPY, XCOPY, GROUPED, GATHER, SWIGLU>(a, blk, m0, v0, t, b0, b1, b2, b3);
}

template <int WM, int WN, int MT, int NT, int R, bool GROUPED, bool GATHER, bool SWIGLU>
__global__ __launch_bounds__(64 * WM * WN, 2) void q8_tile_kernel(Q8Args a) {
  constexpr int WAVES = WM * WN, BM = WM * MT * 32, BN = WN * NT * 32;
  constexpr int WCOPY = BN / 8 / WAVES;  // copies of eight weight rows per wave and step
  constexpr int XCOPY = BM / 8 / WAVES;  // of eight token rows, at most
  static_assert(WCOPY * 8 * WAVES == BN && XCOPY * 8 * WAVES == BM, "whole copies");
  static_assert(!SWIGLU || NT % 2 == 0, "gate and up columns come in pairs");
  // distinct arrays, so that reads of one do not wait for the copies into the other
  __shared__ __attribute__((aligned(1024))) uint8_t b0[(BN + BM) * kStep];
  __shared__ __attribute__((aligned(1024))) uint8_t b1[(BN + BM) * kStep];
  __shared__ __attribute__((aligned(1024))) uint8_t b2[R > 2 ? (BN + BM) * kStep : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t b3[R > 3 ? (BN + BM) * kStep : 16];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int nt = (a.N + BN - 1) / BN;
  static_assert(R >= 2 && R <= 4, "buffers");
  const int nb = GROUPED ? min(*a.n_blocks, a.max_blocks) : (a.rows + BM - 1) / BM;
  int b, ni;
  {
    const int total = nb * nt, per = (total + 7) / 8;
    const int i = static_cast<int>(workgroup() >> 3), tile = static_cast<int>(blockIdx.x & 7) * per + i;
    if (i >= per || tile >= total) return;
    constexpr int G = GROUPED ? 1 : 4;
    const int g = tile / (G * nt), r = tile - g * G * nt, gm = min(G, nb - G * g);
    b = G * g + r % gm;
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
    blk.once = false;
  }
  const int v0 = ni * BN;
  TileWave<WCOPY, XCOPY> t;
  t.lane = lane;
  t.wave = wave;
  t.wm = wave / WN;
  t.wn = wave % WN;
  const int crow = lane >> 3;
  // copy i of a wave starts at row 8 (i WAVES + wave): r / 2 mod 8 is known up to its wave's parity
  static_assert(WAVES % 2 == 0, "copies of a wave share their parity");
  t.piece = ((lane & 7) ^ ((crow >> 1) + 4 * (wave & 1))) * 16;
#pragma unroll
  for (int i = 0; i < WCOPY; ++i) {
    // the eight rows of a copy lie in one run of gate or up rows
    const int v = v0 + (i * WAVES + wave) * 8;
    const int first = uniform(q8_weight_row<SWIGLU, 32>(v, a.N));
    t.wbase[i] = blk.w + static_cast<size_t>(first) * a.K;
    t.woff[i] = static_cast<uint32_t>(q8_weight_row<SWIGLU, 32>(v + crow, a.N) - first) * a.K;
  }
  // blocks have tile_m_max rows at most, which is 256 at most: one pass of the largest tile
  for (int m0 = 0; m0 < (BM >= 256 ? 1 : blk.rows); m0 += BM) {
    const int mt = (min(BM, blk.rows - m0) + WM * 32 - 1) / (WM * 32);
#pragma unroll
    for (int i = 0; i < XCOPY; ++i) {
      const int m = min(m0 + (i * WAVES + wave) * 8 + crow, blk.rows - 1);
      t.xp[i] = a.x + static_cast<size_t>(max(q8_source<GATHER>(a, blk.row0 + m), 0)) * a.K;
    }
    q8_tile_pick<MT, WM, WN, NT, R, WCOPY, XCOPY, GROUPED, GATHER, SWIGLU>(mt, a, blk, m0, v0, t, b0, b1, b2, b3);
    // before the next rows' copies the buffers have been read, and this wave's
    // stores are out of the count that the copies are waited for by
    copies_barrier<0>();
  }
}

int cdiv(int a, int b) { return (a + b - 1) / b; }

template <int W, int CT, int MT, bool GROUPED, bool GATHER, bool SWIGLU>
void launch_stream(const Q8Args& a, int blocks, hipStream_t s) {
  const long long n = static_cast<long long>(blocks) * cdiv(a.N, CT * 16);
  hipLaunchKernelGGL((q8_stream_kernel<W, CT, MT, GROUPED, GATHER, SWIGLU>), dim3(static_cast<unsigned>(n)),
                     dim3(64 * W), 0, s, a);
}

template <int WM, int WN, int MT, int NT, int R, bool GROUPED, bool GATHER, bool SWIGLU>
void launch_tile(const Q8Args& a, int blocks, hipStream_t s) {
  const long long tiles = static_cast<long long>(blocks) * cdiv(a.N, WN * NT * 32);
  hipLaunchKernelGGL((q8_tile_kernel<WM, WN, MT, NT, R, GROUPED, GATHER, SWIGLU>),
                     grid_of(static_cast<unsigned>((tiles + 7) / 8 * 8)), dim3(64 * WM * WN), 0, s, a);
}

// Which kernel.  Every one of them takes any block of a map (rows past its tile
// go in another pass over the weights), so the choice is speed alone.
//
// Dense: few rows stream the weights, with narrower workgroups where there are
// few columns (1 x 2048 x 2048: 16 columns a workgroup 3.3 us, 32 columns 4.1);
// else the largest tile that still gives every CU (256) a workgroup, and below
// that the smallest tile, with four buffers in flight where even those are few.
// Measured at K = 2048, us:        64x8192  333x2048  333x8192  1000x8192  2048x2048
//   64 x 64, four buffers              8.8       8.6      17.7       39.1       21.3
//   64 x 64, two buffers              11.4      11.0      13.8       32.1       18.1
//   128 x 128                         12.9      12.3      16.1       23.7       17.2
// and 16384x8192: 256 x 256 260 (2.1 PFLOP/s; 2.4 at 8192 cubed), 128 x 128 335.
// The rule counts tiles, not rows: 64 rows of 65536 columns take the largest tile
// (34 us), although the other two are faster there (31 and 32).
hipError_t launch_dense(const Q8Args& a, hipStream_t s) {
  const auto tiles = [&](int bm, int bn) { return static_cast<long long>(cdiv(a.rows, bm)) * cdiv(a.N, bn); };
  if (a.rows <= 16) {
    if (a.N <= 32 * 256)
      launch_stream<4, 1, 1, false, false, false>(a, 1, s);
    else
      launch_stream<4, 2, 1, false, false, false>(a, 1, s);
  } else if (a.rows <= 32) {
    launch_stream<4, 2, 2, false, false, false>(a, 1, s);
  } else if (tiles(256, 256) >= 256) {
    launch_tile<2, 4, 4, 2, 2, false, false, false>(a, cdiv(a.rows, 256), s);
  } else if (tiles(128, 128) >= 256) {
    launch_tile<2, 2, 2, 2, 2, false, false, false>(a, cdiv(a.rows, 128), s);
  } else if (tiles(64, 64) > 512) {
    launch_tile<2, 2, 1, 1, 2, false, false, false>(a, cdiv(a.rows, 64), s);
  } else {
    launch_tile<2, 2, 1, 1, 4, false, false, false>(a, cdiv(a.rows, 64), s);
  }
  return hipGetLastError();
}

// Grouped: the map is only known on the device, so the choice goes by the rows
// an expert holds in the mean and by the tallest block to expect: the shared
// expert holds every token, another expert a few times the mean, and the map
// cuts both at tile_m_max.  A block taller than the kernel's tile takes several
// passes and ends last; a tile much taller than the blocks holds less of the
// weights in flight.  Measured on 256 experts of 2048 x 512, eight each and a
// shared one, us by tokens/tile_m_max:
//               128/128  256/128  512/32  512/128  1024/128  2048/128  2048/256  4096/256  16384/256
//   gate/up (1024 columns, K = 2048)
//   stream           98      129     154      179       272       458       509       868
//   32 x 128         97      111     104      130       173       267       291       485       878
//   64 x 256         80       90     101      103       135       173       190       287       537
//   128 x 128        85       90     112       95       112       131       139       185       477
//   256 x 256        90       95     118      101       120       140       138       168       411
//   down (2048 columns, K = 512)
//   stream           49       63      80       88       136       231       250       437
//   32 x 128         50       56      58       68        91       140       156       253       508
//   64 x 256         49       52      60       60        73        94       103       159       366
//   128 x 128        50       57      74       64        70        81        84       127       372
//   256 x 256        52       60      77       66        73        83        82       121       333
// (gate/up of 128 tokens in blocks of at most 32: stream 82, 32 x 128 74; of 512 in
// blocks of at most 16: 146, 122; of 4096 in blocks of at most 128: 128 x 128 176,
// 256 x 256 194.)  Weights that are read once are copied past the caches (512/32:
// gate/up 105 us -> 100, down 61 -> 57).
template <bool GATHER, bool SWIGLU>
hipError_t launch_grouped(const moe_dims& d, const Q8Args& a, hipStream_t s) {
  const int mean = cdiv(d.T * d.k, d.E);
  const int tallest = std::min(d.tile_m_max, d.n_shared ? std::max(d.T, mean) : 4 * mean);
  if (tallest <= 16 && mean <= 4)
    launch_stream<4, 2, 1, true, GATHER, SWIGLU>(a, a.max_blocks, s);
  else if (tallest <= 32)
    launch_tile<1, 2, 1, 2, 2, true, GATHER, SWIGLU>(a, a.max_blocks, s);
  else if (tallest <= 64 || mean <= 8)
    launch_tile<1, 4, 2, 2, 2, true, GATHER, SWIGLU>(a, a.max_blocks, s);
  else if (tallest <= 128 || mean <= 32)
    launch_tile<2, 2, 2, 2, 2, true, GATHER, SWIGLU>(a, a.max_blocks, s);
  else
    launch_tile<2, 4, 4, 2, 2, true, GATHER, SWIGLU>(a, a.max_blocks, s);
  return hipGetLastError();
}

int validate_grouped(const moe_route_out* r, const void* xq, const void* xs, const void* out) {
  int rc = validate_route_out(r, false);
  if (rc) return rc;
  if (!xq || !xs || !out) return MOE_EINVAL;
  if (!aligned(xq, 16) || !aligned(xs, 4) || !aligned(out, 16)) return MOE_EALIGN;
  return MOE_OK;
}

int validate_half(const int8_t* w, const float* s) {
  if (!w || !s) return MOE_EINVAL;
  return aligned(w, 16) && aligned(s, 16) ? MOE_OK : MOE_EALIGN;
}

Q8Args grouped_args(const moe_dims& d, const moe_route_out* r, const int8_t* xq, const float* xs,
                    void* out, int width) {
  Q8Args a{};
  a.x = xq;
  a.xs = xs;
  a.out = out;
  a.rows = d.T * (d.k + d.n_shared);
  a.type = MOE_ELEM_BF16;
  a.stream_out = static_cast<size_t>(a.rows) * width * 2 > kStreamStore;
  a.blocks = r->blocks;
  a.n_blocks = r->n_blocks;
  a.sorted_slot = r->sorted_slot;
  a.status = r->status;
  a.stream_w = cdiv(d.T * d.k, d.E) <= d.tile_m_max;
  a.max_blocks = max_blocks_of(d);
  a.E = d.E;
  a.T = d.T;
  a.k = d.k;
  a.n_shared = d.n_shared;
  a.tile_m_max = d.tile_m_max;
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
  if (d->M == 0) return MOE_OK;
  if (!xq || !xs || !wq || !ws || !out) return MOE_EINVAL;
  if (!aligned(xq, 16) || !aligned(xs, 4) || !aligned(wq, 16) || !aligned(ws, 16) || !aligned(out, 16))
    return MOE_EALIGN;
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
  a.stream_out = static_cast<size_t>(d->M) * d->N * elem_bytes(d->type) > kStreamStore;
  (void)hipGetLastError();
  return launched(launch_dense(a, static_cast<hipStream_t>(stream)));
}

int moe_q8_gate_up(const moe_dims* d, const int8_t* xq, const float* xs, const moe_route_out* r,
                   const moe_q8_bank* routed, const moe_q8_bank* shared, uint16_t* h, void* stream) {
  int rc = validate_dims(d);
  if (rc || d->T == 0) return rc;
  if ((rc = validate_grouped(r, xq, xs, h))) return rc;
  if (!routed || (d->n_shared && !shared)) return MOE_EINVAL;
  if ((rc = validate_half(routed->gu, routed->gu_s))) return rc;
  if (d->n_shared && (rc = validate_half(shared->gu, shared->gu_s))) return rc;
  if ((rc = check_device())) return rc;
  Q8Args a = grouped_args(*d, r, xq, xs, h, d->I);
  a.w = routed->gu;
  a.ws = routed->gu_s;
  a.w_shared = d->n_shared ? shared->gu : nullptr;
  a.ws_shared = d->n_shared ? shared->gu_s : nullptr;
  a.N = 2 * d->I;
  a.K = d->H;
  (void)hipGetLastError();
  return launched(launch_grouped<true, true>(*d, a, static_cast<hipStream_t>(stream)));
}

int moe_q8_down(const moe_dims* d, const moe_route_out* r, const moe_q8_bank* routed,
                const moe_q8_bank* shared, const int8_t* hq, const float* hs, uint16_t* y_slots,
                void* stream) {
  int rc = validate_dims(d);
  if (rc || d->T == 0) return rc;
  if ((rc = validate_grouped(r, hq, hs, y_slots))) return rc;
  if (!routed || (d->n_shared && !shared)) return MOE_EINVAL;
  if ((rc = validate_half(routed->dn, routed->dn_s))) return rc;
  if (d->n_shared && (rc = validate_half(shared->dn, shared->dn_s))) return rc;
  if ((rc = check_device())) return rc;
  Q8Args a = grouped_args(*d, r, hq, hs, y_slots, d->H);
  a.w = routed->dn;
  a.ws = routed->dn_s;
  a.w_shared = d->n_shared ? shared->dn : nullptr;
  a.ws_shared = d->n_shared ? shared->dn_s : nullptr;
  a.N = d->H;
  a.K = d->I;
  (void)hipGetLastError();
  return launched(launch_grouped<false, false>(*d, a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
