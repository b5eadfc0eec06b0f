// 8-bit integer linear and gated half, for one weight or for ragged groups of rows with a
// weight (an expert) each:
//   y[i][j] = xs[r] ws[e][j] sum_k xq[r][k] wq[e][j][k],  r = rows[i], e the expert of row i.
// The sums are exact 32-bit integers that stay in the matrix instruction's accumulators from
// the first input to the last; both scales are applied once, to the finished sum.  Outputs
// are the instruction's rows and tokens its columns, so that a lane holds one token.
#include "int8.h"
#include "int8_plan.h"

namespace mbq {
namespace {

struct Args {
  const uint8_t* codes;  // packed tiles
  const float* ws;       // weight scales [experts][16 rbs], in the tiles' order
  const uint8_t* xq;     // activation codes, rows of ldq bytes, xlim of them readable
  const float* xs;       // activation scales [t]
  const void* x;         // float activations, rows of ldx elements (quantized in the kernel)
  void* y;
  int32_t* part;           // split K: sums [chunks][p][16 rbs], joined by a second launch
  const int32_t* offsets;  // first row of every expert [experts + 1]
  const int32_t* rows;     // the row of x behind a row of y [p], or NULL: the same
  int64_t ldq, ldx, stride;
  int32_t t, p, n, k, kb, rbs, xlim, experts, chunks, chunk_kb;
  bool gelu, y_bf16;
};

// Rows first .. first + count - 1 of y belong to a tile of one expert.
struct Tile {
  int expert, first, count;
};

// The tile-th tile of at most T rows, counted through the experts in their order.  Offsets
// are data: whatever they hold, the rows found lie in 0 .. p - 1.
template <int T>
__device__ __forceinline__ Tile find_tile(const Args& a, int tile) {
  const int lane = threadIdx.x & 63;
  for (int e0 = 0; e0 < a.experts; e0 += 64) {
    int lo = 0, hi = 0;
    if (e0 + lane < a.experts) {
      lo = min(max(a.offsets[e0 + lane], 0), a.p);
      hi = min(max(a.offsets[e0 + lane + 1], lo), a.p);
    }
    const int tiles = (hi - lo + T - 1) / T, upto = scan64(tiles);
    const uint64_t past = __ballot(tile < upto);
    if (past) {
      const int l = __builtin_ctzll(past);
      const int first = __builtin_amdgcn_readlane(lo, l) + (tile - __builtin_amdgcn_readlane(upto - tiles, l)) * T;
      return {e0 + l, first, min(T, __builtin_amdgcn_readlane(hi, l) - first)};
    }
    tile -= __builtin_amdgcn_readlane(upto, 63);
  }
  return {0, 0, 0};
}

// The row of x behind row i of y; there says whether it has one (an index outside x makes a row of zeros).
__device__ __forceinline__ int source(const Args& a, int i, bool& there) {
  const int r = a.rows ? a.rows[i] : i;
  there = uint32_t(r) < uint32_t(a.t);
  return there ? r : 0;
}

// 16 bytes a lane from its own address to LDS (see to_lds).
__device__ __forceinline__ void to_lds_from(const uint8_t* p, const void* l) {
  const uint32_t at = uint32_t(uintptr_t((const __attribute__((address_space(3))) void*)l));
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"{m0}"(at), "v"(p) : "memory");
}

template <int P>
__device__ __forceinline__ void finish(const Args& a, int64_t row, int rb, int c, const i32x4_t (&sum)[P], float xs, const float* ws) {
  float v[P][4];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const f32x4_t w = *reinterpret_cast<const f32x4_t*>(ws + (rb + i) * kRowBlock + 4 * c);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[i][e] = float(sum[i][e]) * (xs * w[e]);
  }
  if constexpr (P == 2) {
    if (a.gelu) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[0][e] = gated<MBQ_ACT_GELU_TANH>(v[0][e], v[1][e]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[0][e] = gated<MBQ_ACT_SILU>(v[0][e], v[1][e]);
    }
  }
  if (a.y_bf16) store4<true>(a.y, row, a.n, rb / P * kRowBlock + 4 * c, v[0]);
  else store4<false>(a.y, row, a.n, rb / P * kRowBlock + 4 * c, v[0]);
}

// Tiles of 16 RN WN packed rows x 16 RT WT tokens on WN x WT waves (16 RN rows x 16 RT tokens
// each); both operands go through NS LDS buffers of 128 inputs.  A block is two halves of 64
// inputs.  While a half's products run, the next half's operands are read from LDS; the
// barrier stands between the halves, where the block's buffer has been read to its end and
// the next block's copies, a whole block old, are in, and frees the buffer for a new copy.
template <int WN, int WT, int RN, int RT, int NS, int P, bool GROUPED>
__global__ __launch_bounds__(64 * WN * WT, 1) void gemm_kernel(Args a) {
  constexpr int kWaves = WN * WT, kRb = WN * RN, kTb = WT * RT, kTok = 16 * kTb;
  constexpr int kCopiesW = 2 * kRb / kWaves, kCopiesX = 2 * kTb / kWaves;  // a wave's 1 KiB copies to LDS a block
  constexpr int kCopies = kCopiesW + kCopiesX;
  static_assert(RN % P == 0, "a gate tile and its up tile in one wave");
  static_assert(2 * kRb % kWaves == 0 && 2 * kTb % kWaves == 0, "every wave makes as many copies as the waits count");
  __shared__ __align__(1024) uint8_t lds[NS][(kRb + kTb) * kFp8TileBytes];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, c = lane >> 4;
  const int wn = wave % WN, wt = wave / WN;
  // neighbouring tiles on one XCD
  const int tiles_n = (a.rbs + kRb - 1) / kRb;
  const int per = gridDim.x / 8, rest = gridDim.x % 8, xcd = blockIdx.x % 8;
  const int wg = blockIdx.x / 8 + xcd * per + min(xcd, rest);
  const int chunk = GROUPED ? 0 : wg % a.chunks, id = GROUPED ? wg : wg / a.chunks;
  const int kb0 = chunk * a.chunk_kb, kb1 = min(kb0 + a.chunk_kb, a.kb);
  Tile tile;
  int rb0;
  if constexpr (GROUPED) {
    rb0 = id % tiles_n * kRb;
    tile = find_tile<kTok>(a, id / tiles_n);
    if (tile.count == 0) return;
  } else {  // four token tiles by as many row tiles as it takes
    const int tiles_t = (a.t + kTok - 1) / kTok;
    const int group = id / (4 * tiles_n), gt = min(4, tiles_t - 4 * group), in = id - group * 4 * tiles_n;
    rb0 = in / gt * kRb;
    const int first = (4 * group + in % gt) * kTok;
    tile = {0, first, min(kTok, a.t - first)};
  }
  const uint8_t* codes = a.codes + int64_t(tile.expert) * a.stride;
  const float* ws = a.ws + int64_t(tile.expert) * a.rbs * kRowBlock;

  const uint8_t* wp[kCopiesW];
#pragma unroll
  for (int i = 0; i < kCopiesW; ++i) {
    const int half = i * kWaves + wave;
    wp[i] = codes + int64_t(min(rb0 + (half >> 1), a.rbs - 1)) * a.kb * kFp8TileBytes + (half & 1) * 1024;
  }
  // A copy takes eight whole 128-byte rows of codes.  Row r's 16-byte piece p goes to place
  // p ^ (r mod 8), so that the eight rows an operand read takes at once lie in different banks.
  const int col = 16 * ((lane & 7) ^ (lane >> 3));  // of this lane's bytes in a block (the same in all its copies)
  const uint8_t* xp[kCopiesX];
#pragma unroll
  for (int i = 0; i < kCopiesX; ++i) {
    bool there;
    xp[i] = a.xq + source(a, tile.first + min((i * kWaves + wave) * 8 + (lane >> 3), tile.count - 1), there) * a.ldq;
  }
  const int xread = r * 128 + 16 * (c ^ (r & 7));  // the lane's first half of an operand in a tile

  auto copy_x = [&](int kb, int buf) __attribute__((always_inline)) {
    // past the end of a row of codes (k no multiple of 128) the lane copies the row's first
    // bytes: they meet weight codes of 0
    const int at = kb * kFp8Block + col;
    const int off = at < a.xlim ? at : 0;
#pragma unroll
    for (int i = 0; i < kCopiesX; ++i) to_lds_from(xp[i] + off, &lds[buf][(2 * kRb + i * kWaves + wave) * 1024]);
  };
  auto copy_w = [&](int kb, int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kCopiesW; ++i)
      to_lds<16>(wp[i] + int64_t(kb) * kFp8TileBytes, uint32_t(lane) * 16, &lds[buf][(i * kWaves + wave) * 1024]);
  };

  i32x4_t acc[RN][RT];
#pragma unroll
  for (int i = 0; i < RN; ++i)
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};
  u32x4_t w[2][RN], x[2][RT];
  auto read_w = [&](int buf, int half, int i) __attribute__((always_inline)) {
    w[half][i] = *(reinterpret_cast<const u32x4_t*>(&lds[buf][(wn * RN + i) * kFp8TileBytes + half * 1024]) + lane);
  };
  auto read_x = [&](int buf, int half, int j) __attribute__((always_inline)) {
    x[half][j] = *reinterpret_cast<const u32x4_t*>(&lds[buf][(kRb + wt * RT + j) * kFp8TileBytes + (xread ^ (64 * half))]);
  };
  auto products = [&](int half) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < RN; ++i)
#pragma unroll
      for (int j = 0; j < RT; ++j) acc[i][j] = mfma_i8(w[half][i], x[half][j], acc[i][j]);
  };
  auto read = [&](int buf, int half) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < RT; ++j) read_x(buf, half, j);
#pragma unroll
    for (int i = 0; i < RN; ++i) read_w(buf, half, i);
  };

  // One path without tests: past the end the last block is copied again, to a buffer that no
  // one reads, so that the copies on their way are always as many as the waits count.
  auto copy = [&](int kb, int buf) __attribute__((always_inline)) {
    copy_x(min(kb, kb1 - 1), buf);
    copy_w(min(kb, kb1 - 1), buf);
  };
#pragma unroll
  for (int i = 0; i < NS; ++i) copy(kb0 + i, i);
  to_lds_wait<(NS - 1) * kCopies>();
  __syncthreads();
  read(0, 0);
  int buf = 0;
  for (int kb = kb0; kb < kb1 - 1; ++kb) {
    read(buf, 1);
    products(0);
    const int next = buf == NS - 1 ? 0 : buf + 1;
    to_lds_wait<(NS - 2) * kCopies>();  // block kb + 1 is in
    __syncthreads();
    read(next, 0);
    copy(kb + NS, buf);
    products(1);
    buf = next;
  }
  read(buf, 1);
  products(0);
  products(1);
  to_lds_wait<0>();  // none of them outlives the workgroup

  const int rbw = rb0 + wn * RN;
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    const int in = (wt * RT + j) * 16 + r;
    if (in >= tile.count) continue;
    const int64_t row = tile.first + in;
    if (!GROUPED && a.chunks > 1) {
      int32_t* sums = a.part + (int64_t(chunk) * a.p + row) * a.rbs * kRowBlock + 4 * c;
#pragma unroll
      for (int i = 0; i < RN; ++i)
        if (rbw + i < a.rbs) *reinterpret_cast<i32x4_t*>(sums + (rbw + i) * kRowBlock) = acc[i][j];
      continue;
    }
    bool there;
    const int from = source(a, int(row), there);
    const float xs = there ? a.xs[from] : 0.f;
#pragma unroll
    for (int i = 0; i < RN; i += P) {
      i32x4_t sum[P];
#pragma unroll
      for (int e = 0; e < P; ++e) sum[e] = acc[i + e][j];
      if (rbw + i < a.rbs) finish<P>(a, row, rbw + i, c, sum, xs, ws);
    }
  }
}

// Joins the chunks of a split K: four outputs of one token a thread.
template <int P>
__global__ __launch_bounds__(256) void join_kernel(Args a) {
  const int quads = a.rbs / P * 4;
  const int64_t stride = int64_t(a.p) * a.rbs * kRowBlock;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < int64_t(a.p) * quads; i += int64_t(gridDim.x) * 256) {
    const int token = int(i / quads), q = int(i - int64_t(token) * quads);
    const int rb = (q >> 2) * P, c = q & 3;
    const int32_t* from = a.part + int64_t(token) * a.rbs * kRowBlock + rb * kRowBlock + 4 * c;
    i32x4_t sum[P];
#pragma unroll
    for (int e = 0; e < P; ++e) sum[e] = *reinterpret_cast<const i32x4_t*>(from + kRowBlock * e);
    for (int s = 1; s < a.chunks; ++s)
#pragma unroll
      for (int e = 0; e < P; ++e) sum[e] += *reinterpret_cast<const i32x4_t*>(from + s * stride + kRowBlock * e);
    finish<P>(a, token, rb, c, sum, a.xs[token], a.ws);
  }
}

// Few tokens: a workgroup streams one row block (gated: the pair) for a tile of at most 16 TT
// tokens; its W waves take every W-th 128-input block, and their sums meet in LDS.  A wave has
// U blocks in its registers and the next U on their way; a block past the end is the last one
// again, met by activations of 0, so that no load stands behind a test.
// XT: the type of x.  Codes (MBQ_INT8) are read from memory; a few float tokens are quantized
// here, once a workgroup into LDS, which saves the quantizing launch.
template <int W, int TT, int XT, int P, bool GROUPED>
__global__ __launch_bounds__(64 * W) void stream_kernel(Args a) {
  constexpr int U = (TT * P >= 4 ? 1 : TT * P == 2 ? 2 : 4) * 8 / W > 0 ? (TT * P >= 4 ? 1 : TT * P == 2 ? 2 : 4) * 8 / W : 1;
  constexpr bool kInline = XT != MBQ_INT8;
  static_assert(!kInline || TT == 1, "a few tokens");
  extern __shared__ __align__(16) uint8_t lx[];  // inline: codes, rows 16 bytes apart in banks
  __shared__ i32x4_t red[W][P * TT][64];
  __shared__ uint32_t amax[kInline ? 16 : 1][W];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, c = lane >> 4;
  const int rb0 = blockIdx.x * P;
  Tile tile{0, 0, a.t};
  if constexpr (GROUPED) {
    tile = find_tile<16 * TT>(a, blockIdx.y);
    if (tile.count == 0) return;
  }
  const uint8_t* wp = a.codes + int64_t(tile.expert) * a.stride + int64_t(rb0) * a.kb * kFp8TileBytes + lane * 16;
  const float* ws = a.ws + int64_t(tile.expert) * a.rbs * kRowBlock;
  const int ldl = a.kb * kFp8Block + 16;
  const uint8_t* xp[TT];
  float xs[TT];
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    const int in = min(j * 16 + r, tile.count - 1);
    if constexpr (kInline) {
      xp[j] = lx + in * ldl + 16 * c;
    } else {
      bool there;
      const int from = source(a, tile.first + in, there);
      xp[j] = a.xq + from * a.ldq;
      xs[j] = there ? a.xs[from] : 0.f;
    }
  }
  u32x4_t wf[2][U][P][2], xf[2][U][TT][2];
  auto load = [&](int s, int k0) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = min(k0 + u * W, a.kb - 1);
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          wf[s][u][i][h] = __builtin_nontemporal_load(
              reinterpret_cast<const u32x4_t*>(wp + (int64_t(i) * a.kb + kb) * kFp8TileBytes + 1024 * h));
      if constexpr (!kInline)
#pragma unroll
        for (int j = 0; j < TT; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int col = kb * kFp8Block + 64 * h + 16 * c;  // past the end of a row: see gemm_kernel
            xf[s][u][j][h] = *reinterpret_cast<const u32x4_t*>(xp[j] + (col < a.xlim ? col : 0));
          }
    }
  };
  i32x4_t acc[P][TT];
#pragma unroll
  for (int i = 0; i < P; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};
  auto products = [&](int s, int k0) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = k0 + u * W;
      const uint32_t keep = kb < a.kb ? ~0u : 0u;
#pragma unroll
      for (int j = 0; j < TT; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          u32x4_t v;
          if constexpr (kInline) v = *reinterpret_cast<const u32x4_t*>(xp[j] + min(kb, a.kb - 1) * kFp8Block + 64 * h);
          else v = xf[s][u][j][h];
          v &= keep;
#pragma unroll
          for (int i = 0; i < P; ++i) acc[i][j] = mfma_i8(wf[s][u][i][h], v, acc[i][j]);
        }
    }
  };

  if constexpr (kInline) {
    constexpr bool kBf = XT == MBQ_BF16;
    const int tid = threadIdx.x;
    Raw8<kBf> ahead;  // the first row's, asked for before the weight
    auto row_of = [&](int i, bool& there) __attribute__((always_inline)) {
      return static_cast<const uint8_t*>(a.x) + source(a, tile.first + i, there) * a.ldx * (kBf ? 2 : 4);
    };
    bool there;
    ahead.load(row_of(0, there), tid * 8, a.k);
    load(0, wave);
    for (int i = 0; i < tile.count; ++i) {
      const uint8_t* row = row_of(i, there);
      uint32_t m = 0;
      float v[8];
      if (i == 0) ahead.get(v);
      else load8<kBf>(row, tid * 8, a.k, v);
      m = amax8(v);
      for (int at = (tid + 64 * W) * 8; at < a.k; at += 64 * W * 8) {
        load8<kBf>(row, at, a.k, v);
        m = max(m, amax8(v));
      }
      m = max64(m);
      if (lane == 0) amax[i][wave] = m;
    }
    __syncthreads();
    for (int i = 0; i < tile.count; ++i) {
      const uint8_t* row = row_of(i, there);
      uint32_t m = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) m = max(m, amax[i][w]);
      const float f = int8_factor(m);
      for (int at = tid * 8; at < a.kb * kFp8Block; at += 64 * W * 8) {
        float v[8];
        load8<kBf>(row, at, a.k, v);
        store_int8x8(lx + i * ldl, at, ldl, v, f);
      }
      if (i == min(r, tile.count - 1)) xs[0] = there ? int8_scale(m) : 0.f;
    }
    __syncthreads();
  } else {
    load(0, wave);
  }
  for (int k0 = wave; k0 < a.kb; k0 += 2 * W * U) {
    if (k0 + W * U < a.kb) load(1, k0 + W * U);
    products(0, k0);
    if (k0 + W * U >= a.kb) break;
    if (k0 + 2 * W * U < a.kb) load(0, k0 + 2 * W * U);
    products(1, k0 + W * U);
  }
#pragma unroll
  for (int i = 0; i < P; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) red[wave][i * TT + j][lane] = acc[i][j];
  __syncthreads();
  if (wave >= TT) return;
  // the wave's token tile (its scale without a register index)
  float scale = xs[0];
#pragma unroll
  for (int j = 1; j < TT; ++j) scale = wave == j ? xs[j] : scale;
  const int in = wave * 16 + r;
  i32x4_t sum[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    sum[i] = red[0][i * TT + wave][lane];
#pragma unroll
    for (int w = 1; w < W; ++w) sum[i] += red[w][i * TT + wave][lane];
  }
  if (in < tile.count) finish<P>(a, tile.first + in, rb0, c, sum, scale, ws);
}

template <int WN, int WT, int RN, int RT, int NS, int P, bool GROUPED>
void launch_tiles(const Args& a, hipStream_t stream) {
  const int64_t tiles_n = (a.rbs + WN * RN - 1) / (WN * RN), tok = 16 * WT * RT;
  const int64_t tiles_t = GROUPED ? a.p / tok + std::min(a.experts, a.p) : (a.p + tok - 1) / tok;
  gemm_kernel<WN, WT, RN, RT, NS, P, GROUPED><<<uint32_t(tiles_n * tiles_t * a.chunks), 64 * WN * WT, 0, stream>>>(a);
}

template <int W, int TT, int P, bool GROUPED>
void launch_stream(const Args& a, mbq_dtype x_dtype, hipStream_t stream) {
  const int tok = 16 * TT;
  const dim3 grid(a.rbs / P, GROUPED ? a.p / tok + std::min(a.experts, a.p) : 1), block(64 * W);
  if constexpr (TT == 1) {
    if (a.x) {
      const size_t lds = size_t(std::min(a.p, 16)) * (a.kb * kFp8Block + 16);
      if (x_dtype == MBQ_BF16) stream_kernel<W, 1, MBQ_BF16, P, GROUPED><<<grid, block, lds, stream>>>(a);
      else stream_kernel<W, 1, MBQ_F32, P, GROUPED><<<grid, block, lds, stream>>>(a);
      return;
    }
  }
  stream_kernel<W, TT, MBQ_INT8, P, GROUPED><<<grid, block, 0, stream>>>(a);
}

template <int P, bool GROUPED>
hipError_t launch(Args& a, const Int8Plan& p, mbq_dtype x_dtype, hipStream_t stream) {
  a.chunks = p.chunks;
  a.chunk_kb = (a.kb + p.chunks - 1) / p.chunks;
  switch (p.form) {
    case Int8Form::kStream8x1: launch_stream<8, 1, P, GROUPED>(a, x_dtype, stream); break;
    case Int8Form::kStream16x1: launch_stream<16, 1, P, GROUPED>(a, x_dtype, stream); break;
    case Int8Form::kStream8x2: launch_stream<8, 2, P, GROUPED>(a, x_dtype, stream); break;
    case Int8Form::kStream8x4: launch_stream<8, 4, P, GROUPED>(a, x_dtype, stream); break;
    case Int8Form::k256x256: launch_tiles<2, 4, 8, 4, 2, P, GROUPED>(a, stream); break;
    case Int8Form::k256x128: launch_tiles<2, 2, 8, 4, 3, P, GROUPED>(a, stream); break;
    case Int8Form::k128x128: launch_tiles<2, 2, 4, 4, 3, P, GROUPED>(a, stream); break;
    case Int8Form::k128x64: launch_tiles<2, 2, 4, 2, 3, P, GROUPED>(a, stream); break;
    case Int8Form::k64x64: launch_tiles<2, 2, 2, 2, 3, P, GROUPED>(a, stream); break;
    case Int8Form::k64x32: launch_tiles<2, 2, 2, 1, 3, P, GROUPED>(a, stream); break;
  }
  if (a.chunks > 1)
    join_kernel<P><<<uint32_t(std::min<int64_t>((int64_t(a.p) * (a.rbs / P) * 4 + 255) / 256, 4096)), 256, 0, stream>>>(a);
  return hipGetLastError();
}

template <int P>
hipError_t launch(Args& a, const Int8Plan& p, mbq_dtype x_dtype, hipStream_t stream) {
  return a.offsets ? launch<P, true>(a, p, x_dtype, stream) : launch<P, false>(a, p, x_dtype, stream);
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

Int8Plan plan_of(const mbq_int8_desc& d, int32_t t, int32_t p, bool grouped, mbq_dtype x_dtype) {
  return plan_int8(t, p, grouped ? d.experts : 0, d.row_blocks / (d.gated + 1), d.gated + 1, d.k_blocks, x_dtype == MBQ_INT8);
}

// Workspace: the activations' codes and scales (codes given in rows that hold no whole 16
// bytes: only their copy), then the partial sums of a split K.
struct Layout {
  size_t codes, scales, part;
};
Layout layout(const mbq_int8_desc& d, int32_t t, int32_t p, const Int8Plan& plan, mbq_dtype x_dtype) {
  Layout l{};
  const size_t codes = align256(size_t(t) * d.k_blocks * kFp8Block);
  if (x_dtype == MBQ_INT8) l.codes = d.k % 16 ? codes : 0;
  else if (!plan.inline_x) l.codes = codes, l.scales = align256(size_t(t) * 4);
  if (plan.chunks > 1) l.part = size_t(plan.chunks) * p * d.row_blocks * kRowBlock * 4;
  return l;
}

}  // namespace

size_t int8_workspace(const mbq_int8_desc& d, int32_t t, int32_t p, bool grouped, mbq_dtype x_dtype) {
  if (t == 0 || p == 0) return 0;
  const Layout l = layout(d, t, p, plan_of(d, t, p, grouped, x_dtype), x_dtype);
  return l.codes + l.scales + l.part;
}

hipError_t launch_int8_linear(const mbq_int8_desc& d, const void* packed, const mbq_int8_args& g, hipStream_t stream) {
  const mbq_dtype x_dtype = mbq_dtype(g.x_dtype);
  const Int8Plan plan = plan_of(d, g.t, g.p, g.offsets != nullptr, x_dtype);
  const Layout l = layout(d, g.t, g.p, plan, x_dtype);
  uint8_t* ws = static_cast<uint8_t*>(g.workspace);
  Args a{};
  a.codes = static_cast<const uint8_t*>(packed);
  a.ws = reinterpret_cast<const float*>(a.codes + d.scales_offset);
  a.y = g.y;
  a.part = reinterpret_cast<int32_t*>(ws + l.codes + l.scales);
  a.offsets = g.offsets;
  a.rows = g.rows;
  a.stride = int64_t(d.expert_stride);
  a.t = g.t;
  a.p = g.p;
  a.n = d.n;
  a.k = d.k;
  a.kb = d.k_blocks;
  a.rbs = d.row_blocks;
  a.experts = d.experts;
  hipError_t e = hipSuccess;
  if (x_dtype == MBQ_INT8) {
    a.xs = g.x_scale;
    if (l.codes) {
      e = launch_fp8_pad_codes(g.t, d.k, g.x, g.ldx, ws, stream);
      a.xq = ws;
      a.ldq = a.xlim = d.k_blocks * kFp8Block;
    } else {
      a.xq = static_cast<const uint8_t*>(g.x);
      a.ldq = g.ldx;
      a.xlim = d.k;
    }
  } else if (plan.inline_x) {
    a.x = g.x;
    a.ldx = g.ldx;
  } else {
    float* scales = reinterpret_cast<float*>(ws + l.codes);
    a.ldq = a.xlim = d.k_blocks * kFp8Block;
    e = launch_int8_quantize(g.t, d.k, g.x, x_dtype == MBQ_BF16, g.ldx, ws, a.ldq, true, scales, stream);
    a.xq = ws;
    a.xs = scales;
  }
  if (e != hipSuccess) return e;
  a.gelu = d.gated && g.act == MBQ_ACT_GELU_TANH;
  a.y_bf16 = g.y_dtype == MBQ_BF16;
  return d.gated ? launch<2>(a, plan, x_dtype, stream) : launch<1>(a, plan, x_dtype, stream);
}

}  // namespace mbq
