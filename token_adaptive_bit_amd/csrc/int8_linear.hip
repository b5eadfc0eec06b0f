// 8-bit integer linear and gated half, for one weight or for ragged groups of rows with a
// weight (an expert) each:
//   y[i][j] = xs[r] ws[e][j] sum_k xq[r][k] wq[e][j][k],  r = rows[i], e the expert of row i.
// The sums are exact 32-bit integers that stay in the matrix instruction's accumulators from
// the first input to the last; both scales are applied once, to the finished sum.  Outputs
// are the instruction's rows and tokens its columns, so that a lane holds one token.
#include "int8.h"
#include "int8_plan.h"

#include <type_traits>

namespace mbq {
namespace {

constexpr int kUnits = 256;  // compute units
constexpr int kCutRoom = kInt8CutRoom;

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

// The experts' rows, and their tiles of at most T rows counted through the experts in their
// order.  Offsets are data: whatever they hold, the rows found lie in 0 .. p - 1.
template <int T>
__device__ __forceinline__ int tiles_at(const Args& a, int e, int& lo, int& hi) {
  lo = hi = 0;
  if (e < a.experts) {
    lo = min(max(a.offsets[e], 0), a.p);
    hi = min(max(a.offsets[e + 1], lo), a.p);
  }
  return (hi - lo + T - 1) / T;
}
template <int T>
__device__ __forceinline__ int count_tiles(const Args& a) {
  int tiles = 0, lo, hi;
#pragma unroll 4
  for (int e = threadIdx.x & 63; e < a.experts; e += 64) tiles += tiles_at<T>(a, e, lo, hi);
  return __builtin_amdgcn_readlane(scan64(tiles), 63);
}
// The expert that a tile belongs to: its rows, and the number of its first tile.
struct Group {
  int expert, first, count, tile0;
};
template <int T>
__device__ __forceinline__ Group find_group(const Args& a, int tile) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int e0 = 0; e0 < a.experts; e0 += 64) {
    int lo, hi;
    const int tiles = tiles_at<T>(a, e0 + lane, lo, hi), upto = before + scan64(tiles);
    const uint64_t past = __ballot(tile < upto);
    if (past) {
      const int l = __builtin_ctzll(past), first = __builtin_amdgcn_readlane(lo, l);
      return {e0 + l, first, __builtin_amdgcn_readlane(hi, l) - first, __builtin_amdgcn_readlane(upto - tiles, l)};
    }
    before = __builtin_amdgcn_readlane(upto, 63);
  }
  return {0, 0, 0, 0};
}
// The part-th tile of a group.
template <int T>
__device__ __forceinline__ Tile tile_of(const Group& g, int part) { return {g.expert, g.first + part * T, min(T, g.count - part * T)}; }

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

// A sum times its token's and then its output's scale: the first product is at most 2^31 times
// the token's scale, and with that in 2^-126 .. 2^97 it is 0 or a normal number, so that nothing
// is lost before the last product, whatever the output's scale.  For other tokens (FAR) the
// mantissas are multiplied, and the exponents come last.  Where both forms serve they give
// the same bits.
template <bool FAR>
__device__ __forceinline__ float scaled(int32_t sum, float xs, float ws) {
  if constexpr (!FAR) return float(sum) * xs * ws;
  return __builtin_ldexpf(float(sum) * __builtin_amdgcn_frexp_mantf(xs) * __builtin_amdgcn_frexp_mantf(ws),
                          __builtin_amdgcn_frexp_expf(xs) + __builtin_amdgcn_frexp_expf(ws));
}
__device__ __forceinline__ bool far_scale(float xs) {
  return (__float_as_uint(xs) & 0x7FFFFFFFu) - 0x00800000u >= 0x70000000u - 0x00800000u;
}

// As to_lds_wait, where among the N operations that may be on their way COPIES are copies and the
// others loads of the compiler's.  Were one of those moved or taken out, a copy too many could be:
// the build looks in the assembly that of the N youngest vector memory operations at this wait, on
// every way to it, no more are copies (build.py).
template <int N, int COPIES>
__device__ __forceinline__ void counted_wait() {
  asm volatile("s_waitcnt vmcnt(%0) ; at most %1 copies of the youngest %0" ::"n"(N), "n"(COPIES) : "memory");
}

// Four outputs of a token from their sums (gated: from both products').
template <int P, bool FAR>
__device__ __forceinline__ void outputs(const Args& a, const i32x4_t (&sum)[P], float xs, const f32x4_t (&ws)[P], float (&v)[4]) {
  float u[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = scaled<FAR>(sum[0][e], xs, ws[0][e]);
    u[e] = scaled<FAR>(sum[P - 1][e], xs, ws[P - 1][e]);
  }
  if constexpr (P == 2) {
    if (a.gelu) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = gated<MBQ_ACT_GELU_TANH>(v[e], u[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = gated<MBQ_ACT_SILU>(v[e], u[e]);
    }
  }
}

template <int P>
__device__ __forceinline__ void finish(const Args& a, int64_t row, int rb, int c, const i32x4_t (&sum)[P], float xs,
                                       const f32x4_t (&ws)[P]) {
  float v[4];
  outputs<P, true>(a, sum, xs, ws, v);  // of four outputs the other form would save less than its choice costs
  if (a.y_bf16) store4<true>(a.y, row, a.n, rb / P * kRowBlock + 4 * c, v);
  else store4<false>(a.y, row, a.n, rb / P * kRowBlock + 4 * c, v);
}

// A wave's 16 RN / P outputs of 16 RT tokens to y, 16 tokens at a time: from the instruction's
// layout, where a lane holds four outputs of one token, through the wave's own LDS to whole
// rows.  (Stored as they lie, in pieces of 8 bytes, a tile of 256 x 256 took 10 us more.)
template <int RN, int RT, int P, bool YBF, bool FAR>
__device__ __forceinline__ void write_rows(const Args& a, const i32x4_t (&acc)[RN][RT], const float (&xs)[RT],
                                           const f32x4_t (&w)[RN], int rb, int64_t first, int count, uint8_t* lds) {
  constexpr int kBytes = YBF ? 2 : 4, kRow = RN / P * kRowBlock * kBytes, kPieces = kRow / 16, kStride = kRow + 16;
  const int lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    if (j * 16 >= count) break;
#pragma unroll
    for (int i = 0; i < RN; i += P) {
      i32x4_t sum[P];
      f32x4_t scale[P];
#pragma unroll
      for (int e = 0; e < P; ++e) {
        sum[e] = acc[i + e][j];
        scale[e] = w[i + e];
      }
      float v[4];
      outputs<P, FAR>(a, sum, xs[j], scale, v);
      uint8_t* at = lds + r * kStride + (i / P * kRowBlock + 4 * c) * kBytes;
      if constexpr (YBF) {
        *reinterpret_cast<uint64_t*>(at) = uint64_t(bf16_pair(v[2], v[3])) << 32 | bf16_pair(v[0], v[1]);
      } else {
        *reinterpret_cast<f32x4_t*>(at) = f32x4_t{v[0], v[1], v[2], v[3]};
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int q = lane; q < 16 * kPieces; q += 64) {
      const int token = j * 16 + q / kPieces, col = rb / P * kRowBlock + q % kPieces * (16 / kBytes);
      const u32x4_t piece = *reinterpret_cast<const u32x4_t*>(lds + q / kPieces * kStride + q % kPieces * 16);
      if (token >= count || col >= a.n) continue;
      uint8_t* out = static_cast<uint8_t*>(a.y) + ((first + token) * a.n + col) * kBytes;
      if (col + 16 / kBytes <= a.n) {
        if constexpr (YBF) *reinterpret_cast<u32x4_a2*>(out) = piece;
        else *reinterpret_cast<f32x4_a4*>(out) = __builtin_bit_cast(f32x4_t, piece);
      } else {
#pragma unroll
        for (int e = 0; e < 16 / kBytes; ++e)
          if (col + e < a.n) {
            if constexpr (YBF) reinterpret_cast<uint16_t*>(out)[e] = uint16_t(piece[e / 2] >> (16 * (e & 1)));
            else reinterpret_cast<uint32_t*>(out)[e] = piece[e];
          }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

template <int RN, int RT, int P>
__device__ __forceinline__ void write_tile(const Args& a, const i32x4_t (&acc)[RN][RT], const float (&xs)[RT], const float* ws,
                                           int rb, int64_t first, int count, uint8_t* lds) {
  const int c = (threadIdx.x & 63) >> 4;
  f32x4_t w[RN];  // asked for before the tokens' scales are looked at
#pragma unroll
  for (int i = 0; i < RN; ++i) w[i] = *reinterpret_cast<const f32x4_t*>(ws + min(rb + i, a.rbs - 1) * kRowBlock + 4 * c);
  bool far = false;
#pragma unroll
  for (int j = 0; j < RT; ++j) far |= far_scale(xs[j]);
  if (__builtin_expect(__ballot(far) != 0, 0)) {  // the wave's tokens together
    if (a.y_bf16) write_rows<RN, RT, P, true, true>(a, acc, xs, w, rb, first, count, lds);
    else write_rows<RN, RT, P, false, true>(a, acc, xs, w, rb, first, count, lds);
  } else {
    if (a.y_bf16) write_rows<RN, RT, P, true, false>(a, acc, xs, w, rb, first, count, lds);
    else write_rows<RN, RT, P, false, false>(a, acc, xs, w, rb, first, count, lds);
  }
}

// Many tokens: tiles of 16 RN WN packed rows x 16 RT WT tokens on WN x WT waves (16 RN rows x
// 16 RT tokens each); both operands go through LDS, in NW buffers for the weight and NX for the
// tokens' codes of 128 inputs each.  A block is two halves of 64 inputs.  While a half's
// products run, the next half's operands are read from LDS; the barrier stands between the
// halves, where the block's buffers have been read to their end and the next block's copies
// are in, and frees the buffers for new ones.  The weight, which comes from farther away, has a
// buffer more (256 x 256, 4096 tokens of 3584 x 18944: 205 us from 213; 8 experts of 4096 x 14336,
// 16384 rows: 820 from 865).  256 x 256 fills LDS to its last byte: its reads and copies
// take 2048 clocks a block, as many as the products, which keep the matrix units busy for 83% of
// those 205 us (2.7 P op/s) and 71% of the experts'.  (Four waves of 128 x 128 would read a
// third less, but have no registers for operands that are read ahead.)
// The smaller tiles, 128 x 128 and 256 x 128, take over where the large ones are too few for the
// units and the direct ones too many for the caches: 128 tokens of 18944 x 3584 18.3 us from 20.3,
// 256 tokens of gated 11008 x 4096 32.2 from 35.9, 8 experts of 4096 x 14336 with 1024 rows 116
// from 138.  They too are eight waves: two a SIMD, of which one multiplies while the other waits
// (256 x 128 on four: 43 us instead of 32).
template <int WN, int WT, int RN, int RT, int NW, int NX, int P, bool GROUPED>
__global__ __launch_bounds__(64 * WN * WT, 1) void shared_kernel(Args a) {
  constexpr int kWaves = WN * WT, kRb = WN * RN, kTb = WT * RT, kTok = 16 * kTb;
  constexpr int kCopiesW = 2 * kRb / kWaves, kCopiesX = 2 * kTb / kWaves;  // a wave's 1 KiB copies to LDS a block
  constexpr int kCopies = kCopiesW + kCopiesX;
  static_assert(RN % P == 0, "a gate tile and its up tile in one wave");
  static_assert(2 * kRb % kWaves == 0 && 2 * kTb % kWaves == 0, "every wave makes as many copies as the waits count");
  static_assert(NW >= NX && NX >= 2, "the order of the copies");
  constexpr int kAhead = NW > NX ? kCopiesW : 0;  // copies issued behind the x of one block that belong to later blocks
  __shared__ __align__(1024) uint8_t lds[(NW * kRb + NX * kTb) * kFp8TileBytes];
  uint8_t *lw = lds, *lx = lds + NW * kRb * kFp8TileBytes;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, c = lane >> 4;
  const int wn = wave % WN, wt = wave / WN;
  const int tiles_n = (a.rbs + kRb - 1) / kRb, tiles_t = GROUPED ? count_tiles<kTok>(a) : (a.t + kTok - 1) / kTok;
  // Neighbouring tiles on one XCD, in rounds of one on each unit.  Tiles left over by the last
  // whole round, if they are half a round or less, are cut into halves or quarters of their
  // tokens, which the units share: the last round then takes about 85 or 75% of a whole one (8
  // experts of 4096 x 14336, 16384 rows: 820 us from 848; 18944 x 3584, 1024 tokens 75 from 84).
  const int64_t tiles = min(int64_t(tiles_n) * tiles_t * (GROUPED ? 1 : a.chunks), int64_t(gridDim.x) - kCutRoom);
  const int left = int(tiles % kUnits), cut = tiles < kUnits || left == 0 || left > kUnits / 2 ? 1 : left > kUnits / 4 ? 2 : 4;
  const int64_t whole = cut > 1 ? tiles - left : tiles;
  const int xcd = blockIdx.x % 8;
  int64_t wg;
  int part = 0;
  if (int64_t(blockIdx.x) < whole) {
    wg = blockIdx.x / 8 + xcd * (whole / 8) + min(xcd, int(whole % 8));
  } else {
    const int b = int(blockIdx.x - whole) / 8;
    wg = whole + b / cut * 8 + xcd;
    part = b % cut;
    if (cut == 1 || wg >= tiles) return;
  }
  const int chunk = GROUPED ? 0 : int(wg % a.chunks), id = GROUPED ? int(wg) : int(wg / a.chunks);
  const int kb0 = chunk * a.chunk_kb, kb1 = min(kb0 + a.chunk_kb, a.kb);
  Group g{0, 0, a.t, 0};
  if constexpr (GROUPED) g = find_group<kTok>(a, id / tiles_n);
  // four token tiles of an expert by as many row tiles as it takes
  const int local = id - g.tile0 * tiles_n, four = local / (4 * tiles_n), in = local - four * 4 * tiles_n;
  const int gt = min(4, (g.count + kTok - 1) / kTok - 4 * four);
  const int rb0 = in / gt * kRb;
  Tile tile = tile_of<kTok>(g, 4 * four + in % gt);
  if (cut > 1 && int64_t(blockIdx.x) >= whole) {
    tile.first += part * (kTok / cut);
    tile.count = min(tile.count - part * (kTok / cut), kTok / cut);
    if (tile.count <= 0) return;
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

  // The i-th copy of a block, the tokens' first.  One path without tests: past the end the last
  // block is copied again, to a buffer that no one reads, so that the copies on their way are
  // always as many as the waits count.
  auto copy_x = [&](int kb, int buf, int i) __attribute__((always_inline)) {
    // past the end of a row of codes (k no multiple of 128) the lane copies the row's first
    // bytes: they meet weight codes of 0
    const int at = min(kb, kb1 - 1) * kFp8Block + col;
    to_lds_from(xp[i] + (at < a.xlim ? at : 0), lx + buf * (kTb * kFp8TileBytes) + (i * kWaves + wave) * 1024);
  };
  auto copy_w = [&](int kb, int buf, int i) __attribute__((always_inline)) {
    to_lds<16>(wp[i] + int64_t(min(kb, kb1 - 1)) * kFp8TileBytes, uint32_t(lane) * 16,
               lw + buf * (kRb * kFp8TileBytes) + (i * kWaves + wave) * 1024);
  };

  i32x4_t acc[RN][RT];
#pragma unroll
  for (int i = 0; i < RN; ++i)
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};
  u32x4_t w[2][RN], x[2][RT];
  auto read_w = [&](int buf, int half, int i) __attribute__((always_inline)) {
    w[half][i] = *(reinterpret_cast<const u32x4_t*>(lw + (buf * kRb + wn * RN + i) * kFp8TileBytes + half * 1024) + lane);
  };
  auto read_x = [&](int buf, int half, int j) __attribute__((always_inline)) {
    x[half][j] = *reinterpret_cast<const u32x4_t*>(lx + (buf * kTb + wt * RT + j) * kFp8TileBytes + (xread ^ (64 * half)));
  };
  // A half's products, a row of them at a time, and between the rows the reads of the half
  // after it (done two rows before the end) and the copies, one by one: left to itself the
  // compiler puts the reads behind the products and waits for them (8 experts of 4096 x 14336,
  // 16384 rows: 868 us against 820; 4096 tokens of 3584 x 18944 221 against 209).
  auto half = [&](int h, bool reads, int wbuf, int xbuf, auto copy) __attribute__((always_inline)) {
    constexpr int kReads = RN + RT, kEach = RN > 2 ? (kReads + RN - 3) / (RN - 2) : kReads;
#pragma unroll
    for (int i = 0; i < RN; ++i) {
#pragma unroll
      for (int j = 0; j < RT; ++j) acc[i][j] = mfma_i8(w[h][i], x[h][j], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);  // the products first: a read before them would be waited for with theirs
      if (reads)
#pragma unroll
        for (int q = i * kEach; q < (i + 1) * kEach && q < kReads; ++q) {
          if (q < RT) read_x(xbuf, 1 - h, q);
          else read_w(wbuf, 1 - h, q - RT);
        }
      copy(i);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto none = [](int) {};

#pragma unroll
  for (int i = 0; i < NW - NX; ++i)
#pragma unroll
    for (int q = 0; q < kCopiesW; ++q) copy_w(kb0 + i, i, q);
#pragma unroll
  for (int i = 0; i < NX; ++i) {
#pragma unroll
    for (int q = 0; q < kCopiesX; ++q) copy_x(kb0 + i, i, q);
#pragma unroll
    for (int q = 0; q < kCopiesW; ++q) copy_w(kb0 + i + NW - NX, i + NW - NX, q);
  }
  to_lds_wait<(NX - 1) * kCopies + kAhead>();
  __syncthreads();
  int wbuf = 0, xbuf = 0;
  if (wt * RT * 16 < tile.count) {
#pragma unroll
    for (int j = 0; j < RT; ++j) read_x(0, 0, j);
#pragma unroll
    for (int i = 0; i < RN; ++i) read_w(0, 0, i);
    for (int kb = kb0; kb < kb1 - 1; ++kb) {
      const int wnext = wbuf == NW - 1 ? 0 : wbuf + 1, xnext = xbuf == NX - 1 ? 0 : xbuf + 1;
      half(0, true, wbuf, xbuf, none);
      to_lds_wait<(NX - 2) * kCopies + kAhead>();  // the next block is in, and this one's buffers are free
      __syncthreads();
      half(1, true, wnext, xnext, [&](int i) __attribute__((always_inline)) {
        constexpr int kEach = (kCopies + RN - 1) / RN;
#pragma unroll
        for (int q = i * kEach; q < (i + 1) * kEach && q < kCopies; ++q) {
          if (q < kCopiesX) copy_x(kb + NX, xbuf, q);
          else copy_w(kb + NW, wbuf, q - kCopiesX);
        }
      });
      wbuf = wnext;
      xbuf = xnext;
    }
    half(0, true, wbuf, xbuf, none);
    half(1, false, 0, 0, none);
  } else {  // a wave without tokens copies for the others
    for (int kb = kb0; kb < kb1 - 1; ++kb) {
      to_lds_wait<(NX - 2) * kCopies + kAhead>();
      __syncthreads();
#pragma unroll
      for (int q = 0; q < kCopiesX; ++q) copy_x(kb + NX, xbuf, q);
#pragma unroll
      for (int q = 0; q < kCopiesW; ++q) copy_w(kb + NW, wbuf, q);
      wbuf = wbuf == NW - 1 ? 0 : wbuf + 1;
      xbuf = xbuf == NX - 1 ? 0 : xbuf + 1;
    }
  }
  to_lds_wait<0>();  // none of them outlives the workgroup

  const int rbw = rb0 + wn * RN;
  if (!GROUPED && a.chunks > 1) {
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      const int in = (wt * RT + j) * 16 + r;
      if (in >= tile.count) continue;
      int32_t* sums = a.part + (int64_t(chunk) * a.p + tile.first + in) * a.rbs * kRowBlock + 4 * c;
#pragma unroll
      for (int i = 0; i < RN; ++i)
        if (rbw + i < a.rbs) *reinterpret_cast<i32x4_t*>(sums + (rbw + i) * kRowBlock) = acc[i][j];
    }
    return;
  }
  float xs[RT];
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    bool there;
    const int from = source(a, tile.first + min((wt * RT + j) * 16 + r, tile.count - 1), there);
    xs[j] = there ? a.xs[from] : 0.f;
  }
  constexpr int kOutBytes = 16 * (RN / P * kRowBlock * 4 + 16);
  static_assert(kWaves * kOutBytes <= sizeof(lds), "the waves' outputs go through the operands' buffers");
  __syncthreads();  // every wave has read its last operands, and no copy is on its way
  uint8_t* own = lds + wave * kOutBytes;
  const int64_t first = tile.first + wt * RT * 16;
  const int count = tile.count - wt * RT * 16;
  write_tile<RN, RT, P>(a, acc, xs, ws, rbw, first, count, own);
}

// Fewer tokens, and ragged groups: tiles of 16 RN WN packed rows x 16 RT tokens on WN waves, which
// share the tokens and have 16 RN rows each: the weight goes from memory to the registers of
// the wave that owns its rows, D blocks ahead, and only the tokens' codes go through LDS (NX
// buffers).  LDS is read for the tokens alone, and two and more workgroups fit a unit, whose
// waits, starts and ends hide one another's.  (256 x 128 against the same tile with both
// operands in LDS: 128 gated experts of 1536 x 4096, 32768 rows 498 us from 515; 11008 x 4096,
// 2048 tokens 88 from 96.)  Large tiles are bound by their loads (of the 498 us the matrix units
// are busy for 55%), small ones by the weight's bytes or by the way of the first of them.
template <int WN, int RN, int RT, int D, int NX, int P, bool GROUPED>
__global__ __launch_bounds__(64 * WN, 2) void direct_kernel(Args a) {
  constexpr int kRb = WN * RN, kTok = 16 * RT;
  constexpr int kCopiesX = (2 * RT + WN - 1) / WN;  // of a wave, or of the first 2 RT waves
  static_assert(RN % P == 0 && (2 * RT % WN == 0 || 2 * RT < WN) && NX >= 2, "");
  constexpr int kOutBytes = 16 * (RN / P * kRowBlock * 4 + 16);
  constexpr int kLds = NX * RT * kFp8TileBytes > WN * kOutBytes ? NX * RT * kFp8TileBytes : WN * kOutBytes;
  __shared__ __align__(1024) uint8_t lds[kLds];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, c = lane >> 4;
  // neighbouring tiles on one XCD: of as many as there are (experts' rows may fill fewer than the grid)
  const int tiles_n = (a.rbs + kRb - 1) / kRb;
  const int all = GROUPED ? min(int64_t(count_tiles<kTok>(a)) * tiles_n, int64_t(gridDim.x)) : gridDim.x;
  if (int(blockIdx.x) >= all) return;
  const int per = all / 8, rest = all % 8, xcd = blockIdx.x % 8;
  const int wg = blockIdx.x / 8 + xcd * per + min(xcd, rest);
  const int chunk = GROUPED ? 0 : wg % a.chunks, id = GROUPED ? wg : wg / a.chunks;
  const int kb0 = chunk * a.chunk_kb, kb1 = min(kb0 + a.chunk_kb, a.kb);
  Group g{0, 0, a.t, 0};
  if constexpr (GROUPED) {
    g = find_group<kTok>(a, id / tiles_n);
    if (g.count == 0) return;
  }
  // as many token tiles of an expert as make it square, by as many row tiles as it takes
  constexpr int kSide = 8;
  const int local = id - g.tile0 * tiles_n, side = local / (kSide * tiles_n), in = local - side * kSide * tiles_n;
  const int tiles_t = (g.count + kTok - 1) / kTok, gt = min(kSide, tiles_t - kSide * side);
  const int rbw = in / gt * kRb + wave * RN;
  const Tile tile = tile_of<kTok>(g, kSide * side + in % gt);
  const uint8_t* codes = a.codes + int64_t(tile.expert) * a.stride;
  const float* ws = a.ws + int64_t(tile.expert) * a.rbs * kRowBlock;
  const uint8_t* wp[RN];
#pragma unroll
  for (int i = 0; i < RN; ++i) wp[i] = codes + int64_t(min(rbw + i, a.rbs - 1)) * a.kb * kFp8TileBytes;
  const int col = 16 * ((lane & 7) ^ (lane >> 3));
  const uint8_t* xp[kCopiesX];
#pragma unroll
  for (int i = 0; i < kCopiesX; ++i) {
    bool there;
    xp[i] = a.xq + source(a, tile.first + min((i * WN + wave) * 8 + (lane >> 3), tile.count - 1), there) * a.ldq;
  }
  const int xread = r * 128 + 16 * (c ^ (r & 7));
  auto copy_x = [&](int kb, int buf) __attribute__((always_inline)) {
    const int at = min(kb, kb1 - 1) * kFp8Block + col;
    const int off = at < a.xlim ? at : 0;
    if (2 * RT < WN && wave >= 2 * RT) return;
#pragma unroll
    for (int i = 0; i < kCopiesX; ++i) to_lds_from(xp[i] + off, lds + buf * (RT * kFp8TileBytes) + (i * WN + wave) * 1024);
  };
  u32x4_t w[D][2][RN], x[RT];
  auto load_w = [&](int kb, int s, int half) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < RN; ++i)
      w[s][half][i] = *reinterpret_cast<const u32x4_t*>(wp[i] + int64_t(min(kb, kb1 - 1)) * kFp8TileBytes + half * 1024 + lane * 16);
  };
  auto read_x = [&](int buf, int half, int j) __attribute__((always_inline)) {
    x[j] = *reinterpret_cast<const u32x4_t*>(lds + (buf * RT + j) * kFp8TileBytes + (xread ^ (64 * half)));
  };
  i32x4_t acc[RN][RT];
#pragma unroll
  for (int i = 0; i < RN; ++i)
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};

#pragma unroll
  for (int i = 0; i < NX; ++i) copy_x(kb0 + i, i);
#pragma unroll
  for (int i = 0; i < D; ++i) {
    load_w(kb0 + i, i, 0);
    load_w(kb0 + i, i, 1);
  }
  counted_wait<(NX - 1) * kCopiesX + D * 2 * RN, (NX - 1) * kCopiesX>();
  __syncthreads();
#pragma unroll
  for (int j = 0; j < RT; ++j) read_x(0, 0, j);
  // Left to itself the compiler puts the reads behind the products and waits for them (13824 x
  // 5120, 64 tokens in 128 x 64: 19.0 us against 18.3); the largest tile has no registers for
  // another order.
  constexpr bool kPinned = RN * RT <= 16;
  int buf = 0;
  // The weight's block is in slot s. The wait leaves on their way what is issued after the next
  // block's codes: copies, and with ahead set the weight's loads. The blocks behind the loop load
  // nothing: what no product uses the compiler takes out, and the wait would count loads not made.
  auto block = [&](int kb, int s, auto ahead) __attribute__((always_inline)) {
    constexpr bool kAhead = decltype(ahead)::value;
    const int next = buf == NX - 1 ? 0 : buf + 1;
#pragma unroll
    for (int j = 0; j < RT; ++j) {
#pragma unroll
      for (int i = 0; i < RN; ++i) acc[i][j] = mfma_i8(w[s][0][i], x[j], acc[i][j]);
      read_x(buf, 1, j);
      if constexpr (kPinned) __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (kAhead) load_w(kb + D, s, 0);
    counted_wait<(NX - 2) * kCopiesX + (kAhead ? ((NX - 2) * 2 + 2) * RN : 0), (NX - 2) * kCopiesX>();
    __syncthreads();
    copy_x(kb + NX, buf);
#pragma unroll
    for (int j = 0; j < RT; ++j) {
#pragma unroll
      for (int i = 0; i < RN; ++i) acc[i][j] = mfma_i8(w[s][1][i], x[j], acc[i][j]);
      read_x(next, 0, j);
      if constexpr (kPinned) __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (kAhead) load_w(kb + D, s, 1);
    buf = next;
  };
  int kb = kb0;
  for (; kb + D <= kb1; kb += D)
#pragma unroll
    for (int s = 0; s < D; ++s) block(kb + s, s, std::true_type{});
#pragma unroll
  for (int s = 0; s < D - 1; ++s)
    if (kb + s < kb1) block(kb + s, s, std::false_type{});
  to_lds_wait<0>();  // none of them outlives the workgroup
  if (!GROUPED && a.chunks > 1) {
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      const int at = j * 16 + r;
      if (at >= tile.count) continue;
      int32_t* sums = a.part + (int64_t(chunk) * a.p + tile.first + at) * a.rbs * kRowBlock + 4 * c;
#pragma unroll
      for (int i = 0; i < RN; ++i)
        if (rbw + i < a.rbs) *reinterpret_cast<i32x4_t*>(sums + (rbw + i) * kRowBlock) = acc[i][j];
    }
    return;
  }
  float xs[RT];
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    bool there;
    const int from = source(a, tile.first + min(j * 16 + r, tile.count - 1), there);
    xs[j] = there ? a.xs[from] : 0.f;
  }
  __syncthreads();  // every wave has read its last operands, and no copy is on its way
  uint8_t* own = lds + wave * kOutBytes;
  write_tile<RN, RT, P>(a, acc, xs, ws, rbw, tile.first, tile.count, own);
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
    f32x4_t w[P];
#pragma unroll
    for (int e = 0; e < P; ++e) w[e] = *reinterpret_cast<const f32x4_t*>(a.ws + (rb + e) * kRowBlock + 4 * c);
    finish<P>(a, token, rb, c, sum, a.xs[token], w);
  }
}

// Few tokens: a workgroup streams one row block (gated: the pair) for a tile of at most 16 TT
// tokens; its W waves take every W-th 128-input block, and their sums meet in LDS.  A wave has
// U blocks in its registers and the next U on their way; blocks past the end are loads out of
// the buffer's range, so that no load of a step stands behind a test.  Bound by the weight's
// bytes where they are many (4096 x 14336, one token 12.8 us with the launch: 4.6 TB/s) and by
// the ways of x, a block and the sums where they are few (5120 x 5120 7.3 us without it).
// XT: the type of x.  Codes (MBQ_INT8) are read from memory; a few float tokens are quantized
// here, once a workgroup into LDS, which saves the quantizing launch.
template <int W, int TT, int XT, int P, bool GROUPED>
__global__ __launch_bounds__(64 * W) void stream_kernel(Args a) {
  constexpr int U = (TT * P >= 4 ? 1 : TT * P == 2 ? 2 : 4) * 8 / W > 0 ? (TT * P >= 4 ? 1 : TT * P == 2 ? 2 : 4) * 8 / W : 1;
  constexpr bool kInline = XT != MBQ_INT8;
  constexpr int kNt = 2;  // the weight is read once: it need not stay in the caches
  static_assert(!kInline || TT == 1, "a few tokens");
  extern __shared__ __align__(16) uint8_t lx[];  // inline: codes, rows 16 bytes apart in banks
  __shared__ i32x4_t red[W][P * TT][64];
  __shared__ uint32_t amax[W];
  __shared__ float ls[16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, c = lane >> 4;
  const int rb0 = blockIdx.x * P;
  Tile tile{0, 0, a.t};
  if constexpr (GROUPED) {
    const Group g = find_group<16 * TT>(a, blockIdx.y);
    if (g.count == 0) return;
    tile = tile_of<16 * TT>(g, int(blockIdx.y) - g.tile0);
  }
  __amdgpu_buffer_rsrc_t rows[P];  // a row block each: loads past its end return 0 and touch no memory
#pragma unroll
  for (int i = 0; i < P; ++i)
    rows[i] = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(a.codes + int64_t(tile.expert) * a.stride + int64_t(rb0 + i) * a.kb * kFp8TileBytes), 0,
        a.kb * kFp8TileBytes, 0x00020000);
  f32x4_t wscale[P];  // asked for now: after the sums their way would be waited for
#pragma unroll
  for (int i = 0; i < P; ++i)
    wscale[i] = *reinterpret_cast<const f32x4_t*>(a.ws + (int64_t(tile.expert) * a.rbs + rb0 + i) * kRowBlock + 4 * c);
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
      const int kb = k0 + u * W;
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          wf[s][u][i][h] = __builtin_bit_cast(
              u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rows[i], kb * kFp8TileBytes + 1024 * h + lane * 16, 0, kNt));
      if constexpr (!kInline)
#pragma unroll
        for (int j = 0; j < TT; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int col = kb * kFp8Block + 64 * h + 16 * c;  // past the end of a row: see shared_kernel
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
#pragma unroll
      for (int j = 0; j < TT; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          u32x4_t v;
          if constexpr (kInline) v = *reinterpret_cast<const u32x4_t*>(xp[j] + min(kb, a.kb - 1) * kFp8Block + 64 * h);
          else v = xf[s][u][j][h];
#pragma unroll
          for (int i = 0; i < P; ++i) acc[i][j] = mfma_i8(wf[s][u][i][h], v, acc[i][j]);
        }
    }
  };

  if constexpr (kInline) {
    constexpr bool kBf = XT == MBQ_BF16;
    const int tid = threadIdx.x, end = a.kb * kFp8Block;
    bool there;
    auto row_of = [&](int i) __attribute__((always_inline)) {
      return static_cast<const uint8_t*>(a.x) + source(a, tile.first + i, there) * a.ldx * (kBf ? 2 : 4);
    };
    if (tile.count == 1) {  // one row by all waves; its first elements are asked for before the weight
      const uint8_t* row = row_of(0);
      Raw8<kBf> ahead;
      ahead.load(row, tid * 8, a.k);
      load(0, wave);
      float v[8];
      ahead.get(v);
      uint32_t m = amax8(v);
      for (int at = (tid + 64 * W) * 8; at < a.k; at += 64 * W * 8) {
        load8<kBf>(row, at, a.k, v);
        m = max(m, amax8(v));
      }
      m = max64(m);
      if (lane == 0) amax[wave] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < W; ++w) m = max(m, amax[w]);
      const float f = int8_factor(m);
      if (tid * 8 < end) {
        ahead.get(v);
        store_int8x8<false>(lx, tid * 8, ldl, v, f);
      }
      for (int at = (tid + 64 * W) * 8; at < end; at += 64 * W * 8) {
        load8<kBf>(row, at, a.k, v);
        store_int8x8<false>(lx, at, ldl, v, f);
      }
      if (tid == 0) ls[0] = there ? int8_scale(m) : 0.f;
    } else {  // a wave a row
      load(0, wave);
      for (int i = wave; i < tile.count; i += W) {
        const uint8_t* row = row_of(i);
        uint32_t m = 0;
        float v[8];
#pragma unroll 4
        for (int at = lane * 8; at < a.k; at += 512) {
          load8<kBf>(row, at, a.k, v);
          m = max(m, amax8(v));
        }
        m = max64(m);
        const float f = int8_factor(m);
#pragma unroll 4
        for (int at = lane * 8; at < end; at += 512) {
          load8<kBf>(row, at, a.k, v);
          store_int8x8<false>(lx + i * ldl, at, ldl, v, f);
        }
        if (lane == 0) ls[i] = there ? int8_scale(m) : 0.f;
      }
    }
    __syncthreads();
    xs[0] = ls[min(r, tile.count - 1)];
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
  if (in < tile.count) finish<P>(a, tile.first + in, rb0, c, sum, scale, wscale);
}

// The plan counts a form's tiles and threads by its table.
template <Int8Form F>
constexpr bool is_form(int rows, int tokens, int threads) {
  return kInt8Costs[int(F)].rows == rows && kInt8Costs[int(F)].tokens == tokens && kInt8Threads[int(F)] == threads;
}
template <Int8Form F, int WN, int WT, int RN, int RT, int NW, int NX, int P, bool GROUPED>
void launch_shared(const Args& a, dim3 grid, hipStream_t stream) {
  static_assert(is_form<F>(16 * RN * WN, 16 * RT * WT, 64 * WN * WT));
  shared_kernel<WN, WT, RN, RT, NW, NX, P, GROUPED><<<grid, 64 * WN * WT, 0, stream>>>(a);
}

template <Int8Form F, int WN, int RN, int RT, int D, int NX, int P, bool GROUPED>
void launch_direct(const Args& a, dim3 grid, hipStream_t stream) {
  static_assert(is_form<F>(16 * RN * WN, 16 * RT, 64 * WN));
  direct_kernel<WN, RN, RT, D, NX, P, GROUPED><<<grid, 64 * WN, 0, stream>>>(a);
}

template <Int8Form F, int W, int TT, int P, bool GROUPED>
void launch_stream(const Args& a, dim3 grid, mbq_dtype x_dtype, hipStream_t stream) {
  static_assert(is_form<F>(16, 16 * TT, 64 * W));
  const dim3 block(64 * W);
  if constexpr (TT == 1) {
    if (a.x) {
      const size_t lds = size_t(std::min(a.p, 16)) * (a.kb * kFp8Block + 16);
      if (x_dtype == MBQ_BF16) stream_kernel<W, 1, MBQ_BF16, P, GROUPED><<<grid, block, lds, stream>>>(a);
      else stream_kernel<W, 1, MBQ_F32, P, GROUPED><<<grid, block, lds, stream>>>(a);
      return;
    }
  }
  if constexpr (serves_int8(F, GROUPED, false)) stream_kernel<W, TT, MBQ_INT8, P, GROUPED><<<grid, block, 0, stream>>>(a);
}

template <int P, bool GROUPED>
hipError_t launch(Args& a, const Int8Plan& p, dim3 grid, mbq_dtype x_dtype, hipStream_t stream) {
  a.chunks = p.chunks;
  a.chunk_kb = (a.kb + p.chunks - 1) / p.chunks;
  using F = Int8Form;
  switch (p.form) {
    case F::kStream8x1: launch_stream<F::kStream8x1, 8, 1, P, GROUPED>(a, grid, x_dtype, stream); break;
    case F::kStream16x1: launch_stream<F::kStream16x1, 16, 1, P, GROUPED>(a, grid, x_dtype, stream); break;
    case F::kStream8x2: launch_stream<F::kStream8x2, 8, 2, P, GROUPED>(a, grid, x_dtype, stream); break;
    case F::kDirect64x16: launch_direct<F::kDirect64x16, 2, 2, 1, 6, 4, P, GROUPED>(a, grid, stream); break;
    case F::kDirect128x16: launch_direct<F::kDirect128x16, 4, 2, 1, 4, 4, P, GROUPED>(a, grid, stream); break;
    case F::kDirect128x32: launch_direct<F::kDirect128x32, 4, 2, 2, 4, 4, P, GROUPED>(a, grid, stream); break;
    case F::kDirect128x64: launch_direct<F::kDirect128x64, 4, 2, 4, 3, 3, P, GROUPED>(a, grid, stream); break;
    case F::kDirect256x64: launch_direct<F::kDirect256x64, 4, 4, 4, 2, 3, P, GROUPED>(a, grid, stream); break;
    case F::kDirect256x128: launch_direct<F::kDirect256x128, 4, 4, 8, 2, 2, P, GROUPED>(a, grid, stream); break;
    case F::kShared128x128: launch_shared<F::kShared128x128, 2, 4, 4, 2, 3, 3, P, GROUPED>(a, grid, stream); break;
    case F::kShared256x128: launch_shared<F::kShared256x128, 4, 2, 4, 4, 3, 3, P, GROUPED>(a, grid, stream); break;
    case F::kShared256x192: launch_shared<F::kShared256x192, 2, 4, 8, 3, 3, 2, P, GROUPED>(a, grid, stream); break;
    case F::kShared256x256: launch_shared<F::kShared256x256, 2, 4, 8, 4, 3, 2, P, GROUPED>(a, grid, stream); break;
  }
  if (a.chunks > 1)
    join_kernel<P><<<uint32_t(std::min<int64_t>((int64_t(a.p) * (a.rbs / P) * 4 + 255) / 256, 4096)), 256, 0, stream>>>(a);
  return hipGetLastError();
}

template <int P>
hipError_t launch(Args& a, const Int8Plan& p, dim3 grid, mbq_dtype x_dtype, hipStream_t stream) {
  return a.offsets ? launch<P, true>(a, p, grid, x_dtype, stream) : launch<P, false>(a, p, grid, x_dtype, stream);
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
  const Int8Grid n = grid_int8(plan, g.p, g.offsets ? d.experts : 0, d.row_blocks / (d.gated + 1), d.gated + 1);
  if (!holds_int8(n)) return hipErrorInvalidConfiguration;
  if (!serves_int8(plan.form, g.offsets ? d.experts : 0, plan.inline_x)) return hipErrorInvalidValue;
  const dim3 grid(uint32_t(n.x), uint32_t(n.y));
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
  return d.gated ? launch<2>(a, plan, grid, x_dtype, stream) : launch<1>(a, plan, grid, x_dtype, stream);
}

}  // namespace mbq
