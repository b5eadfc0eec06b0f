// 8-bit linear and the gated half of a feed-forward block:
//   y[t][i] = sum_kb xs[kb][t] ws[i / 128][kb] sum_{k in kb} xq[t][k] wq[i][k],
// one 128-input block per matrix instruction.  The instruction starts every block from
// zero; its result is scaled by xs ws and added to the float32 sums on the vector ALU, in
// the shadow of the next instructions.  Outputs are the instruction's rows and tokens its
// columns: a lane then holds one token, so a block needs one scale per lane and 16 tokens.
#include "fp8.h"
#include "fp8_plan.h"

namespace mbq {
namespace {

struct LinArgs {
  const uint8_t* codes;  // packed tiles
  const float* ws;       // weight scales [parts][nblk][kb]
  const uint8_t* xq;     // activation codes, rows of ldq bytes, xlim of them readable
  const float* xs;       // activation scales [kb][t]
  void* y;
  float* part;           // split K: sums [chunks][t][16 rbs], joined by a second launch
  const void* x;         // float activations, rows of ldx elements (quantized in the kernel)
  int64_t ldq, ldx;
  int32_t t, n, k, kb, rbs, nblk, xlim;
  int32_t chunks, chunk_kb;  // chunks of the blocks, chunk_kb each (the last one less)
};

// Tiles of 32 RN packed rows x 64 RT tokens on 2 x 4 waves (16 RN rows x 16 RT tokens each);
// both operands and the tokens' scales of a block go through NS LDS buffers, NS - 1 blocks
// ahead.  With few tiles K is split into chunks, one workgroup each.
template <int RN, int RT, int NS, int ACT, bool YBF>
__global__ __launch_bounds__(512, 2) void gemm_kernel(LinArgs a) {
  constexpr int kRb = 2 * RN, kTb = 4 * RT, kTok = 16 * kTb;
  constexpr int kCopiesW = 2 * kRb / 8, kCopiesX = RT;  // a wave's 1 KiB copies to LDS a block
  constexpr int kCopies = kCopiesW + kCopiesX + 1;
  static_assert(ACT == kPlain || RN % 2 == 0, "a gate tile and its up tile in one wave");
  static_assert(2 * kRb % 8 == 0, "every wave makes as many copies as the waits count");
  __shared__ __align__(1024) uint8_t lds[NS][(kRb + kTb) * kFp8TileBytes];
  __shared__ float lxs[NS][kTok];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, c = lane >> 4;
  const int wn = wave & 1, wt = wave >> 1;
  // neighbouring tiles (four token tiles by as many row tiles as it takes) on one XCD
  const int tiles_t = (a.t + kTok - 1) / kTok, tiles_n = (a.rbs + kRb - 1) / kRb;
  const int per = gridDim.x / 8, rest = gridDim.x % 8, xcd = blockIdx.x % 8;
  const int wg = blockIdx.x / 8 + xcd * per + min(xcd, rest);
  const int chunk = wg % a.chunks, id = wg / a.chunks;
  const int kb0 = chunk * a.chunk_kb, kb1 = min(kb0 + a.chunk_kb, a.kb);
  const int group = id / (4 * tiles_n), gt = min(4, tiles_t - 4 * group), in = id - group * 4 * tiles_n;
  const int rb0 = in / gt * kRb, tok0 = (4 * group + in % gt) * kTok;

  // a wave's rows lie in one 128-row block of each weight
  static_assert(ACT == kPlain ? 8 % RN == 0 : 16 % RN == 0, "one scale a weight");
  const int rbw = rb0 + wn * RN, rbl = min(rbw, a.rbs - 1);
  constexpr int P = ACT == kPlain ? 1 : 2;
  const ConstFloat* wsp = (const ConstFloat*)a.ws + int64_t(rbl / (8 * P)) * a.kb;
  auto scale_at = [&](int part, int kb) __attribute__((always_inline)) { return wsp[int64_t(part) * a.nblk * a.kb + kb]; };

  const uint8_t* wp[kCopiesW];
#pragma unroll
  for (int i = 0; i < kCopiesW; ++i) {
    const int half = i * 8 + wave;
    wp[i] = a.codes + int64_t(min(rb0 + (half >> 1), a.rbs - 1)) * a.kb * kFp8TileBytes + (half & 1) * 1024;
  }
  const uint8_t* xb = a.xq + tok0 * a.ldq;
  // A copy takes eight whole 128-byte rows of codes (copies of half rows of sixteen tokens
  // look up twice the cache lines: 296 us against 257 for 4096 x 3584 x 18944).  Row r's
  // 16-byte piece p goes to place p ^ (r mod 8), so that the eight rows an operand read
  // takes at once lie in different banks.
  const int col = 16 * ((lane & 7) ^ (lane >> 3));  // of this lane's bytes in a block (the same in all its copies)
  uint32_t xo[kCopiesX];  // their place from xb: 256 rows of at most 2^24 bytes
#pragma unroll
  for (int i = 0; i < kCopiesX; ++i)
    xo[i] = uint32_t(min((i * 8 + wave) * 8 + (lane >> 3), a.t - 1 - tok0)) * uint32_t(a.ldq) + col;
  const int xread = r * 128 + 16 * (c ^ (r & 7));  // the lane's first half of an operand in a tile
  const int xchunk = wave % RT;
  const uint32_t so = uint32_t(min(tok0 + xchunk * 64 + lane, a.t - 1)) * 4;

  auto copy_x = [&](int kb, int buf) __attribute__((always_inline)) {
    // Past the end of a row of codes (k no multiple of 128) the lane copies the row's first
    // bytes: they meet weight codes of 0, and a NaN among them has its token's row already.
    if (kb * kFp8Block + kFp8Block <= a.xlim) {
#pragma unroll
      for (int i = 0; i < kCopiesX; ++i)
        to_lds<16>(xb + int64_t(kb) * kFp8Block, xo[i], &lds[buf][(2 * kRb + i * 8 + wave) * 1024]);
    } else {
      const uint32_t at = kb * kFp8Block + col < a.xlim ? uint32_t(kb) * kFp8Block : 0u - uint32_t(col);
#pragma unroll
      for (int i = 0; i < kCopiesX; ++i) to_lds<16>(xb, xo[i] + at, &lds[buf][(2 * kRb + i * 8 + wave) * 1024]);
    }
    to_lds<4>(a.xs + int64_t(kb) * a.t, so, &lxs[buf][xchunk * 64]);
  };
  auto copy_w = [&](int kb, int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kCopiesW; ++i)
      to_lds<16>(wp[i] + int64_t(kb) * kFp8TileBytes, uint32_t(lane) * 16, &lds[buf][(i * 8 + wave) * 1024]);
  };

  float ws[P];  // the block's weight scales, loaded a block ahead
#pragma unroll
  for (int i = 0; i < P; ++i) ws[i] = scale_at(i, kb0);

  f32x4_t acc[RN][RT];
#pragma unroll
  for (int i = 0; i < RN; ++i)
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

#pragma unroll
  for (int i = 0; i < NS - 1; ++i)
    if (kb0 + i < kb1) {
      copy_x(kb0 + i, i);
      copy_w(kb0 + i, i);
    }
  int buf = 0;
  for (int kb = kb0; kb < kb1; ++kb) {
    const int next = kb + NS - 1, free = buf == 0 ? NS - 1 : buf - 1;
    // block kb is in (the copies of the blocks after it may be on their way), and every wave
    // has left the buffer of block kb - 1
    if (next <= kb1) to_lds_wait<(NS - 2) * kCopies>();
    else to_lds_wait<0>();
    __syncthreads();
    // a block's copies in two parts: all at once hold up the reads of this block
    if (next < kb1) copy_x(next, free);
    float ws_now[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      ws_now[i] = ws[i];
      ws[i] = scale_at(i, min(kb + 1, kb1 - 1));
    }
    auto frag = [&](int tile) __attribute__((always_inline)) {
      const u32x4_t* p = reinterpret_cast<const u32x4_t*>(&lds[buf][tile * kFp8TileBytes]) + lane;
      return join(p[0], p[64]);
    };
    auto frag_x = [&](int tile) __attribute__((always_inline)) {
      const uint8_t* p = &lds[buf][tile * kFp8TileBytes];
      return join(*reinterpret_cast<const u32x4_t*>(p + xread), *reinterpret_cast<const u32x4_t*>(p + (xread ^ 64)));
    };
    i32x8_t x[RT];
    float xs[RT], s[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      x[j] = frag_x(kRb + wt * RT + j);
      xs[j] = lxs[buf][(wt * RT + j) * 16 + r];
    }
    // row tiles in the order 0 .. RN - 1; gated: all gate tiles, then all up tiles
    constexpr auto tile_of = [](int q) { return ACT == kPlain ? q : q < RN / 2 ? 2 * q : 2 * q - RN + 1; };
    // A product is added two products later, so that no wave waits for its own instruction.
    constexpr int M = RN * RT, D = M < 3 ? M : 3;
    f32x4_t d[D];
    i32x8_t w[2] = {frag(wn * RN + tile_of(0)), {}};
#pragma unroll
    for (int m = 0; m < M + D - 1; ++m) {
      if (m == M / 4 && next < kb1) copy_w(next, free);
      if (m < M) {
        const int q = m / RT;
        if (m % RT == 0 && q + 1 < RN) w[(q + 1) & 1] = frag(wn * RN + tile_of(q + 1));
        d[m % D] = block_product<!YBF>(w[q & 1], x[m % RT]);
      }
      if (m >= D - 1) {
        const int f = m - (D - 1), i = tile_of(f / RT), j = f % RT;
        if (f % (M / P) == 0) {
#pragma unroll
          for (int e = 0; e < RT; ++e) s[e] = xs[e] * ws_now[f / (M / P)];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(d[f % D][e], s[j], acc[i][j][e]);
      }
    }
    buf = buf == NS - 1 ? 0 : buf + 1;
  }

#pragma unroll
  for (int j = 0; j < RT; ++j) {
    const int token = tok0 + (wt * RT + j) * 16 + r;
    if (token >= a.t) continue;
    if (a.chunks > 1) {
      float* row = a.part + (int64_t(chunk) * a.t + token) * a.rbs * 16 + 4 * c;
#pragma unroll
      for (int i = 0; i < RN; ++i)
        if (rbw + i < a.rbs) *reinterpret_cast<f32x4_t*>(row + (rbw + i) * 16) = acc[i][j];
      continue;
    }
#pragma unroll
    for (int i = 0; i < RN; i += ACT == kPlain ? 1 : 2) {
      const int rb = rbw + i;
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (ACT == kPlain) v[e] = acc[i][j][e];
        else v[e] = gated<ACT>(acc[i][j][e], acc[i + 1][j][e]);
      }
      if (rb < a.rbs) store4<YBF>(a.y, token, a.n, (ACT == kPlain ? rb : rb / 2) * 16 + 4 * c, v);
    }
  }
}

// Joins the chunks of a split K in their order: four outputs of one token a thread.
template <int ACT, bool YBF>
__global__ __launch_bounds__(256) void join_kernel(LinArgs a) {
  constexpr int R = ACT == kPlain ? 1 : 2;
  const int quads = a.rbs / R * 4;
  const int64_t stride = int64_t(a.t) * a.rbs * 16;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < int64_t(a.t) * quads; i += int64_t(gridDim.x) * 256) {
    const int token = int(i / quads), q = int(i - int64_t(token) * quads);
    const float* p = a.part + int64_t(token) * a.rbs * 16 + (q >> 2) * 16 * R + (q & 3) * 4;
    f32x4_t sum[R];
#pragma unroll
    for (int e = 0; e < R; ++e) sum[e] = *reinterpret_cast<const f32x4_t*>(p + 16 * e);
    for (int s = 1; s < a.chunks; ++s)
#pragma unroll
      for (int e = 0; e < R; ++e) {
        const f32x4_t v = *reinterpret_cast<const f32x4_t*>(p + s * stride + 16 * e);
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[e][k] += v[k];
      }
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (ACT == kPlain) v[e] = sum[0][e];
      else v[e] = gated<ACT>(sum[0][e], sum[R - 1][e]);
    }
    store4<YBF>(a.y, token, a.n, q * 4, v);
  }
}

// Up to 16 TT tokens: every workgroup streams one row block (gated: the pair), its W
// waves take every W-th 128-input block, and their sums meet in LDS in a fixed order.  Of
// the U blocks of a step a wave has one in flight at a time: the compiler puts each block's
// loads behind the test that ends the row.  What keeps memory busy is therefore the number of
// waves on a unit.  (18944 x 3584, 16 tokens, codes in: 14.3 us, 4.8 TB/s.)
// XT: the type of x.  Codes (MBQ_E4M3) are read from memory, with every block of the weight;
// a few float tokens are quantized here, once a workgroup into LDS, which saves the quantizing
// launch.  Their loads come after the first U weight tiles' and are waited for in order, so
// the quantization begins when those tiles are in.
constexpr int kInlineBlocks = 192;  // most that are quantized in the kernel (their place in LDS)

template <int W, int TT, int XT, int ACT, bool YBF>
__global__ __launch_bounds__(64 * W) void stream_kernel(LinArgs a) {
  constexpr int R = ACT == kPlain ? 1 : 2, U = TT == 1 ? 4 : 2;
  constexpr bool kInline = XT != MBQ_E4M3;
  static_assert(!kInline || TT == 1, "a few tokens");
  __shared__ f32x4_t red[W][R * TT][64];
  __shared__ __align__(16) uint8_t lx[kInline ? kInlineBlocks * kFp8Block + 16 * 16 : 16];  // rows 16 bytes apart in banks
  __shared__ float ls[kInline ? kInlineBlocks : 1];                                         // [kb][t]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, c = lane >> 4;
  const int rb0 = blockIdx.x * R;
  const ConstFloat* wsp = (const ConstFloat*)a.ws + int64_t(rb0 / (8 * R)) * a.kb;
  const ConstFloat* wsu = wsp + int64_t(a.nblk) * a.kb;
  const uint8_t* wp = a.codes + int64_t(rb0) * a.kb * kFp8TileBytes + lane * 16;
  const int row = a.kb * kFp8Block + 16;
  u32x4_t wf[U][R][2];
  auto load_w = [&](int k0) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = min(k0 + u * W, a.kb - 1);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const uint8_t* p = wp + (int64_t(i) * a.kb + kb) * kFp8TileBytes;
        wf[u][i][0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p));
        wf[u][i][1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p + 1024));
      }
    }
  };
  load_w(wave);
  if constexpr (kInline) {
    const int g = threadIdx.x & 15;
    for (int b = threadIdx.x >> 4; b < a.t * a.kb; b += 4 * W) {  // block b / t of token b % t
      const int blk = b / a.t, tok = b - blk * a.t, i = blk * kFp8Block + g * 8;
      float v[8];
      load8<XT == MBQ_BF16>(static_cast<const uint8_t*>(a.x) + tok * a.ldx * (XT == MBQ_BF16 ? 2 : 4), i, a.k, v);
      const uint32_t m = max16(amax8(v));
      store_codes8(lx + tok * row, i, row, v, fp8_factor(m));
      if (g == 0) ls[b] = fp8_scale(m);
    }
    __syncthreads();
  }
  f32x4_t acc[R][TT];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int k0 = wave; k0 < a.kb; k0 += W * U) {
    if (k0 != wave) load_w(k0);
    u32x4_t xf[U][TT][2];
    float xs[U][TT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = min(k0 + u * W, a.kb - 1);
#pragma unroll
      for (int j = 0; j < TT; ++j) {
        const int tok = min(j * 16 + r, a.t - 1), col = kb * kFp8Block + 16 * c;
        if constexpr (kInline) {
          const uint8_t* p = lx + tok * row + col;
          xf[u][j][0] = *reinterpret_cast<const u32x4_t*>(p);
          xf[u][j][1] = *reinterpret_cast<const u32x4_t*>(p + 64);
          xs[u][j] = ls[kb * a.t + tok];
        } else {
          const uint8_t* p = a.xq + tok * a.ldq;  // past the end of a row: see gemm_kernel
          xf[u][j][0] = *reinterpret_cast<const u32x4_t*>(p + (col < a.xlim ? col : 0));
          xf[u][j][1] = *reinterpret_cast<const u32x4_t*>(p + (col + 64 < a.xlim ? col + 64 : 0));
          xs[u][j] = a.xs[int64_t(kb) * a.t + tok];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = k0 + u * W;
      if (kb >= a.kb) break;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float ws = i == 0 ? wsp[kb] : wsu[kb];
#pragma unroll
        for (int j = 0; j < TT; ++j) {
          const f32x4_t d = block_product<!YBF>(join(wf[u][i][0], wf[u][i][1]), join(xf[u][j][0], xf[u][j][1]));
          const float s = xs[u][j] * ws;
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(d[e], s, acc[i][j][e]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) red[wave][i * TT + j][lane] = acc[i][j];
  __syncthreads();
  if (wave >= TT) return;
  const int j = wave, token = j * 16 + r;
  f32x4_t sum[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    sum[i] = red[0][i * TT + j][lane];
#pragma unroll 5
    for (int w = 1; w < W; ++w)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[i][e] += red[w][i * TT + j][lane][e];
  }
  if (token >= a.t) return;
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (ACT == kPlain) v[e] = sum[0][e];
    else v[e] = gated<ACT>(sum[0][e], sum[R - 1][e]);
  }
  store4<YBF>(a.y, token, a.n, int32_t(blockIdx.x) * 16 + 4 * c, v);
}

template <int RN, int RT, int NS, int ACT, bool YBF>
void launch_gemm(const LinArgs& a, hipStream_t stream) {
  const int64_t tiles = int64_t((a.rbs + 2 * RN - 1) / (2 * RN)) * ((a.t + 64 * RT - 1) / (64 * RT));
  gemm_kernel<RN, RT, NS, ACT, YBF><<<uint32_t(tiles * a.chunks), 512, 0, stream>>>(a);
}

template <int W, int TT, int ACT, bool YBF>
void launch_stream(const LinArgs& a, mbq_dtype x_dtype, hipStream_t stream) {
  const dim3 grid(a.rbs / (ACT == kPlain ? 1 : 2)), block(64 * W);
  if constexpr (TT == 1) {
    if (a.x && x_dtype == MBQ_BF16) {
      stream_kernel<W, 1, MBQ_BF16, ACT, YBF><<<grid, block, 0, stream>>>(a);
      return;
    }
    if (a.x) {
      stream_kernel<W, 1, MBQ_F32, ACT, YBF><<<grid, block, 0, stream>>>(a);
      return;
    }
  }
  stream_kernel<W, TT, MBQ_E4M3, ACT, YBF><<<grid, block, 0, stream>>>(a);
}

template <int ACT, bool YBF>
hipError_t launch(LinArgs& a, mbq_dtype x_dtype, hipStream_t stream) {
  constexpr int R = ACT == kPlain ? 1 : 2;
  if (a.x || streams(a.t, a.rbs / R, a.kb)) {  // float x (at most 16 tokens): only the streaming kernel reads it
    const StreamPlan p = plan_stream(a.t, a.rbs / R, a.kb);
    if (p.waves == 16) launch_stream<16, 1, ACT, YBF>(a, x_dtype, stream);
    else if (p.token_tiles == 1) launch_stream<8, 1, ACT, YBF>(a, x_dtype, stream);
    else if (p.token_tiles == 2) launch_stream<8, 2, ACT, YBF>(a, x_dtype, stream);
    else launch_stream<8, 4, ACT, YBF>(a, x_dtype, stream);
    return hipGetLastError();
  }
  const Plan p = plan_gemm(a.t, a.rbs, a.kb, !YBF);
  a.chunks = p.chunks;
  a.chunk_kb = (a.kb + p.chunks - 1) / p.chunks;
  switch (p.tile) {
    case 0:
      if constexpr (YBF) launch_gemm<8, 4, 2, ACT, YBF>(a, stream);
      break;
    case 1:
      if constexpr (YBF) launch_gemm<8, 3, 2, ACT, YBF>(a, stream);
      break;
    case 2:
      if constexpr (YBF) launch_gemm<8, 2, 3, ACT, YBF>(a, stream);
      break;
    case 3: launch_gemm<4, 2, 3, ACT, YBF>(a, stream); break;
    case 4: launch_gemm<2, 2, 3, ACT, YBF>(a, stream); break;
    case 5: launch_gemm<4, 1, 3, ACT, YBF>(a, stream); break;
    default: launch_gemm<2, 1, 3, ACT, YBF>(a, stream); break;
  }
  if (a.chunks > 1)
    join_kernel<ACT, YBF><<<uint32_t(std::min<int64_t>((int64_t(a.t) * (a.rbs / R) * 4 + 255) / 256, 4096)), 256, 0, stream>>>(a);
  return hipGetLastError();
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }
size_t codes_bytes(const mbq_fp8_desc& d, int32_t t) { return size_t(t) * d.k_blocks * kFp8Block; }

}  // namespace

// Float activations quantized inside the streaming kernel: its workgroups each do all of it,
// so a few blocks only, more where there is one workgroup a unit or less.  us within / in a
// launch before, by blocks: 5120 x 5120 (320 workgroups) 40 7.9 / 9.0, 80 8.4 / 9.1, 120 9.6 /
// 9.2; 18944 x 3584 (1184) 56 13.2 / 14.2, 112 14.7 / 14.4, 140 16.0 / 14.5; 3584 x 18944 (224)
// 148 13.8 / 15.3; 4096 x 4096 (256) 128 6.6 / 7.7, 192 7.6 / 7.7, 256 8.6 / 7.9.
bool quantize_inline(const mbq_fp8_desc& d, int32_t t, mbq_dtype x_dtype) {
  return x_dtype != MBQ_E4M3 && t <= 16 && int64_t(t) * d.k_blocks <= (d.row_blocks / (d.gated + 1) <= 256 ? kInlineBlocks : 96);
}

// Workspace: the activations' codes and scales (codes given in rows that hold no whole 16
// bytes: only their copy), then the partial sums of a split K.
size_t fp8_linear_workspace(const mbq_fp8_desc& d, int32_t t, mbq_dtype x_dtype) {
  size_t bytes = 0;
  if (quantize_inline(d, t, x_dtype)) return 0;
  if (x_dtype != MBQ_E4M3) bytes = codes_bytes(d, t) + align256(size_t(d.k_blocks) * t * 4);
  else if (d.k % 16 != 0) bytes = codes_bytes(d, t);
  size_t part = 0;
  if (!streams(t, d.row_blocks / (d.gated + 1), d.k_blocks))
    for (bool exact : {false, true}) {  // y's type is not known here
      const int chunks = plan_gemm(t, d.row_blocks, d.k_blocks, exact).chunks;
      if (chunks > 1) part = std::max(part, size_t(chunks) * t * d.row_blocks * 64);
    }
  return bytes + part;
}

hipError_t launch_fp8_linear(const mbq_fp8_desc& d, const void* packed, int32_t t, const void* x, mbq_dtype x_dtype,
                             int64_t ldx, const float* x_scale, int act, void* y, bool y_bf16, void* ws,
                             hipStream_t stream) {
  if (t == 0) return hipSuccess;
  const uint8_t* base = static_cast<const uint8_t*>(packed);
  LinArgs a{};
  a.codes = base;
  a.ws = reinterpret_cast<const float*>(base + d.scales_offset);
  a.y = y;
  a.t = t;
  a.n = d.n;
  a.k = d.k;
  a.kb = d.k_blocks;
  a.rbs = d.row_blocks;
  a.nblk = (d.n + 127) / 128;
  if (x_dtype == MBQ_E4M3 && d.k % 16 != 0) {
    a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + codes_bytes(d, t));
    a.ldq = a.xlim = d.k_blocks * kFp8Block;
    const hipError_t e = launch_fp8_pad_codes(t, d.k, x, ldx, ws, stream);
    if (e != hipSuccess) return e;
    a.xq = static_cast<const uint8_t*>(ws);
    a.xs = x_scale;
  } else if (x_dtype == MBQ_E4M3) {
    a.part = static_cast<float*>(ws);
    a.xq = static_cast<const uint8_t*>(x);
    a.ldq = ldx;
    a.xs = x_scale;
    a.xlim = d.k;
  } else if (quantize_inline(d, t, x_dtype)) {
    a.x = x;
    a.ldx = ldx;
  } else {
    uint8_t* q = static_cast<uint8_t*>(ws);
    float* s = reinterpret_cast<float*>(q + codes_bytes(d, t));
    a.part = reinterpret_cast<float*>(q + codes_bytes(d, t) + align256(size_t(d.k_blocks) * t * 4));
    a.ldq = a.xlim = d.k_blocks * kFp8Block;
    const hipError_t e = launch_fp8_quantize(t, d.k, x, x_dtype == MBQ_BF16, ldx, q, a.ldq, true, s, stream);
    if (e != hipSuccess) return e;
    a.xq = q;
    a.xs = s;
  }
  if (act == kPlain) return y_bf16 ? launch<kPlain, true>(a, x_dtype, stream) : launch<kPlain, false>(a, x_dtype, stream);
  if (act == MBQ_ACT_SILU)
    return y_bf16 ? launch<MBQ_ACT_SILU, true>(a, x_dtype, stream) : launch<MBQ_ACT_SILU, false>(a, x_dtype, stream);
  return y_bf16 ? launch<MBQ_ACT_GELU_TANH, true>(a, x_dtype, stream) : launch<MBQ_ACT_GELU_TANH, false>(a, x_dtype, stream);
}

}  // namespace mbq
