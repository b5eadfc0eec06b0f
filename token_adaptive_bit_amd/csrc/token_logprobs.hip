// Log probabilities of given tokens, entropy, rank and the top alternatives, in one pass
// over the logits.  With c = inv_temperature log2 e, a running reference r and d = c (x - r),
//   s = sum 2^d,  q = sum 2^d d
// give the log probability ln 2 d - ln s of x and the entropy ln s - ln 2 q / s; both sums
// are kept per lane in float32 about one reference a wave, which follows the wave's largest
// logit to within a factor of 2^1.5 in the terms.  (Where terms lead it further, ln s and d
// are large numbers whose difference is the answer: with a lead of up to 2^16 the entropy of
// rows near one certain token was off by 4e-6, now by a tenth of that.)  The rank counts
// lanes' comparisons on the scalar unit.  The top list is a sorted list of 64-bit keys
// (value, then lower index first), one entry a lane; a vector of logits is looked at only if
// it reaches the list's last entry.
// A row is split over several waves when there are few rows; beyond one workgroup's waves a
// second launch joins the parts.
#include "fp8.h"

namespace mbq {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

struct LpArgs {
  const void* logits;
  const void* targets;
  float *logprob, *entropy;
  int32_t *rank, *top_ids;
  float* top_logprobs;
  struct Part* part;  // [t][parts]
  uint64_t* keys;     // [t][parts][top]
  int64_t ld;
  int32_t t, v, top, parts, per;  // parts a row, one wave each; per: logits a part, a multiple of 8
  float inv_temperature;
  bool wide;
};

__device__ __forceinline__ uint32_t ordered(float x) {  // order of the values as unsigned numbers; -0 as 0
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ uint64_t key_of(float x, uint32_t i) { return uint64_t(ordered(x)) << 32 | uint32_t(~i); }
__device__ __forceinline__ uint64_t lane_key(uint64_t k, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane(uint32_t(k), lane), hi = __builtin_amdgcn_readlane(uint32_t(k >> 32), lane);
  return uint64_t(hi) << 32 | lo;
}

// The wave's best 64 keys, descending by lane (0: no entry).
struct TopList {
  uint64_t mine = 0;  // this lane's entry
  uint64_t last = 0;  // entry top - 1
  float floor = -__builtin_inff();  // no value below it can enter
  float gate = -__builtin_inff();   // nor, from a vector of higher indexes, one below this
  // More keys at once than this are absorbed, fewer offered (5, 12 and 24 measured alike).
  static constexpr int kMany = 12;

  // A full list takes no equal value of a higher index: from the next vector on.
  __device__ __forceinline__ void close_vector() {
    gate = last ? from_ordered(uint32_t(last >> 32) + 1) : floor;
  }
  // Every lane takes the larger of its entry and of the smaller of k and the entry before it.
  __device__ __forceinline__ void insert(uint64_t k, int top) {
    const uint32_t lo = __builtin_amdgcn_update_dpp(-1, int(uint32_t(mine)), 0x138, 0xF, 0xF, false);  // wave_shr 1
    const uint32_t hi = __builtin_amdgcn_update_dpp(-1, int(uint32_t(mine >> 32)), 0x138, 0xF, 0xF, false);
    const uint64_t before = uint64_t(hi) << 32 | lo;
    mine = max(mine, min(before, k));
    last = lane_key(mine, top - 1);
    if (last) floor = from_ordered(uint32_t(last >> 32));
  }
  // Offers one key a lane (0: none).
  __device__ __forceinline__ void offer(uint64_t k, int top) {
    uint64_t m = __ballot(k > last);
    while (m) {
      insert(lane_key(k, __builtin_ctzll(m)), top);
      m &= m - 1;
      if (m) m &= __ballot(k > last);
    }
  }
  // Fills an empty list with one key a lane: a bitonic sort of the wave.
  __device__ __forceinline__ void fill(uint64_t k, int lane, int top) {
    sort<2>(k, lane);
    mine = k;
    last = lane_key(mine, top - 1);
    if (last) floor = from_ordered(uint32_t(last >> 32));
  }
  // Takes in many keys at once: `back` ascends by lane.  (Top 64 with every key offered:
  // one row of 131072 27.7 us against 18.8, 4096 x 5000 54 against 43.)
  __device__ __forceinline__ void absorb(uint64_t back, int lane, int top) {
    mine = max(mine, back);
    merge<64, 32>(mine, lane);
    last = lane_key(mine, top - 1);
    if (last) floor = from_ordered(uint32_t(last >> 32));
  }
  __device__ __forceinline__ void absorb_any(uint64_t k, int lane, int top) {
    sort<2>(k, lane);
    absorb(__shfl(k, 63 - lane), lane, top);
  }
  // Fills an empty list from one descending list of `top` entries a lane (`has`: it has one):
  // their best, then their second ...; the first round without an entry is the last.
  __device__ __forceinline__ void take(const uint64_t* keys, bool has, int lane, int top) {
    fill(has ? keys[0] : 0, lane, top);
    for (int j = 1; j < top; ++j) {
      const uint64_t k = has ? keys[j] : 0;
      const int in = __popcll(__ballot(k > last));
      if (in == 0) break;
      if (in > kMany) absorb_any(k, lane, top);
      else offer(k, top);
    }
  }
  template <int SIZE>
  static __device__ __forceinline__ void sort(uint64_t& k, int lane) {
    merge<SIZE, SIZE / 2>(k, lane);
    if constexpr (SIZE < 64) sort<SIZE * 2>(k, lane);
  }
  template <int SIZE, int STEP>
  static __device__ __forceinline__ void merge(uint64_t& k, int lane) {
    const uint64_t o = across<STEP>(k);
    const bool larger = ((lane & STEP) == 0) == ((lane & SIZE) == 0 || SIZE == 64);  // this lane keeps the larger key
    if ((o > k) == larger) k = o;
    if constexpr (STEP > 1) merge<SIZE, STEP / 2>(k, lane);
  }
  // Raises the floor of a list without real values yet to one that at least `top` of the
  // lanes' x and y (maxima of several logits each) reach, found bit by bit over the upper
  // half of the ordered value: the list then fills with little more than `top` entries, not
  // with top (1 + ln(n / top)).  (One maximum a lane: 64 x 50021, top 64, 46.6 us against
  // 21.6.  NaN sorts above all; its row has no list.)
  __device__ __forceinline__ void start(float x, float y, int top) {
    const uint32_t o = ordered(x), p = ordered(y);
    uint32_t t = 0;
#pragma unroll
    for (int b = 31; b >= 16; --b)
      if (__popcll(__ballot(o >= (t | 1u << b))) + __popcll(__ballot(p >= (t | 1u << b))) >= top) t |= 1u << b;
    floor = fmaxf(floor, from_ordered(t));  // t == 0 maps to a NaN, which fmaxf drops
    gate = fmaxf(gate, floor);
  }
};

constexpr int kFirst = 256;  // keys of a part's first step that are sorted at once

constexpr float kLn2 = 0.69314718f;

// What a set of sums is about.  The reference of the exponents is one of two: a whole
// number M in units of ln 2 (m = 0), so that c x - M is a single FMA and rounds once; or,
// for values that c x would overflow or blur, a logit m (M = 0).
struct Reference {
  float m, M;
  static constexpr float kNone = -3e38f;  // M while nothing above -infinity has been seen

  __device__ __forceinline__ float exponent(float x, float c) const { return fmaf(x - m, c, -M); }
  // ln of 2^exponent, without its overflow far from the reference.
  __device__ __forceinline__ float natural(float x, float c, float inv_t) const {
    const float d = exponent(x, c);
    return fabsf(d) < 1e6f ? d * kLn2 : fmaf(x - m, inv_t, -M * kLn2);
  }
  // The exponent of this reference about r, which lies above it; less than 2^-10000 is 0
  // (finite, and at most 0 for the empty set's reference too, so that an empty sum stays 0).
  __device__ __forceinline__ float below(Reference r, float c) const {
    return fminf(fmaxf(fmaf(m - r.m, c, M - r.M), -1e4f), 0.f);
  }
};

// A lane's sums of a wave's part.
struct Sums {
  Reference r;  // the same in all lanes
  float s, q;

  __device__ __forceinline__ void refer(float x, float c) {
    const bool plain = fabsf(x * c) < 1e6f;
    const Reference to = {plain ? 0.f : x, plain ? rintf(x * c) : 0.f};
    const float d = r.below(to, c), f = __builtin_amdgcn_exp2f(d);
    q = f * fmaf(d, s, q);
    s *= f;
    r = to;
  }
};

// The sums of a part or of a row.  Lanes and parts meet in double, once a row: in float32
// the dozen small sums added to one near 1 would cost a confident row its last digits.
struct Total {
  Reference r;
  double s, q;

  __device__ __forceinline__ void join(Total o, float c) {
    if (o.s == 0.) return;
    if (s == 0. || r.m + r.M / c < o.r.m + o.r.M / c) {
      const Total t = *this;
      *this = o;
      o = t;
    }
    const float d = o.r.below(r, c);
    const double f = __builtin_amdgcn_exp2f(d);
    s += f * o.s;
    q += f * (o.q + d * o.s);
  }
  template <int STEP = 1>
  __device__ __forceinline__ void join_wave(float c) {
    join({{across<STEP>(r.m), across<STEP>(r.M)}, across<STEP>(s), across<STEP>(q)}, c);
    if constexpr (STEP < 32) join_wave<STEP * 2>(c);
  }
};

template <int STEP = 32>
__device__ __forceinline__ double wave_sum(double v) {
  v += across<STEP>(v);
  if constexpr (STEP > 1) v = wave_sum<STEP / 2>(v);
  return v;
}
__device__ __forceinline__ Total wave_total(const Sums& a) {
  return {a.r, wave_sum(double(a.s)), wave_sum(double(a.q))};
}

__device__ __forceinline__ int wave_sum(int v) {
  v += int(across<8>(uint32_t(v)));
  v += int(across<4>(uint32_t(v)));
  v += int(across<2>(uint32_t(v)));
  v += int(across<1>(uint32_t(v)));
  v += int(across<16>(uint32_t(v)));
  return v + int(across<32>(uint32_t(v)));
}

__device__ __forceinline__ float wave_max(float v) {  // NaN lanes take no part
  v = fmaxf(v, across<8>(v));
  v = fmaxf(v, across<4>(v));
  v = fmaxf(v, across<2>(v));
  v = fmaxf(v, across<1>(v));
  v = fmaxf(v, across<16>(v));
  return fmaxf(v, across<32>(v));
}

struct Part {
  Total total;
  int count, unused;
};

// A row's target (-1: none) and its logit.  Two reads that wait for one another, so they are
// asked for early.
struct Target {
  int at;
  float x;
};

template <bool BF16>
__device__ __forceinline__ float logit(const LpArgs& a, int row, int64_t i) {
  return load_x(a.logits, size_t(row) * size_t(a.ld) + size_t(i), BF16);
}

// The last rounding takes no probability above 1 and no entropy below 0 (NaN stays).
__device__ __forceinline__ float at_most_0(float v) { return v > 0.f ? 0.f : v; }

template <bool BF16>
__device__ __forceinline__ Target target_of(const LpArgs& a, int row) {
  const int64_t t = a.wide ? static_cast<const int64_t*>(a.targets)[row] : static_cast<const int32_t*>(a.targets)[row];
  Target r = {t >= 0 && t < a.v ? int(t) : -1, 0.f};
  if (r.at >= 0) r.x = logit<BF16>(a, row, r.at);
  return r;
}

// Between the LDS writes of a wave's lanes and the reads of its others: a wave's LDS accesses
// complete in order, so this only keeps the compiler from moving one past the other.
__device__ __forceinline__ void wave_exchange() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Writes a row's results from its sums and its top list (one wave).
__device__ __forceinline__ void finish(const LpArgs& a, int row, const Total& total, int count, const TopList& list,
                                       Target target, float c, int lane) {
  const float s = float(total.s);
  const bool valid = target.at >= 0;
  const bool none = s == 0.f, bad = s != s;  // nothing but -infinity; a NaN or +infinity
  const float log_s = logf(s) + float(total.s - s) / s, inf = __builtin_inff();
  if (lane == 0) {
    a.logprob[row] = !valid ? 0.f : none ? -inf : at_most_0(total.r.natural(target.x, c, a.inv_temperature) - log_s);
    a.entropy[row] = none ? 0.f : -at_most_0(kLn2 * (float(total.q) / s) - log_s);
    a.rank[row] = valid && !bad ? count + 1 : 0;
  }
  if (lane < a.top) {
    const float x = from_ordered(uint32_t(list.mine >> 32));
    a.top_ids[int64_t(row) * a.top + lane] = bad ? -1 : int32_t(~uint32_t(list.mine));
    a.top_logprobs[int64_t(row) * a.top + lane] = none ? -inf : bad ? s : at_most_0(total.r.natural(x, c, a.inv_temperature) - log_s);
  }
}

// One part of a row a wave.  The waves of a row meet in LDS when they fit one workgroup
// (1, 2 or 4 parts), else their results go to memory for the merging launch.
template <bool BF16, bool TOP>
__global__ __launch_bounds__(kThreads) void part_kernel(LpArgs a) {
  __shared__ Part parts[kWaves];
  __shared__ uint64_t lists[TOP ? kWaves : 1][TOP ? kFirst : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t id = int64_t(blockIdx.x) * kWaves + wave;
  const int row = __builtin_amdgcn_readfirstlane(int(min(id / a.parts, int64_t(a.t - 1)))), part = int(id - int64_t(row) * a.parts);
  const uint8_t* base = static_cast<const uint8_t*>(a.logits) + int64_t(row) * a.ld * (BF16 ? 2 : 4);
  const float c = a.inv_temperature * 1.4426950408889634f;
  Sums sums = {{0.f, Reference::kNone}, 0.f, 0.f};
  Total total = {};
  int count = 0;
  TopList list;
  Target target = {-1, 0.f};
  if (part < a.parts) {  // else the last workgroup's spare waves, with nothing to add
    const int begin = min(part * a.per, a.v), end = min(begin + a.per, a.v);
    int tied = 0;
    constexpr int U = 4, kStep = 64 * 8 * U;
    Raw8<BF16> next[U];
    auto load = [&](int i0) __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < U; ++u) next[u].load(base, i0 + (u * 64 + lane) * 8, end, -__builtin_inff());
    };
    load(begin);
    target = target_of<BF16>(a, row);
    const float xt = target.at >= 0 ? target.x : __builtin_inff();
    // x > xt as x >= the next value above it
    const float above = target.at >= 0 ? from_ordered(ordered(xt) + 1) : __builtin_inff();
    for (int i0 = begin; i0 < end; i0 += kStep) {
      Raw8<BF16> raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) raw[u] = next[u];
      if (i0 + kStep < end) load(i0 + kStep);
      float best[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float x[8];
        raw[u].get(x);
        best[u] = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
      }
      // The same reference in every lane: after the first step the wave's maximum grows a few
      // times a row, where lanes of their own would each outgrow theirs.  (Following it within
      // 2^1.5 and not 2^16.5 costs 2048 x 128000, top 8, 123.9 us against 121.1.)
      const float top_of = fmaxf(fmaxf(best[0], best[1]), fmaxf(best[2], best[3]));
      if (__ballot(top_of > -__builtin_inff() && (sums.r.M == Reference::kNone || sums.r.exponent(top_of, c) > 1.f)))
        sums.refer(wave_max(top_of), c);
      bool listed = false;  // this step's entries are in the list already
      if constexpr (TOP) {
        if (list.floor == -__builtin_inff()) {
          list.start(fmaxf(best[0], best[1]), fmaxf(best[2], best[3]), a.top);
          if (a.top > 12 && __ballot(list.mine != 0) == 0) {
            // an empty list: what reaches the floor, side by side in LDS, sorted at once (us
            // sorted / offered: 64 x 50021 top 8 14.7 / 13.7, top 12 15.4 / 14.8, top 16 15.6 /
            // 15.8, top 20 15.7 / 16.8)
            int n = 0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const int i = i0 + (u * 64 + lane) * 8;
              float x[8];
              raw[u].get(x);
              if (__ballot(best[u] >= list.floor && i < end)) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const bool in = x[e] >= list.floor && i + e < end;
                  const uint64_t m = __ballot(in);
                  const int at = n + __builtin_amdgcn_mbcnt_hi(uint32_t(m >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(m), 0));
                  if (in && at < kFirst) lists[wave][at] = key_of(x[e], uint32_t(i + e));
                  n += __popcll(m);
                }
              }
            }
            wave_exchange();
            if (n <= kFirst) {
              list.fill(lane < n ? lists[wave][lane] : 0, lane, a.top);
              for (int j = 64; j < n; j += 64) list.absorb_any(j + lane < n ? lists[wave][j + lane] : 0, lane, a.top);
              list.close_vector();
              listed = true;
            }
            wave_exchange();  // the next writes come after these reads
          }
        }
      }
      // A step's 32 terms are summed apart, by the vector, and then added: the lane's long
      // chain has few roundings.
      float ps = 0.f, pq = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + (u * 64 + lane) * 8;
        float x[8];
        raw[u].get(x);
        float vs = 0.f, vq = 0.f;
        if (__ballot(sums.r.m != 0.f)) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float d = sums.r.exponent(x[e], c), p = __builtin_amdgcn_exp2f(d);
            vs += p;
            vq = fmaf(p, fmaxf(d, -1e4f), vq);  // finite, so that p = 0 adds 0
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float d = fmaf(x[e], c, -sums.r.M), p = __builtin_amdgcn_exp2f(d);
            vs += p;
            vq = fmaf(p, fmaxf(d, -1e4f), vq);
          }
        }
        ps += vs;
        pq += vq;
        // a part ends on a vector; what is read past it counts for nothing
        const float bound = i >= end ? __builtin_inff() : i + 8 <= target.at ? xt : above;
#pragma unroll
        for (int e = 0; e < 8; ++e) count += __popcll(__ballot(x[e] >= bound));
        if (target.at >= i && target.at < i + 8) {  // the vector that holds the target: equal logits before it
#pragma unroll
          for (int e = 0; e < 8; ++e) tied += i + e < target.at && x[e] == xt;
        }
        if constexpr (TOP) {
          if (!listed && __ballot(best[u] >= list.gate && i < end)) {
            int at = i;
            asm("" : "+v"(at));  // the indexes are computed here and not in every step
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (__ballot(x[e] >= list.floor && at + e < end))
                list.offer(at + e < end && x[e] >= list.floor ? key_of(x[e], uint32_t(at + e)) : 0, a.top);
            list.close_vector();
          }
        }
      }
      sums.s += ps;
      sums.q += pq;
    }
    total = wave_total(sums);
    count += wave_sum(tied);
    if (a.parts > kWaves) {
      const int64_t at = int64_t(row) * a.parts + part;
      if (lane == 0) a.part[at] = {total, count, 0};
      if (TOP && lane < a.top) a.keys[at * a.top + lane] = list.mine;
    } else if (a.parts == 1) {
      finish(a, row, total, count, list, target, c, lane);
    }
  }
  if (a.parts == 1 || a.parts > kWaves) return;
  if (lane == 0) parts[wave] = {total, count, 0};
  if constexpr (TOP) lists[wave][lane] = list.mine;
  __syncthreads();
  if (part) return;
  for (int w = 1; w < a.parts; ++w) {
    total.join(parts[wave + w].total, c);
    count += parts[wave + w].count;
    if constexpr (TOP) {
      const uint64_t k = lane < a.top ? lists[wave + w][lane] : 0;
      if (__popcll(__ballot(k > list.last)) > TopList::kMany)
        list.absorb(63 - lane < a.top ? lists[wave + w][63 - lane] : 0, lane, a.top);
      else
        list.offer(k, a.top);
    }
  }
  finish(a, row, total, count, list, target, c, lane);
}

constexpr int kMaxParts = 64;

// Joins the parts of a row (more than one workgroup's), one lane each.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void merge_kernel(LpArgs a) {
  __shared__ uint64_t keys[kMaxParts * MBQ_MAX_TOP];
  const int row = blockIdx.x, lane = threadIdx.x & 63, all = a.parts * a.top;
  const Target target = target_of<BF16>(a, row);
  Total total = {{0.f, Reference::kNone}, 0., 0.};
  int count = 0;
  if (lane < a.parts) {
    total = a.part[int64_t(row) * a.parts + lane].total;
    count = a.part[int64_t(row) * a.parts + lane].count;
  }
  for (int i = threadIdx.x; i < all; i += kThreads) keys[i] = a.keys[int64_t(row) * all + i];
  __syncthreads();
  if (threadIdx.x >= 64) return;
  const float c = a.inv_temperature * 1.4426950408889634f;
  total.join_wave(c);
  count = wave_sum(count);
  TopList list;
  if (a.top) list.take(keys + (lane < a.parts ? lane : 0) * a.top, lane < a.parts, lane, a.top);
  finish(a, row, total, count, list, target, c, lane);
}

// Parts of a row: at least 4096 waves (four a SIMD), each with at least one full step of its
// loop.  (2048 x 128000 bfloat16, top 8: 124 us with two parts a row, 140 with one.  Sixteen
// parts in one workgroup, which would save the second launch of a short row, put them on one
// unit: an earlier form of this kernel took 17.2 us so against 15.8 for one row of 32000, top
// 20, and 29.7 against 14 for one of 131072, top 8.)
int parts_of(int32_t t, int32_t v) {
  const int64_t want = (4096 + int64_t(t) - 1) / std::max(t, 1), most = (int64_t(v) + 2047) / 2048;
  const int p = int(std::max<int64_t>(1, std::min<int64_t>(std::min(want, most), kMaxParts)));
  return p == 3 ? 4 : p;  // up to four parts share a workgroup, which holds whole rows
}

}  // namespace

size_t token_logprobs_workspace(int32_t t, int32_t v, int32_t top) {
  const int p = parts_of(t, v);
  return t == 0 || p <= kWaves ? 0 : size_t(t) * p * (sizeof(Part) + 8 * size_t(top));
}

hipError_t launch_token_logprobs(int32_t t, int32_t v, const void* logits, bool bf16, int64_t ld, const void* targets,
                                 bool wide, float inv_temperature, int32_t top, float* logprob, float* entropy,
                                 int32_t* rank, int32_t* top_ids, float* top_logprobs, void* ws, hipStream_t stream) {
  if (t == 0) return hipSuccess;
  LpArgs a{};
  a.logits = logits;
  a.targets = targets;
  a.logprob = logprob;
  a.entropy = entropy;
  a.rank = rank;
  a.top_ids = top_ids;
  a.top_logprobs = top_logprobs;
  a.ld = ld;
  a.t = t;
  a.v = v;
  a.top = top;
  a.parts = parts_of(t, v);
  a.per = ((v + a.parts - 1) / a.parts + 7) / 8 * 8;
  a.part = static_cast<Part*>(ws);
  a.keys = reinterpret_cast<uint64_t*>(a.part + int64_t(t) * a.parts);
  a.inv_temperature = inv_temperature;
  a.wide = wide;
  const dim3 grid(uint32_t((int64_t(t) * a.parts + kWaves - 1) / kWaves));
  if (bf16) {
    if (top) part_kernel<true, true><<<grid, kThreads, 0, stream>>>(a);
    else part_kernel<true, false><<<grid, kThreads, 0, stream>>>(a);
    if (a.parts > kWaves) merge_kernel<true><<<t, kThreads, 0, stream>>>(a);
  } else {
    if (top) part_kernel<false, true><<<grid, kThreads, 0, stream>>>(a);
    else part_kernel<false, false><<<grid, kThreads, 0, stream>>>(a);
    if (a.parts > kWaves) merge_kernel<false><<<t, kThreads, 0, stream>>>(a);
  }
  return hipGetLastError();
}

}  // namespace mbq
