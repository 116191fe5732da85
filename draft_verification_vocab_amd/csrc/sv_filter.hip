// Filtered sampling and verification for gfx950: the token distribution of a
// logit row under temperature, top-k, top-p and min-p, drawn from (the
// sampler) or used as the target of rejection sampling (the verify).  The
// definitions are in sv_filter.h and include/spec_verify.h.
//
//   filter_rows_kernel     one workgroup per row: the row's kept set as a filter
//                          row (its last token, maximum and 1 / sum), and for
//                          the sampler the drawn token and the dense q;
//   filter_stream_kernel   before it where rows are few and long: the pass over
//                          the logits by all CUs;
//   filter_left_kernel     after it where rows are many: those whose kept set
//                          does not fit its candidate list;
//   filtered_verify_kernel one workgroup per sequence: the accept scan from the
//                          filter rows, then the residual draw on the list of
//                          the row of the first rejection;
//   residual_kernel        that draw where the row has no list, over all CUs.
//
// The cuts are exact without a sort: a threshold from the groups' maxima picks
// some hundred candidates, their weights become integers, and the cut and the
// draw are found digit by digit in sums that do not depend on their order.
// What bounds it (MI355X, vocabulary 151936 in bf16):
//   many rows   HBM, then the exponentials: 7168 rows (2.18 GB) take 395-455 us
//               under top-k, min-p or greedy settings (4.8 to 5.5 TB/s), 690-780
//               under top-p alone (fp32 sums), 860-900 without a filter (fp64
//               sums, whose multiplications take two turns each); mixed 540-580;
//   few rows    the chain of steps of one workgroup: streaming or loading the
//               groups 4 us, threshold 2-5, candidates 3-6, cut and draw 3-9;
//               one row 15 us in all, 256 rows 74 us.
#include <algorithm>
#include <type_traits>

#include "sv_filter.h"
#include "sv_internal.h"

namespace sv {

namespace {

constexpr int kVerifyThreads = 256;
constexpr int kBins = 2048;            // 11 key bits per level
constexpr int kDrawTile = 2048;        // elements per tile of the draw
constexpr int kDrawTiles = SV_MAX_V / kDrawTile;
constexpr double kMassUnit = 17592186044416.0;   // 2^44: V <= 2^19 weights fit 64 bits

// ---------------------------------------------------------------- the draw
struct DrawShared {
  double mass[kDrawTiles];
  int token;
};

// The token drawn from masses mass(e) >= 0, e < V, with uniform u: the first
// whose running total exceeds u * sum, the last with any mass if rounding
// leaves none, -1 if no token has mass.  Every thread gets it.
template <int THREADS, typename F>
__device__ __forceinline__ int block_draw(int V, float u, DrawShared& sh, F mass) {
  const int w = threadIdx.x / kWave, l = lane_id();
  const int tiles = (V + kDrawTile - 1) / kDrawTile;
  __syncthreads();
  for (int t = w; t < tiles; t += THREADS / kWave) {
    double s = 0.0;
#pragma unroll 4
    for (int i = 0; i < kDrawTile / kWave; ++i) {
      const int e = t * kDrawTile + i * kWave + l;
      if (e < V) s += mass(e);
    }
    s = wave_sum(s);
    if (l == 0) sh.mass[t] = s;
  }
  __syncthreads();
  if (w == 0) {
    constexpr int PER = kDrawTiles / kWave;
    double m[PER], mine = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      m[i] = l * PER + i < tiles ? sh.mass[l * PER + i] : 0.0;
      mine += m[i];
    }
    const double incl = wave_inclusive_scan(mine);
    const double S = __shfl(incl, kWave - 1);
    const double target = (double)u * S;
    double run = incl - mine, before = 0.0;
    int hit = -1, any = -1;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (m[i] > 0.0) {
        any = l * PER + i;
        if (hit < 0 && run + m[i] > target) { hit = l * PER + i; before = run; }
      }
      run += m[i];
    }
    const unsigned long long hits = __ballot(hit >= 0), anys = __ballot(any >= 0);
    int token = -1;
    if (anys) {
      const int src = hits ? __ffsll((long long)hits) - 1 : 63 - __clzll((long long)anys);
      const int tile = __shfl(hits ? hit : any, src);
      double at = __shfl(before, src);
      int lastpos = -1;
#pragma unroll 1
      for (int i = 0; i < kDrawTile / kWave && token < 0; ++i) {
        const int e = tile * kDrawTile + i * kWave + l;
        const double x = e < V ? mass(e) : 0.0;
        const double in = wave_inclusive_scan(x);
        const unsigned long long pos = __ballot(x > 0.0);
        if (pos) lastpos = tile * kDrawTile + i * kWave + 63 - __clzll((long long)pos);
        const unsigned long long over = __ballot(x > 0.0 && at + in > target);
        if (hits && over) token = tile * kDrawTile + i * kWave + __ffsll((long long)over) - 1;
        at += __shfl(in, kWave - 1);
      }
      if (token < 0) token = lastpos;
    }
    if (l == 0) sh.token = token;
  }
  __syncthreads();
  return sh.token;
}

// ---------------------------------------------------------------- the kept set
template <int THREADS>
struct FilterShared {
  uint32_t cnt[kBins];
  unsigned long long mass[kBins];
  double red[THREADS / kWave];
  int redi[THREADS / kWave];
  int bin, ties;
  double above;
};

// The last token of a prefix of the order: kept iff key > this key, or key =
// this key and index <= last.
struct Cut {
  uint32_t key;
  int last;
};
__device__ __forceinline__ bool cut_keeps(const Cut& c, uint32_t key, int e) {
  return key > c.key || (key == c.key && e <= c.last);
}

// Index of the t-th token (t >= 1, in index order) whose key is `key`.
template <typename LT, int THREADS>
__device__ __forceinline__ int nth_tie(const LT* row, int V, uint32_t key, int t, uint32_t* cnt,
                                       int* slot) {
  const int tiles = (V + kDrawTile - 1) / kDrawTile;
  __syncthreads();
  for (int i = threadIdx.x; i < tiles; i += THREADS) cnt[i] = 0;
  __syncthreads();
  each_logit<LT, THREADS>(row, V, [&](float z, int e) {
    if (logit_key(z) == key) atomicAdd(&cnt[e / kDrawTile], 1u);
  });
  __syncthreads();
  if (threadIdx.x < kWave) {
    const int l = lane_id();
    int tile = 0, before = 0;
    for (; tile < tiles - 1; ++tile) {
      const int n = (int)cnt[tile];
      if (before + n >= t) break;
      before += n;
    }
    int found = V - 1;
#pragma unroll 1
    for (int i = 0; i < kDrawTile / kWave; ++i) {
      const int e = tile * kDrawTile + i * kWave + l;
      const bool is = e < V && logit_key(clean_logit(logit_at(row, e))) == key;
      unsigned long long b = __ballot(is);
      const int n = __popcll(b);
      if (before + n >= t) {
        for (int s = before + 1; s < t; ++s) b &= b - 1;
        found = tile * kDrawTile + i * kWave + __ffsll((long long)b) - 1;
        break;
      }
      before += n;
    }
    if (l == 0) *slot = found;
  }
  __syncthreads();
  const int r = *slot;
  __syncthreads();
  return r;
}

// Radix search, 11 key bits a level, for the key at which a running total
// over the order reaches a target: the number of tokens (MASS false) or their
// weights' sum in units of 2^-44 (integers, so that the order of the atomic
// additions does not matter; the rounding to a unit is below 2^-45 of the
// largest weight).  Only tokens that `in` keeps count.  Gives the key, the
// number of its tokens (ties) and the total above it.
template <typename LT, int THREADS, bool MASS>
__device__ __forceinline__ uint32_t radix_cut(const LT* row, int V, const Cut& in, float m, double c,
                              double target, int& ties, double& above, FilterShared<THREADS>& sh) {
  constexpr int PER = kBins / THREADS;
  static_assert(kBins % THREADS == 0, "whole bins per thread");
  const int w = threadIdx.x / kWave, l = lane_id();
  uint32_t prefix = 0, mask = 0;
  double base = 0.0;
  int n = 0;
#pragma unroll 1
  for (int level = 0; level < 3; ++level) {
    const int shift = level == 0 ? 21 : level == 1 ? 10 : 0;
    const uint32_t low = level == 2 ? 1023u : 2047u;
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += THREADS) { sh.cnt[i] = 0; sh.mass[i] = 0; }
    if (threadIdx.x == 0) { sh.bin = -1; sh.ties = -1; }
    __syncthreads();
    each_logit<LT, THREADS>(row, V, [&](float z, int e) {
      const uint32_t key = logit_key(z);
      if ((key & mask) == prefix && key > kKeyNegInf && cut_keeps(in, key, e)) {
        const uint32_t b = (key >> shift) & low;
        atomicAdd(&sh.cnt[b], 1u);
        if (MASS) atomicAdd(&sh.mass[b], (unsigned long long)rint(weight(z, m, c) * kMassUnit));
      }
    });
    __syncthreads();
    // thread t: bins kBins-1 - t*PER and down
    double part = 0.0;
    int lowest = -1;                                // lowest bin of mine with any token
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int b = kBins - 1 - ((int)threadIdx.x * PER + i);
      part += MASS ? (double)sh.mass[b] : (double)sh.cnt[b];
      if (sh.cnt[b]) lowest = b;
    }
    double run = wave_inclusive_scan(part);
    if (l == kWave - 1) sh.red[w] = run;
    if (lowest >= 0) atomicMax(&sh.ties, kBins - 1 - lowest);     // the order's last bin
    __syncthreads();
    double off = base;
    for (int i = 0; i < w; ++i) off += sh.red[i];
    run = off + run - part;                         // before my first bin
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int b = kBins - 1 - ((int)threadIdx.x * PER + i);
      const double x = MASS ? (double)sh.mass[b] : (double)sh.cnt[b];
      if (run < target && run + x >= target) { sh.bin = b; sh.above = run; }
      run += x;
    }
    __syncthreads();
    if (sh.bin < 0 && threadIdx.x == 0) {           // the target lies past the last token
      sh.bin = kBins - 1 - sh.ties;
      sh.above = -1.0;
    }
    __syncthreads();
    const int b = sh.bin;
    if (sh.above < 0.0) {                           // everything but that bin is above it
      double s = base;
      for (int i = kBins - 1; i > b; --i) s += MASS ? (double)sh.mass[i] : (double)sh.cnt[i];
      base = s;
    } else {
      base = sh.above;
    }
    n = (int)sh.cnt[b];
    prefix |= (uint32_t)b << shift;
    mask |= low << shift;
  }
  ties = n;
  above = base;
  return prefix;
}

// The kept set of one row.  Workgroup-wide; every thread gets the filter row.
template <typename LT, int THREADS>
__device__ __forceinline__ sv_filter_row filter_row(const LT* row, int V, const FilterSettings& s,
                                    FilterShared<THREADS>& sh) {
  float mx = -INFINITY;
  int nfin = 0;
  each_logit<LT, THREADS>(row, V, [&](float z, int) {
    mx = z > mx ? z : mx;
    nfin += z > -INFINITY;
  });
  float* redf = reinterpret_cast<float*>(sh.redi);
  const float m = block_reduce<THREADS>(mx, redf, OpMax());
  nfin = block_reduce<THREADS>(nfin, sh.redi, OpAdd());
  sv_filter_row f;
  f.scale = s.c;
  f.max = m;
  if (nfin == 0) {
    f.inv_sum = 0.0;
    f.min_kept = INFINITY;
    f.last = -1;
    f.n_kept = 0;
    return f;
  }
  Cut cut{0u, V};                                   // keeps everything
  if (s.k < nfin) {
    int ties;
    double above;
    const uint32_t key = radix_cut<LT, THREADS, false>(row, V, cut, m, s.c, (double)s.k, ties,
                                                       above, sh);
    const int keep = s.k - (int)above;
    cut = Cut{key, keep >= ties ? V : nth_tie<LT, THREADS>(row, V, key, keep, sh.cnt, &sh.bin)};
  }
  if (s.p < 1.0) {
    double part = 0.0;
    each_logit<LT, THREADS>(row, V, [&](float z, int e) {
      if (cut_keeps(cut, logit_key(z), e)) part += weight(z, m, s.c);
    });
    const double target = s.p * block_reduce<THREADS>(part, sh.red, OpAdd());
    int ties;
    double above;
    const uint32_t key = radix_cut<LT, THREADS, true>(row, V, cut, m, s.c, target * kMassUnit,
                                                      ties, above, sh);
    // the exact sum above the key, then how many of its tokens start below the target
    part = 0.0;
    each_logit<LT, THREADS>(row, V, [&](float z, int) {
      if (logit_key(z) > key) part += weight(z, m, s.c);
    });
    const double left = target - block_reduce<THREADS>(part, sh.red, OpAdd());
    const double w = weight(key_logit(key), m, s.c);
    const double need = w > 0.0 ? ceil(left / w) : (double)ties;
    const int keep = need >= (double)ties ? ties : need < 1.0 ? 1 : (int)need;
    if (key > cut.key || keep < ties)
      cut = Cut{key, keep >= ties ? V : nth_tie<LT, THREADS>(row, V, key, keep, sh.cnt, &sh.bin)};
  }
  if (s.mp > 0.0) {
    uint32_t lk = 0xffffffffu;
    each_logit<LT, THREADS>(row, V, [&](float z, int) {
      const uint32_t key = logit_key(z);
      if (key > cut.key && key < lk && weight(z, m, s.c) >= s.mp) lk = key;
    });
    // tokens of the cut's own key as well
    const bool whole = cut.key > kKeyNegInf && weight(key_logit(cut.key), m, s.c) >= s.mp;
    lk = block_reduce<THREADS>(lk, reinterpret_cast<uint32_t*>(sh.redi), OpMin());
    if (!whole) cut = Cut{lk, V};                   // the maximum is always kept
  }
  // count, sum and last token
  double part = 0.0;
  int n = 0, last = -1;
  uint32_t lk = 0xffffffffu;
  each_logit<LT, THREADS>(row, V, [&](float z, int e) {
    const uint32_t key = logit_key(z);
    if (key > kKeyNegInf && cut_keeps(cut, key, e)) {
      part += weight(z, m, s.c);
      ++n;
      if (key < lk) { lk = key; last = e; }
      else if (key == lk) last = e;                 // a thread's indices increase
    }
  });
  const uint32_t key = block_reduce<THREADS>(lk, reinterpret_cast<uint32_t*>(sh.redi), OpMin());
  last = block_reduce<THREADS>(lk == key ? last : -1, sh.redi, OpMax());
  n = block_reduce<THREADS>(n, sh.redi, OpAdd());
  const double S = block_reduce<THREADS>(part, sh.red, OpAdd());
  f.inv_sum = 1.0 / S;
  f.min_kept = s.off ? -INFINITY : key_logit(key);
  f.last = s.off ? V - 1 : last;
  f.n_kept = s.off ? V : n;
  return f;
}

// ---------------------------------------------------------------- one pass over a row
// The logits are streamed once.  A wave takes tiles of 4096 elements, lane l
// the octets u = 0..7 at 512 u + 8 l of a tile; G adjacent octets are a group,
// whose largest logit's key, its upper 16 bits, goes to LDS (V / (8 G) of
// them).  At least k logits reach the k-th largest of these, so only groups that
// reach a threshold found among them (candidate groups) can hold kept tokens,
// and only those are read again.  Where a filter needs the row's whole sum
// (top-p without top-k, no filter at all) the pass also leaves every tile's
// maximum and sum of weights.
constexpr int kRowTile = 4096;
constexpr int kRowTiles = SV_MAX_V / kRowTile;
constexpr int kCand = 2048;            // candidate tokens of a row's list in the workspace, and in
                                       // LDS where many rows are worked on
constexpr int kCandFew = 4096;         // ... in LDS elsewhere
constexpr int kQueue = 4096;           // candidate groups
constexpr int kBuckets = 512;          // of a digit search
constexpr int kTopBins = 256;          // histogram of the group maxima
constexpr int kFirst = 96;             // groups a nucleus row falls back to
constexpr int kGeneralRow = -2;        // list_counts: the row takes the general path
constexpr int kMaxListK = 1024;        // largest top-k taken through the candidate list
constexpr int kWaveList = 128;         // most candidates that one wave cuts and draws from

// Octets per group: 1, 2, 4 or 8, for at most `most` groups where that does.
// Smaller groups cost LDS and spare reading again: a candidate comes with G
// octets.
int group_octets(int V, int most) {
  int G = 1;
  while (G < 8 && (V + 7) / 8 > most * G) G *= 2;
  return G;
}
constexpr int kGroups = 5120;          // ... where many rows are worked on
constexpr int kGroupsFew = 10240;      // ... elsewhere

template <int THREADS>
struct RowShared {
  union {
    unsigned long long top[kTopBins];  // groups << 32 | their weights in 2^-18
    uint16_t queue[kQueue];
    unsigned long long bucket[kBuckets];
    struct { unsigned long long entry[kWaveList]; double w[kWaveList]; int id[kWaveList]; } sorted;
  };
  double tile_s[kRowTiles];
  float tile_m[kRowTiles];
  ExpEntry table[kExpTable];
  double red[3 * (THREADS / kWave)];
  int redi[THREADS / kWave];
  unsigned long long* list;            // candidates: order_entry; cap of them at most
  int cap;
  int n, nq, token, bin, above;
  float frac;
  // what the first wave finds in a short list
  int found;
  double got;
  sv_filter_row row;
};

// Exclusive running totals over the workgroup's threads, and the total.
template <int THREADS>
__device__ __forceinline__ double block_scan(double x, double* sm, double& total) {
  const double incl = wave_prefix(x);
  __syncthreads();
  if (lane_id() == kWave - 1) sm[threadIdx.x / kWave] = incl;
  __syncthreads();
  double off = 0.0, all = 0.0;
#pragma unroll
  for (int i = 0; i < THREADS / kWave; ++i) {
    if (i < (int)threadIdx.x / kWave) off += sm[i];
    all += sm[i];
  }
  total = uniform(all);
  return off + (incl - x);
}

// An entry of the list; their order is that of the tokens.
__device__ __forceinline__ unsigned long long order_entry(uint32_t key, int e) {
  return ((unsigned long long)~key << 32) | (uint32_t)e;
}

// Whether a row's filters need the sum of all its weights: no top-k bounds the
// tokens that matter, and they do not all fit the candidate list.
__device__ __forceinline__ bool row_needs_sum(const FilterSettings& s, int V) {
  return V > kCand && s.k >= V && (s.p < 1.0 || s.off);
}

// How the stream takes it.  For 7168 nucleus rows of 151936 in bf16 SUM_F32 takes
// 690-780 us against 990-1050 of SUM_F64, though about one row in a hundred has to
// be streamed again for its cut; 3584 in fp32 take 464-543 against 619-653 us.  For
// few rows that one row costs all (79 against 59 us for 64).
enum RowSum { NO_SUM, SUM_F32, SUM_F64 };

// The maximum over N = 2, 4 or 8 adjacent lanes (from the maximum over N / 2,
// for N = 4; the whole for N = 8).
template <int N>
__device__ __forceinline__ float max_adjacent(float x) {
  const auto other = [&](auto dpp) {
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(x), __float_as_int(x),
                                                      decltype(dpp)::value, 0xf, 0xf, false));
  };
  if constexpr (N != 4) x = fmaxf(x, other(std::integral_constant<int, 0xB1>()));   // 1 0 3 2
  if constexpr (N != 2) x = fmaxf(x, other(std::integral_constant<int, 0x4E>()));   // 2 3 0 1
  if constexpr (N == 8) x = fmaxf(x, other(std::integral_constant<int, 0x141>()));  // 7 .. 0
  return x;
}

// One wave's tile t of a row: its groups' keys to gm (the row's), with a sum
// its maximum and sum of weights to *tile_m, *tile_s.  Gives the lane's largest
// logit.  128 bytes a lane are in flight:
// a bf16 tile at once, an fp32 tile in two parts.
template <typename LT, RowSum SUM>
__device__ __forceinline__ void stream_tile(const LT* row, int V, int t, double c, int G, uint16_t* gm,
                                            float* tile_m, double* tile_s, const ExpEntry* table,
                                            float& top) {
  constexpr int OCTS = 16 / sizeof(LT);
  int l = lane_id();
  asm volatile("" : "+v"(l));                       // its addresses are not kept past a tile
  float ref = -INFINITY;                            // the sum's reference logit
  double sum = 0.0;
#pragma unroll 1
  for (int part = 0; part < 8 / OCTS; ++part) {
    Raw<LT> raw[OCTS];
    const int e0 = t * kRowTile + part * OCTS * kTile + 8 * l;
    if ((t + 1) * kRowTile <= V) {
#pragma unroll
      for (int u = 0; u < OCTS; ++u) raw8(row + e0 + u * kTile, raw[u]);
    } else {
#pragma unroll
      for (int u = 0; u < OCTS; ++u) {
        const int e = e0 + u * kTile;
        if (e + 8 <= V) raw8(row + e, raw[u]);
        else raw8_end(row, e, V, raw[u]);
      }
    }
    float mt = -INFINITY;
#pragma unroll
    for (int u = 0; u < OCTS; ++u) {
      float z[8];
      unpack(raw[u], z);
      float g = fmaxf(fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])),
                      fmaxf(fmaxf(z[4], z[5]), fmaxf(z[6], z[7])));
      g = clean_logit(g);
      mt = fmaxf(mt, g);
      // G is uniform
      if (G == 8) g = max_adjacent<8>(g);
      else if (G >= 2) g = max_adjacent<2>(g);
      if (G == 4) g = max_adjacent<4>(g);
      if ((l & (G - 1)) == 0)
        gm[(t * (kRowTile / 8) + (part * OCTS + u) * kWave + l) / G] =
            (uint16_t)(logit_key(g) >> 16);
    }
    top = fmaxf(top, mt);
    if constexpr (SUM != NO_SUM) {
      mt = wave_reduce(mt, OpMax());
      double s = 0.0, s1 = 0.0;
      const double mc = (double)mt * c;
      if (SUM == SUM_F32 && fabs(mc) < 4096.0 && c > 0x1p-100 && c < 0x1p100) {
        // The exponents z c + shift, shift near -mt c; what is left, 2^-(mt c +
        // shift), scales the sum.  An exponent x is off by 2^-24 |x| from its
        // rounding and as much from c's, the exponential by 2^-23 relative: a term
        // is exact to (0.7 |x| + 1) 2^-23.  -inf and NaN count 0.  Eight terms are
        // added in fp32, then in fp64.
        const float c32 = (float)c, shift = -(float)mc;
#pragma unroll
        for (int u = 0; u < OCTS; ++u) {
          keep_raw(raw[u]);
          float z[8], e[8];
          unpack(raw[u], z);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            e[j] = __builtin_amdgcn_exp2f(fmaxf(__builtin_fmaf(z[j], c32, shift), -500.f));
          s += (double)tree_sum8(e);
          __builtin_amdgcn_sched_barrier(0);        // one octet in flight: registers
        }
        s *= TwoTo()(-fma((double)mt, (double)c32, (double)shift));
      } else if (SUM == SUM_F64 && fabs(mc) < 4096.0) {
        // Here shift is a multiple of 1/64: z c added to `magic` is rounded to
        // such a multiple as well.  Logits 500 octaves and more below the maximum
        // (and -inf, NaN) count 2^-500.
        double opaque = c;                          // its reciprocal is not kept
        asm volatile("" : "+v"(opaque));
        const double floor = (double)mt - 500.0 * __builtin_amdgcn_rcp(opaque);
        const double shift = -rint(mc * kExpTable) / kExpTable;
        const double magic = kExpRound + shift;
        const TwoTo two_to;
#pragma unroll
        for (int u = 0; u < OCTS; ++u) {
          keep_raw(raw[u]);
          float z[8];
          unpack(raw[u], z);
          const auto add = [&](float z, double& sum) {
            const double x = fmax((double)z, floor), y = fma(x, c, magic);
            sum = fma(table_entry(y, table), two_to(fma(x, c, magic - y)), sum);
          };
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            add(z[j], s);
            add(z[j + 1], s1);
            if (j == 2) __builtin_amdgcn_sched_barrier(0);   // registers
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        s = (s + s1) * two_to(-(mc + shift));
      } else if (mt > -INFINITY) {
#pragma unroll 1
        for (int i = 0; i < OCTS * 8; ++i) {
          const int e = t * kRowTile + part * OCTS * kTile + i * kWave + l;
          if (e < V) s += weight(clean_logit(logit_at(row, e)), mt, c, table);
        }
      }
      s = wave_reduce(s, OpAdd());
      if constexpr (OCTS == 8) {                    // the whole tile
        ref = mt;
        sum = s;
        continue;
      }
      if (mt > ref) {
        sum *= ref > -INFINITY ? weight(ref, mt, c, table) : 0.0;
        ref = mt;
      }
      if (mt > -INFINITY) sum += s * weight(mt, ref, c, table);
    }
  }
  if constexpr (SUM != NO_SUM)
    if (l == 0) { *tile_m = ref; *tile_s = sum; }
}

// A whole row by one workgroup, into LDS.
template <typename LT, int THREADS, RowSum SUM>
__device__ __forceinline__ void stream_row(const LT* row, int V, double c, int G, uint16_t* gm,
                                           RowShared<THREADS>& sh, float& top) {
  const int tiles = (V + kRowTile - 1) / kRowTile;
  for (int t = threadIdx.x / kWave; t < tiles; t += THREADS / kWave)
    stream_tile<LT, SUM>(row, V, t, c, G, gm, &sh.tile_m[t], &sh.tile_s[t], sh.table, top);
}

// What a row's stream leaves, where a kernel of its own made it: into LDS.
template <int THREADS>
__device__ __forceinline__ void load_streamed(const FilterLaunch& A, long r, int groups, int tiles,
                                              bool sum, uint16_t* gm, RowShared<THREADS>& sh,
                                              float& top) {
  int t0 = threadIdx.x;
  asm volatile("" : "+v"(t0));                      // its addresses are not kept past this
  // groups is even: a pair of keys at a time
  const uint32_t* g = reinterpret_cast<const uint32_t*>(A.group_key + r * groups);
  for (int i = t0; i < groups / 2; i += THREADS) reinterpret_cast<uint32_t*>(gm)[i] = g[i];
  for (int t = t0; t < tiles; t += THREADS) top = fmaxf(top, A.tile_max[r * tiles + t]);
  if (sum)
    for (int t = t0; t < tiles; t += THREADS) {
      sh.tile_m[t] = A.tile_max[r * tiles + t];
      sh.tile_s[t] = A.tile_sum[r * tiles + t];
    }
}

// The key (its upper 16 bits) from which on logits can be kept, from the
// groups' keys: at least k of them reach it (by count, k > 0), or the weights of
// the logits that do are about `aim` times that of logit z0 (by mass, k = 0).
// One histogram of the 256 keys from `hi` down, two binades; where that does not
// reach, one of all keys below and, if the threshold's bin is crowded, of that
// bin.  A group's largest logit stands for its tokens of that size; in the
// estimate of the mass, those hidden behind a larger one of their group are
// added from the share of groups without a larger one.  `above` groups lie above
// `hi`.  The lowest finite key if nothing reaches it.
constexpr uint32_t kLowest = (kKeyNegInf + 1) >> 16;
template <typename LT, int THREADS>
__device__ __forceinline__ uint32_t threshold_key(const uint16_t* gm, int groups, uint32_t hi,
                                                  int above, float z0, float c, int k,
                                                  float aim, RowShared<THREADS>& sh) {
  const bool by_mass = k == 0;
  if (hi < kLowest) return kLowest;
  float mass = 0.f;                    // estimated mass found
  bool near = hi - kLowest >= kTopBins;
  uint32_t lo = near ? hi - (kTopBins - 1) : kLowest;
#pragma unroll 1
  for (int level = 0; level < 3; ++level) {
    const int shift = hi - lo < kTopBins ? 0 : 8;
    __syncthreads();
    for (int i = threadIdx.x; i < kTopBins; i += THREADS) sh.top[i] = 0;
    if (threadIdx.x == 0) sh.bin = -1;
    __syncthreads();
    // four keys at a time (groups are whole tiles'); by mass, one LDS addition
    // counts a group and its weight, and weights under 2^-18 are left out
    const uint32_t least =
        by_mass ? max(lo, logit_key(clean_logit(z0 - 18.f / uniform(c))) >> 16) : lo;
#pragma unroll 1
    for (int i = threadIdx.x; i < groups / 4; i += THREADS) {
      const uint2 keys = reinterpret_cast<const uint2*>(gm)[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t two = j < 2 ? keys.x : keys.y, key = j % 2 ? two >> 16 : two & 0xffffu;
        if (key <= hi && key >= least) {
          uint32_t w = 0;
          if (by_mass) {
            // the logit: exactly (bf16), or the middle of those with this half of a key
            const float g = key_logit(key << 16 | (sizeof(LT) == 4 ? 0x8000u
                                                   : key & 0x8000u ? 0u : 0xffffu));
            w = g >= z0 ? 262144u
                        : (uint32_t)(__builtin_amdgcn_exp2f((g - z0) * c) * 262144.f);
          }
          atomicAdd(&sh.top[(hi - key) >> shift], 1ull << 32 | w);
        }
      }
    }
    __syncthreads();
    if (threadIdx.x < kWave) {
      constexpr int PER = kTopBins / kWave;
      const int l = lane_id();
      int n[PER], mine = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) { n[i] = (int)(sh.top[l * PER + i] >> 32); mine += n[i]; }
      int run = wave_prefix(mine) + above - mine;
      int hit = -1, before = 0;
      float fbefore = 0.f;
      if (!by_mass) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          if (hit < 0 && run < k && run + n[i] >= k) { hit = l * PER + i; before = run; }
          run += n[i];
        }
      } else {
        // elements per group maximum of a bin: at most groups / (groups not
        // yet reached at its end); over the whole bin the logarithm's mean
        float f[PER], most[PER], fmine = 0.f;
        int r = run;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const float x = (float)(uint32_t)sh.top[l * PER + i] * (1.f / 262144.f) * (float)groups;
          const float left = (float)max(1, groups - r), after = (float)max(1, groups - r - n[i]);
          most[i] = x * __builtin_amdgcn_rcpf(after);
          f[i] = n[i] ? x * 0.69314718f *
                            __builtin_amdgcn_logf(left * __builtin_amdgcn_rcpf(after)) *
                            __builtin_amdgcn_rcpf((float)n[i])
                      : 0.f;
          r += n[i];
          fmine += f[i];
        }
        float frun = wave_prefix(fmine) + mass - fmine;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          if (hit < 0 && n[i] && frun + most[i] >= aim) {
            hit = l * PER + i; before = run; fbefore = frun;
          }
          run += n[i];
          frun += f[i];
        }
      }
      const unsigned long long hits = __ballot(hit >= 0);
      if (hits && l == __ffsll((long long)hits) - 1) {
        sh.bin = hit; sh.above = before; sh.frac = fbefore;
      }
    }
    __syncthreads();
    const int b = uniform(sh.bin);
    if (b < 0) {
      if (near) {
        near = false;
        lo = kLowest;
        continue;
      }
      // not reached: every token, or (by mass, inside a bin that seemed to
      // reach it) what there is
      return lo;
    }
    if (shift == 0) return hi - b;
    near = false;
    above = uniform(sh.above);
    mass = uniform(sh.frac);
    const int in = (int)(uniform(sh.top[b]) >> 32);
    const uint32_t top = hi - ((uint32_t)b << shift);
    const uint32_t bottom = top - lo > 255 ? top - 255 : lo;
    if (in <= above / 4 + 32) return bottom;
    hi = top;
    lo = bottom;
  }
  return lo;
}

// The tokens whose key is at least kt into sh.list, in any order.  Returns their number, or -1 if they or their groups
// are more than the lists hold.
template <typename LT, int THREADS>
__device__ __forceinline__ int gather_tokens(const LT* row, int V, int G, int groups,
                                             const uint16_t* gm, uint32_t kt,
                                             RowShared<THREADS>& sh) {
  const float zt = key_logit(kt);
  const uint32_t kg = kt >> 16;
  __syncthreads();
  if (threadIdx.x == 0) { sh.nq = 0; sh.n = 0; }
  __syncthreads();
  // Places for each lane's c entries, by one addition per wave: of its own, the
  // compiler would add up the lanes of a divergent addition one after the other.
  const auto place = [](int* counter, int c) {
    const int incl = wave_prefix(c), all = of_lane(incl, kWave - 1);
    int base = 0;
    if (all && lane_id() == 0) base = atomicAdd(counter, all);
    return uniform(base) + incl - c;
  };
  int mine = 0;
#pragma unroll 4
  for (int i = threadIdx.x; i < groups; i += THREADS) mine += gm[i] >= kg;
  int q = place(&sh.nq, mine);
  if (mine) {
#pragma unroll 4
    for (int i = threadIdx.x; i < groups; i += THREADS)
      if (gm[i] >= kg) {
        if (q < kQueue) sh.queue[q] = (uint16_t)i;
        ++q;
      }
  }
  __syncthreads();
  const int nq = uniform(sh.nq);
  if (nq > kQueue) return -1;
  // two octets a thread at a time
  constexpr int BATCH = 2;
  const int items = nq * G;
#pragma unroll 1
  for (int base = 0; base < items; base += BATCH * THREADS) {
    const int i0 = base + threadIdx.x;
    Raw<LT> raw[BATCH];
    int e[BATCH];
#pragma unroll
    for (int p = 0; p < BATCH; ++p) {
      const int i = min(i0 + p * THREADS, items - 1);
      e[p] = (sh.queue[i / G] * G + i % G) * 8;
      if (e[p] + 8 <= V) raw8(row + e[p], raw[p]);
      else raw8_end(row, e[p], V, raw[p]);
    }
    uint32_t hits = 0;                              // bit 8 p + j
#pragma unroll
    for (int p = 0; p < BATCH; ++p) {
      float z[8];
      unpack(raw[p], z);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        hits |= (uint32_t)(clean_logit(z[j]) >= zt && i0 + p * THREADS < items) << (8 * p + j);
    }
    int at = place(&sh.n, (int)__popc(hits));
    if (hits) {
#pragma unroll
      for (int p = 0; p < BATCH; ++p) {
        keep_raw(raw[p]);
        float z[8];
        unpack(raw[p], z);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if ((hits >> (8 * p + j)) & 1u) {
            if (at < sh.cap) sh.list[at] = order_entry(logit_key(clean_logit(z[j])), e[p] + j);
            ++at;
          }
      }
    }
  }
  __syncthreads();
  const int n = uniform(sh.n);
  return n > sh.cap ? -1 : n;
}

// Search of a running total over n numbers, digit by digit (9 bits, most
// significant first): the smallest key(i) of `bits` bits at which the sum of x(i)
// over the keys up to it reaches target (STRICT: exceeds it), or the largest key
// with x > 0 if none does.  x are integers, so the sums do not depend on the
// order in which LDS adds them.  Also the sums over smaller keys and over that
// key.  Workgroup-wide; thread t sees the numbers t, t + THREADS, ...
template <int THREADS, bool STRICT, typename K, typename X>
__device__ __forceinline__ uint32_t digit_search(int n, int bits, K key, X x, double target,
                                                 unsigned long long* bucket,
                                                 unsigned long long& before,
                                                 unsigned long long& inside) {
  constexpr int DIGIT = 9, PER = kBuckets / kWave;
  static_assert(kBuckets == 1 << DIGIT, "a bucket per digit");
  uint32_t prefix = 0;
  before = inside = 0;
  bool past = false;                                // no crossing: the last key
#pragma unroll 1
  for (int rest = bits; rest > 0;) {
    const int now = min(rest, DIGIT), shift = rest - now;
    for (int i = threadIdx.x; i < kBuckets; i += THREADS) bucket[i] = 0;
    __syncthreads();
#pragma unroll 1
    for (int i = threadIdx.x; i < n; i += THREADS) {
      const uint32_t d = key(i);
      if (rest == bits || d >> rest == prefix) {
        const unsigned long long v = x(i);
        if (v) atomicAdd(&bucket[(d >> shift) & ((1u << now) - 1)], v);
      }
    }
    __syncthreads();
    // every wave finds the same bucket: the lane whose eight buckets hold it,
    // then the bucket among those, a lane each
    const int l = lane_id();
    const auto over = [&](unsigned long long sum) {
      return STRICT ? (double)sum > target : (double)sum >= target;
    };
    const auto find = [&](unsigned long long x, unsigned long long& run) {
      // the first lane at whose x the total is over the target, else the last with any
      const unsigned long long hits = __ballot(x && !past && over(run + x)), any = __ballot(x != 0);
      const int src =
          uniform(hits ? __ffsll((long long)hits) - 1 : any ? 63 - __clzll((long long)any) : 0);
      past = past || !hits;
      run = of_lane(run, src);
      return src;
    };
    unsigned long long mine = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) mine += bucket[l * PER + i];
    unsigned long long run = wave_prefix(mine) + before - mine;
    const int lane = find(mine, run);
    const unsigned long long x8 = l < PER ? bucket[lane * PER + l] : 0;
    run += wave_prefix(x8) - x8;
    const int at = find(x8, run);
    prefix = prefix << now | (uint32_t)(lane * PER + at);
    before = run;
    inside = of_lane(x8, at);
    __syncthreads();
    rest -= now;
  }
  return prefix;
}
// Bits of the numbers 0 .. x, at least 1.
__device__ __forceinline__ int bits_of(uint32_t x) { return 32 - __clz((int)(x | 1u)); }

// What a list's cut came to.
enum ListCut { CUT_DONE, CUT_SHORT, CUT_AMBIGUOUS };

// Number of equal weights w, the first of which lies `before` into a running
// total, that start below target: at least 1, at most ties.
__device__ __forceinline__ int ties_below(double target, double before, double w, int ties) {
  const double need = w > 0.0 ? ceil((target - before) / w) : (double)ties;
  return need >= (double)ties ? ties : need < 1.0 ? 1 : (int)need;
}

// Top-k, top-p and min-p on n candidates in sh.list, and with `draw` the token
// of uniform u among the kept ones (sh.token).  sum: the row's sum of weights,
// or negative where the candidates' (after top-k) counts; slack: how far the
// target may be off; complete: the list holds every kept token.  Also got, the
// sum of the candidates' weights.
//
// Weights are integers in units of 2^-50 here (sums of 4096 of them fit 62
// bits and are exact whatever their order).
template <typename LT, int THREADS>
__device__ __forceinline__ ListCut cut_list(RowShared<THREADS>& sh, int n, const FilterSettings& s,
                                            int V, float m, uint32_t kt, double sum, double slack,
                                            bool complete, bool draw, float u, sv_filter_row& f,
                                            double& got) {
  static_assert(kCandFew <= 32 * 512 && kCand <= 32 * 256, "a bit per entry of a thread");
  constexpr double UNIT = 0x1p50;
  constexpr int W = THREADS / kWave;
  unsigned kept = ~0u;                              // bit i / THREADS: entry i
  const auto is_kept = [&](int i) { return (kept >> (i / THREADS)) & 1u; };
  const auto drop = [&](int i) { kept &= ~(1u << (i / THREADS)); };
  // how far below the maximum's a key lies: increases along the order; bf16
  // keys differ in their upper halves only
  constexpr int LOW = sizeof(LT) == 2 ? 16 : 0;
  const uint32_t kmax = logit_key(m) >> LOW;
  const int key_bits = bits_of(kmax - (kt >> LOW)), id_bits = bits_of((uint32_t)(V - 1));
  const auto digits = [&](int i) { return kmax - (~(uint32_t)(sh.list[i] >> 32) >> LOW); };
  const auto id = [&](int i) { return (uint32_t)sh.list[i]; };
  const auto weight_of = [&](int i) {
    return weight(key_logit(~(uint32_t)(sh.list[i] >> 32)), m, s.c, sh.table);
  };
  const auto one = [&](int i) { return (unsigned long long)is_kept(i); };
  const auto mass = [&](int i) {
    return is_kept(i) ? (unsigned long long)rint(weight_of(i) * UNIT) : 0ull;
  };
  const auto each = [&](auto f) {
#pragma unroll 1
    for (int i = threadIdx.x; i < n; i += THREADS) f(i);
  };
  unsigned long long before, inside;
  // of the kept entries: those before digits d, and of those with digits d the
  // first `keep` by index
  const auto cut_at = [&](uint32_t d, int keep, int ties) {
    uint32_t last = 0xffffffffu;
    if (keep < ties) {
      unsigned long long x, y;
      last = digit_search<THREADS, false>(
          n, id_bits, id, [&](int i) { return digits(i) == d ? one(i) : 0ull; }, (double)keep,
          sh.bucket, x, y);
    }
    each([&](int i) {
      const uint32_t e = digits(i);
      if (e > d || (e == d && id(i) > last)) drop(i);
    });
  };
  // sum, sum and maximum over the workgroup, in one go
  const auto reduce = [&](unsigned long long& a, unsigned long long& b, unsigned long long& c) {
    a = wave_reduce(a, OpAdd());
    b = wave_reduce(b, OpAdd());
    c = wave_reduce(c, OpMax());
    unsigned long long* red = reinterpret_cast<unsigned long long*>(sh.red);
    __syncthreads();
    if (lane_id() == 0) {
      const int w = threadIdx.x / kWave;
      red[w] = a;
      red[W + w] = b;
      red[2 * W + w] = c;
    }
    __syncthreads();
    a = red[0];
    b = red[W];
    c = red[2 * W];
#pragma unroll
    for (int i = 1; i < W; ++i) {
      a += red[i];
      b += red[W + i];
      c = max(c, red[2 * W + i]);
    }
    a = uniform(a);
    b = uniform(b);
    c = uniform(c);
  };
  __syncthreads();                                  // the queue is read, the list written
  if (s.k < n) {
    const uint32_t d =
        digit_search<THREADS, false>(n, key_bits, digits, one, (double)s.k, sh.bucket, before, inside);
    cut_at(d, s.k - (int)before, (int)inside);
  }
  if (s.p < 1.0) {
    unsigned long long total = 0, x = 0, y = 0;
    each([&](int i) { total += mass(i); });
    reduce(total, x, y);
    got = (double)total / UNIT;
    const double target = s.p * (sum >= 0.0 ? sum : got);
    if (!complete && got < target + slack) return CUT_SHORT;
    const uint32_t d = digit_search<THREADS, false>(n, key_bits, digits, mass, target * UNIT,
                                                    sh.bucket, before, inside);
    // the tokens with digits d, and their weight
    unsigned long long ties = 0, w_bits = 0;
    x = 0;
    each([&](int i) {
      if (is_kept(i) && digits(i) == d) {
        ++ties;
        w_bits = (unsigned long long)__double_as_longlong(weight_of(i));
      }
    });
    reduce(ties, x, w_bits);
    const double w = __longlong_as_double((long long)w_bits), ahead = (double)before / UNIT;
    const int keep = ties_below(target, ahead, w, (int)ties);
    if (slack > 0.0 && (target - (ahead + (keep - 1) * w) <= slack ||
                        ahead + keep * w - target <= slack))
      return CUT_AMBIGUOUS;
    cut_at(d, keep, (int)ties);
  }
  if (s.mp > 0.0)
    each([&](int i) { if (weight_of(i) < s.mp) drop(i); });
  // the kept entries' sum, number and last one
  unsigned long long total = 0, count = 0, last = 0;
  each([&](int i) {
    total += mass(i);
    if (is_kept(i)) { ++count; last = max(last, sh.list[i]); }
  });
  reduce(total, count, last);
  f.inv_sum = UNIT / (double)total;
  f.min_kept = key_logit(~(uint32_t)(last >> 32));
  f.last = (int)(uint32_t)last;
  f.n_kept = (int)count;
  if (draw) {
    const uint32_t t = digit_search<THREADS, true>(n, id_bits, id, mass,
                                                   (double)uniform(u) * (double)total, sh.bucket, before,
                                                   inside);
    if (threadIdx.x == 0) sh.token = (int)t;
    __syncthreads();
  }
  return CUT_DONE;
}

// The same for a short list by the first wave, two entries a lane, without
// barriers but the last: entries sorted by counting the smaller ones, running
// totals by wave scans in fp64.
template <int THREADS>
__device__ __forceinline__ ListCut cut_short_list(RowShared<THREADS>& sh, int n,
                                                  const FilterSettings& s, float m, double sum,
                                                  double slack, bool complete, bool draw, float u,
                                                  sv_filter_row& f, double& got) {
  __syncthreads();                                  // the queue is read, the list written
  if (threadIdx.x < kWave) {
    const int l = lane_id();
    auto& so = sh.sorted;
    const unsigned long long e0 = l < n ? sh.list[l] : ~0ull;
    const unsigned long long e1 = l + kWave < n ? sh.list[l + kWave] : ~0ull;
    int r0 = 0, r1 = 0;
    if (n <= kWave) {
#pragma unroll 4
      for (int j = 0; j < n; ++j) r0 += sh.list[j] < e0;
    } else {
#pragma unroll 4
      for (int j = 0; j < n; ++j) {
        const unsigned long long y = sh.list[j];
        r0 += y < e0;
        r1 += y < e1;
      }
    }
    if (l < n) so.entry[r0] = e0;
    if (l + kWave < n) so.entry[r1] = e1;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    // lane l: places 2l and 2l + 1 of the order
    const int nk = min(n, s.k);
    unsigned long long e[2];
    double w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      e[i] = 2 * l + i < n ? so.entry[2 * l + i] : 0;
      w[i] = 2 * l + i < nk ? weight(key_logit(~(uint32_t)(e[i] >> 32)), m, s.c, sh.table) : 0.0;
    }
    const double incl = wave_prefix(w[0] + w[1]);
    const double total = of_lane(incl, kWave - 1);
    const double run0 = incl - (w[0] + w[1]), run1 = run0 + w[0];
    const double target = s.p * (sum >= 0.0 ? sum : total);
    ListCut c = CUT_DONE;
    int keep = 0;
    if (s.p < 1.0 && !complete && total < target + slack) {
      c = CUT_SHORT;
    } else {
      bool k[2];
      int most = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const double run = i ? run1 : run0;
        const bool in = 2 * l + i < nk && w[i] >= s.mp;
        k[i] = in && (s.p >= 1.0 || run < target - slack);
        most += in && (s.p >= 1.0 || run < target + slack);
        keep += k[i];
      }
      keep = wave_reduce(keep, OpAdd());
      if (slack > 0.0) {
        most = wave_reduce(most, OpAdd());
        if (most != keep) c = CUT_AMBIGUOUS;
      }
      if (c == CUT_DONE) {
        const double part = (k[0] ? w[0] : 0.0) + (k[1] ? w[1] : 0.0);
        const double S = wave_reduce(part, OpAdd());
        const unsigned long long last = so.entry[keep - 1];
        f.inv_sum = 1.0 / S;
        f.min_kept = key_logit(~(uint32_t)(last >> 32));
        f.last = (int)(uint32_t)last;
        f.n_kept = keep;
        if (draw) {
          // the kept entries by index
          int q0 = 0, q1 = 0;
#pragma unroll 4
          for (int j = 0; j < keep; ++j) {
            const uint32_t y = (uint32_t)so.entry[j];
            q0 += y < (uint32_t)e[0];
            q1 += y < (uint32_t)e[1];
          }
          if (k[0]) { so.w[q0] = w[0]; so.id[q0] = (int)(uint32_t)e[0]; }
          if (k[1]) { so.w[q1] = w[1]; so.id[q1] = (int)(uint32_t)e[1]; }
          __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
          double x[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) x[i] = 2 * l + i < keep ? so.w[2 * l + i] : 0.0;
          const double at = wave_prefix(x[0] + x[1]);
          const double goal = (double)uniform(u) * of_lane(at, kWave - 1);
          const double before = at - (x[0] + x[1]);
          int first = INT32_MAX, any = -1;
          if (x[0] > 0.0) { any = 2 * l; if (before + x[0] > goal) first = 2 * l; }
          if (x[1] > 0.0) { any = 2 * l + 1; if (at > goal) first = min(first, 2 * l + 1); }
          first = wave_reduce(first, OpMin());
          any = wave_reduce(any, OpMax());
          if (l == 0) sh.token = so.id[first == INT32_MAX ? any : first];
        }
      }
    }
    if (l == 0) {
      sh.found = c;
      sh.got = total;
      sh.row = f;
    }
  }
  __syncthreads();
  f.inv_sum = uniform(sh.row.inv_sum);
  f.min_kept = uniform(sh.row.min_kept);
  f.last = uniform(sh.row.last);
  f.n_kept = uniform(sh.row.n_kept);
  got = uniform(sh.got);
  return (ListCut)uniform(sh.found);
}

// The kept set of one row through the candidate list, and with `draw` the token
// of uniform u.  Returns false where the row has to take the general path
// (filter_row): more candidates than the list holds, or a large top-k.  The
// candidates (the kept tokens and some more) stay in sh.list[0 .. count); count
// is -1 for rows without a list, whose token is not drawn here.
template <typename LT, int THREADS, bool PRE>
__device__ __forceinline__ bool filter_row_list(const FilterLaunch& A, long r, const LT* row, int V,
                                                const FilterSettings& s, bool draw, float u,
                                                uint16_t* gm, RowShared<THREADS>& sh,
                                                sv_filter_row& f, int& count) {
  const int G = A.group_octets;
  const int tiles = (V + kRowTile - 1) / kRowTile;
  const int groups = tiles * (kRowTile / 8) / G;
  const bool by_k = s.k < V;
  const bool all = V <= kCand;                      // every token fits the list
  const bool need_sum = row_needs_sum(s, V);
  const bool nucleus = need_sum && !s.off;
  count = -1;
  if (by_k && !all && s.k > kMaxListK) return false;
  // The sum of a nucleus row is first taken in fp32 (unless a kernel of its own
  // took it in fp64), and again in fp64 where its error could move the cut.
  constexpr bool TWICE = !PRE;
#pragma unroll 1
  for (bool exact = !TWICE || !nucleus;; exact = true) {
    float top = -INFINITY;
    if constexpr (PRE) load_streamed<THREADS>(A, r, groups, tiles, need_sum, gm, sh, top);
    else if (!need_sum) stream_row<LT, THREADS, NO_SUM>(row, V, s.c, G, gm, sh, top);
    else if (!TWICE || exact) stream_row<LT, THREADS, SUM_F64>(row, V, s.c, G, gm, sh, top);
    else stream_row<LT, THREADS, SUM_F32>(row, V, s.c, G, gm, sh, top);
    const float m = block_reduce<THREADS>(top, reinterpret_cast<float*>(sh.redi), OpMax());
    f = sv_filter_row{s.c, 0.0, m, INFINITY, -1, 0};
    if (m == -INFINITY) { count = 0; return true; }
    double S = -1.0;                                // the sum of all weights
    if (need_sum) {
      double part = 0.0;
#pragma unroll 1
      for (int t = threadIdx.x; t < tiles; t += THREADS) {
        const double x = sh.tile_m[t] > -INFINITY
                             ? sh.tile_s[t] * weight(sh.tile_m[t], m, s.c, sh.table) : 0.0;
        sh.tile_s[t] = x;
        part += x;
      }
      S = block_reduce<THREADS>(part, sh.red, OpAdd());
      if (s.off) {
        f.inv_sum = 1.0 / S;
        f.min_kept = -INFINITY;
        f.last = V - 1;
        f.n_kept = V;
        return true;
      }
    }
    // The fp32 sum's error: 2^-19 covers terms of |x| < 20; those below weigh
    // under 2^-20.
    const double slack = !TWICE || exact ? 0.0 : s.p * S * 0x1p-19;
    // the lowest key a kept token can have
    const uint32_t kmax = logit_key(m);
    uint32_t mp_key = kKeyNegInf + 1;
    if (s.mp > 0.0 && s.c > 0.0) {
      // z >= m + log2(min_p) / c, a little lower: the exact test follows
      const float z =
          (float)((double)m + ((double)__builtin_amdgcn_logf(uniform(s.mp)) - 1e-4) / s.c);
      mp_key = max(mp_key, min(kmax, logit_key(clean_logit(z)) - 2));
    }
    bool complete = true;                           // the list holds every kept token
    bool first = false;
    double got = 0.0;
    uint32_t kt = kKeyNegInf + 1;
    ListCut cut = CUT_SHORT;
#pragma unroll 1
    for (int attempt = 0; attempt < 8; ++attempt) {
      if (!all) {
        if (by_k || nucleus) {
          // A nucleus row's share p of the sum, and a tenth of the rest, is
          // estimated from the group maxima (without that tenth half of the rows
          // need a second turn: 60 against 50 us for 64 rows); what the tokens
          // found lack of it, and a tenth more, from those below.  Heavy tokens behind heavier ones of their group are
          // missing from the first estimate: where it gave too many tokens,
          // those of the kFirst largest groups come first.
          const bool est = nucleus && !first, more = est && got > 0.0;
          const int k = nucleus ? (est ? 0 : min(kFirst, groups)) : s.k;
          const float z0 = more ? key_logit(kt) : m;
          const double lack = more ? 1.1 * (s.p * S - got) : (0.9f * uniform(s.p) + 0.1f) * S;
          const float aim = est ? (float)(lack / weight(z0, m, s.c, sh.table)) : 0.f;
          kt = (s.k == 1 ? kmax >> 16
                         : threshold_key<LT, THREADS>(
                               gm, groups, (more ? kt : kmax + 0x10000u) / 0x10000u - 1,
                               more ? uniform(sh.nq) : 0, z0, (float)s.c, k, aim, sh))
               << 16;
          complete = !nucleus || kt <= mp_key;
          if (nucleus || s.p >= 1.0) kt = max(kt, mp_key);
        } else {
          kt = mp_key;
        }
      }
      const int n = gather_tokens<LT, THREADS>(row, V, G, groups, gm, kt, sh);
      if (n < 0) {
        if (!nucleus || attempt > 0) return false;
        first = true;
        continue;
      }
      first = false;
      count = n;
      cut = n <= kWaveList
                ? cut_short_list<THREADS>(sh, n, s, m, S, slack, complete, draw, u, f, got)
                : cut_list<LT, THREADS>(sh, n, s, V, m, kt, S, slack, complete, draw, u, f, got);
      if (cut != CUT_SHORT) break;
    }
    if (cut == CUT_SHORT) return false;
    __syncthreads();
    if (cut == CUT_DONE) {
      if (s.off) {
        f.min_kept = -INFINITY;
        f.last = V - 1;
        f.n_kept = V;
      }
      return true;
    }
  }
}

// The tile in which the running total of the tiles' masses first exceeds
// target (the last with mass if rounding leaves none; -1 if none has mass), and
// the total before it.  Every wave finds the same.
__device__ __forceinline__ int find_tile(const double* mass, int tiles, float u, double& target,
                                         double& before) {
  constexpr int PER = kRowTiles / kWave;
  const int l = lane_id();
  double x[PER], mine = 0.0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    x[i] = l * PER + i < tiles ? mass[l * PER + i] : 0.0;
    mine += x[i];
  }
  const double incl = wave_prefix(mine);
  target = (double)uniform(u) * of_lane(incl, kWave - 1);
  double run = incl - mine, at = 0.0;
  int hit = -1, any = -1;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (x[i] > 0.0) {
      any = l * PER + i;
      if (hit < 0 && run + x[i] > target) { hit = l * PER + i; at = run; }
    }
    run += x[i];
  }
  const unsigned long long hits = __ballot(hit >= 0), anys = __ballot(any >= 0);
  if (!anys) return -1;
  const int src = hits ? __ffsll((long long)hits) - 1 : 63 - __clzll((long long)anys);
  before = __shfl(at, src);
  if (!hits) target = INFINITY;                     // its last token with mass
  return __shfl(hits ? hit : any, src);
}

// The token of tile t at which the running total, `before` ahead of the tile,
// exceeds target; the tile's last with mass if none does.
template <int THREADS, typename F>
__device__ __forceinline__ int find_in_tile(int t, int V, double before, double target, double* red,
                                            int* redi, F mass) {
  constexpr int PER = kRowTile / THREADS;
  const int e0 = t * kRowTile + threadIdx.x * PER;
  double x[PER], part = 0.0, total;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    x[j] = e0 + j < V ? mass(e0 + j) : 0.0;
    part += x[j];
  }
  double run = before + block_scan<THREADS>(part, red, total);
  int first = INT32_MAX, any = -1;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    run += x[j];
    if (x[j] > 0.0) {
      any = e0 + j;
      if (run > target) first = min(first, e0 + j);
    }
  }
  first = block_reduce<THREADS>(first, redi, OpMin());
  any = block_reduce<THREADS>(any, redi, OpMax());
  return first == INT32_MAX ? any : first;
}

// The token drawn from a row without filters, whose tile masses are in
// sh.tile_s.
template <typename LT, int THREADS>
__device__ __forceinline__ int draw_tiles(const LT* row, int V, RowShared<THREADS>& sh, float u,
                                          float m, double c) {
  double target, before = 0.0;
  const int t = find_tile(sh.tile_s, (V + kRowTile - 1) / kRowTile, u, target, before);
  return find_in_tile<THREADS>(t, V, before, target, sh.red, sh.redi, [&](int e) {
    return weight(clean_logit(logit_at(row, e)), m, c, sh.table);
  });
}

// The stream of few rows by all CUs: one wave per tile.
constexpr int kStreamThreads = 256;
template <typename LT>
__global__ __launch_bounds__(kStreamThreads) void filter_stream_kernel(FilterLaunch A) {
  __shared__ ExpEntry table[kExpTable];
  const long r = blockIdx.x;
  const int V = A.V, G = A.group_octets;
  const int tiles = (V + kRowTile - 1) / kRowTile;
  int errors = 0;
  const FilterSettings s = filter_settings(A.temperatures, A.temperature, A.top_ks, A.top_ps,
                                           A.min_ps, (int)(r / A.per_seq), V, errors);
  const long ri = A.row_index ? (long)A.row_index[r] : r;
  if (ri < 0 || ri >= A.n_rows) return;
  const LT* row = static_cast<const LT*>(A.logits) + ri * A.row_stride;
  const bool sum = row_needs_sum(s, V);
  if (sum) {                                        // uniform
    fill_exp_table(table);
    __syncthreads();
  }
  const int t = blockIdx.y * (kStreamThreads / kWave) + threadIdx.x / kWave;
  if (t >= tiles) return;
  uint16_t* gm = A.group_key + r * ((long)tiles * (kRowTile / 8) / G);
  float* tm = A.tile_max + r * tiles + t;
  double* ts = A.tile_sum + r * tiles + t;
  float top = -INFINITY;
  if (sum) stream_tile<LT, SUM_F64>(row, V, t, s.c, G, gm, tm, ts, table, top);
  else stream_tile<LT, NO_SUM>(row, V, t, s.c, G, gm, tm, ts, table, top);
  top = wave_reduce(top, OpMax());
  if (lane_id() == 0) *tm = top;
}

// Sets up a workgroup's LDS: RowShared, the list of `cap` entries, the groups'
// keys (returned).
template <int THREADS>
__device__ __forceinline__ uint16_t* row_shared(unsigned char* lds, int cap, RowShared<THREADS>& sh) {
  unsigned long long* list = reinterpret_cast<unsigned long long*>(lds + sizeof(RowShared<THREADS>));
  fill_exp_table(sh.table);
  if (threadIdx.x == 0) {
    sh.list = list;
    sh.cap = cap;
  }
  return reinterpret_cast<uint16_t*>(list + cap);
}

// A row by the general path: the kept set by radix searches over the whole row,
// the token by its tiles' masses.
template <typename LT, int THREADS>
__device__ __forceinline__ sv_filter_row general_row(const LT* row, int V, const FilterSettings& s,
                                                     bool draw, float u, unsigned char* lds,
                                                     int& token) {
  __syncthreads();
  const sv_filter_row f =
      filter_row<LT, THREADS>(row, V, s, *reinterpret_cast<FilterShared<THREADS>*>(lds));
  token = 0;                                        // of an empty row
  if (draw && f.n_kept > 0)
    token = block_draw<THREADS>(V, u, *reinterpret_cast<DrawShared*>(lds), [&](int e) {
      const float z = clean_logit(logit_at(row, e));
      return row_keeps(f, z, e) ? weight(z, f.max, f.scale) : 0.0;
    });
  return f;
}

// The dense q of a row from its filter row alone.
template <typename LT, int THREADS>
__device__ __forceinline__ void write_probs(const LT* row, int V, const sv_filter_row& f, float* q) {
  for (int e = threadIdx.x; e < V; e += THREADS)
    __builtin_nontemporal_store((float)row_prob(f, logit_at(row, e), e), q + e);
}

// Row r by one workgroup.  PRE: the row was streamed by filter_stream_kernel.
// GENERAL: rows that do not fit the list are done here as well; otherwise they are
// left to filter_left_kernel.
template <typename LT, int THREADS, bool PRE, bool GENERAL>
__device__ __forceinline__ void filter_one_row(const FilterLaunch& A, long r, unsigned char* lds) {
  RowShared<THREADS>& sh = *reinterpret_cast<RowShared<THREADS>*>(lds);
  const int b = (int)(r / A.per_seq);
  const int V = A.V;
  int errors = 0;
  FilterSettings s = filter_settings(A.temperatures, A.temperature, A.top_ks, A.top_ps, A.min_ps,
                                     b, V, errors);
  s.c = uniform(s.c);
  s.p = uniform(s.p);
  s.mp = uniform(s.mp);
  s.k = uniform(s.k);
  const long ri = A.row_index ? (long)A.row_index[r] : r;
  const bool there = ri >= 0 && ri < A.n_rows;
  sv_filter_row f{0.0, 0.0, -INFINITY, INFINITY, -1, 0};
  const LT* row = static_cast<const LT*>(A.logits) + (there ? ri : 0) * A.row_stride;
  const bool sampled = A.out_tokens && s.c != 0.0;
  const float u = sampled ? A.uniforms[r] : 0.f;
  uint16_t* gm = row_shared<THREADS>(lds, A.list_cap, sh);
  if (A.pending && r == 0 && threadIdx.x == 0) *A.pending = 0;
  __syncthreads();
  int count = 0;                                    // candidates in sh.list; -1: no list
  int token = there ? 0 : -1;
  if (there) {
    if (filter_row_list<LT, THREADS, PRE>(A, r, row, V, s, sampled, u, gm, sh, f, count)) {
      if (f.n_kept > 0) {
        if (s.c == 0.0) token = f.last;
        else if (!sampled) token = 0;
        else if (count >= 0) token = sh.token;
        else token = draw_tiles<LT, THREADS>(row, V, sh, u, f.max, s.c);
      }
    } else {
      if constexpr (!GENERAL) {
        if (threadIdx.x == 0) A.list_counts[r] = kGeneralRow;
        return;
      } else {
        f = general_row<LT, THREADS>(row, V, s, sampled, u, lds, token);
        if (s.c == 0.0 && f.n_kept > 0) token = f.last;
        count = -1;
      }
    }
  }
  if (!there) errors |= SV_DEVERR_ROW_INDEX;
  else if (f.n_kept == 0) errors |= SV_DEVERR_EMPTY_ROW;
  if (threadIdx.x == 0) {
    if (errors) flag_error(A.device_error, errors);
    if (A.out_rows) A.out_rows[r] = f;
    A.list_counts[r] = count <= kCand ? count : -1;
    if (A.out_tokens) A.out_tokens[r] = token;
  }
  if (A.lists && count <= kCand)
    for (int i = threadIdx.x; i < count; i += THREADS)
      A.lists[r * kCand + i] = (int32_t)(uint32_t)sh.list[i];
  if (A.out_probs) {
    float* q = A.out_probs + r * V;
    if (count >= 0) {
      for (int e = threadIdx.x; e < V; e += THREADS) __builtin_nontemporal_store(0.f, q + e);
      __syncthreads();                              // the kept tokens' own values after the zeros
      for (int i = threadIdx.x; i < count; i += THREADS) {
        const unsigned long long x = sh.list[i];
        const float z = key_logit(~(uint32_t)(x >> 32));
        if (row_keeps(f, z, (uint32_t)x))
          q[(uint32_t)x] = (float)(weight(z, f.max, f.scale, sh.table) * f.inv_sum);
      }
    } else {
      write_probs<LT, THREADS>(row, V, f, q);
    }
  }
}

template <typename LT, int THREADS, bool PRE, bool GENERAL>
__global__ __launch_bounds__(THREADS) __attribute__((amdgpu_waves_per_eu(4))) void
filter_rows_kernel(FilterLaunch A) {
  extern __shared__ __align__(16) unsigned char lds[];
  filter_one_row<LT, THREADS, PRE, GENERAL>(A, blockIdx.x, lds);
}

// The rows that filter_rows_kernel left (their counts say so) with a longer list
// and, where that does not do, by the general path: each workgroup looks at the
// counts of rows a grid apart, all at once, and takes those left in turn.
constexpr int kLeftThreads = 512;
template <typename LT>
__global__ __launch_bounds__(kLeftThreads) __attribute__((amdgpu_waves_per_eu(2))) void
filter_left_kernel(FilterLaunch A) {
  extern __shared__ __align__(16) unsigned char lds[];
  __shared__ unsigned long long left[kLeftThreads / kWave];
  const long rows = (long)A.B * A.per_seq, step = gridDim.x;
#pragma unroll 1
  for (long base = blockIdx.x; base < rows; base += step * kLeftThreads) {
    const long mine = base + threadIdx.x * step;
    const unsigned long long mask = __ballot(mine < rows && A.list_counts[mine] == kGeneralRow);
    if (lane_id() == 0) left[threadIdx.x / kWave] = mask;
    __syncthreads();
#pragma unroll 1
    for (int w = 0; w < kLeftThreads / kWave; ++w) {
#pragma unroll 1
      for (unsigned long long m = uniform(left[w]); m; m &= m - 1) {
        const int i = w * kWave + __ffsll((long long)m) - 1;
        filter_one_row<LT, kLeftThreads, false, true>(A, base + i * step, lds);
        __syncthreads();
      }
    }
    __syncthreads();
  }
}

// q of the drafts of one sequence, dense or from the drafter's logits.
template <typename LT, bool QL>
struct DrafterQ {
  const float* probs;                // draft k's row of dense q
  const LT* logits;                  // its drafter row, NULL if there is none (q = 0)
  sv_filter_row row;
  bool missing;
  __device__ __forceinline__ DrafterQ(const FilteredVerifyLaunch& A, int b, int k) {
    const long i = (long)b * A.K + k;
    missing = false;
    if constexpr (QL) {
      const long dr = A.drows ? (long)A.drows[i] : i;
      missing = dr < 0 || dr >= A.d_rows;
      logits = missing ? nullptr : static_cast<const LT*>(A.dlogits) + dr * A.d_stride;
      row = A.ddesc[i];
    } else {
      probs = A.draft_probs + i * A.V;
    }
  }
  __device__ __forceinline__ double at(int x) const {
    if constexpr (QL) return logits ? row_prob(row, logit_at(logits, x), x) : 0.0;
    else return (double)probs[x];
  }
};

// The accept scan and, where the row of the first rejection has a list, the new
// token; other sequences are left to residual_kernel.
template <typename LT, bool QL>
__global__ __launch_bounds__(kVerifyThreads) void filtered_verify_kernel(FilteredVerifyLaunch A) {
  __shared__ double red[kVerifyThreads / kWave];
  __shared__ unsigned long long bucket[kBuckets];
  __shared__ double mass[kCand];
  __shared__ int id[kCand];
  __shared__ int sh_a;
  const int b = blockIdx.x, K = A.K, V = A.V;
  const int l = lane_id();
  const long row0 = (long)b * (K + 1);
  const LT* z0 = static_cast<const LT*>(A.logits) + row0 * A.row_stride;
  int errors = 0;
  if (threadIdx.x < kWave) {
    bool accepted = false;
    if (l < K) {
      const sv_filter_row f = A.rows[row0 + l];
      const int x = A.draft_tokens[(long)b * K + l];
      double p = 0.0;
      if (x >= 0 && x < V) {
        p = row_prob(f, logit_at(z0 + l * A.row_stride, x), x);
        if (f.scale == 0.0) {                        // greedy
          accepted = x == f.last;
        } else if (p > 0.0) {
          const DrafterQ<LT, QL> q(A, b, l);
          if (q.missing) errors |= SV_DEVERR_ROW_INDEX;
          accepted = (double)A.uniforms[row0 + l] * q.at(x) < p;
        }
      } else {
        errors |= SV_DEVERR_DRAFT_TOKEN;
      }
      if (A.out_p) A.out_p[(long)b * K + l] = (float)p;
    }
    const unsigned long long ok = __ballot(accepted);
    const int a = __ffsll((long long)~ok) - 1;       // K <= 63: lane K is never accepted
    if (l < a) A.out_tokens[row0 + l] = A.draft_tokens[(long)b * K + l];
    else if (l > a && l <= K) A.out_tokens[row0 + l] = -1;
    if (l == 0) { sh_a = a; A.out_num_accepted[b] = a; }
    if (errors) flag_error(A.device_error, errors);
  }
  __syncthreads();
  const int a = sh_a;
  const sv_filter_row f = A.rows[row0 + a];
  const LT* za = z0 + (long)a * A.row_stride;
  int token = 0;                                     // of an empty row
  if (f.n_kept > 0 && f.scale == 0.0) {
    token = f.last;
  } else if (f.n_kept > 0) {
    const float u = A.uniforms[row0 + K];
    const int count = A.list_counts[row0 + a];
    if (count < 0) {
      if (threadIdx.x == 0) {
        A.done[b] = 0;
        A.pending[1 + atomicAdd(A.pending, 1)] = b;
      }
      return;
    }
    const int32_t* list = A.lists + (row0 + a) * kCand;
    // the residual's masses, and p's
    const auto each = [&](auto f) {
      for (int i = threadIdx.x; i < count; i += kVerifyThreads) f(i);
    };
    double most = 0.0;
    each([&](int i) {
      const int x = list[i];
      id[i] = x;
      mass[i] = row_prob(f, logit_at(za, x), x);
    });
    if (a < K) {
      const DrafterQ<LT, QL> q(A, b, a);
      each([&](int i) {
        if (mass[i] > 0.0) most = fmax(most, mass[i] - q.at(id[i]));
      });
      most = block_reduce<kVerifyThreads>(most, red, OpMax());
      if (most > 0.0)
        each([&](int i) {
          mass[i] = mass[i] > 0.0 ? fmax(0.0, mass[i] - q.at(id[i])) : 0.0;
        });
    }
    if (!(most > 0.0)) {                             // a = K, or q covers p
      each([&](int i) { most = fmax(most, mass[i]); });
      most = block_reduce<kVerifyThreads>(most, red, OpMax());
    }
    // as integers, the largest between 2^50 and 2^51
    const int up = 50 - ilogb(most);
    unsigned long long total = 0, before, inside;
    each([&](int i) {
      const unsigned long long x = (unsigned long long)rint(ldexp(mass[i], up));
      mass[i] = __longlong_as_double(x);
      total += x;
    });
    total = block_reduce<kVerifyThreads>(total, reinterpret_cast<unsigned long long*>(red), OpAdd());
    __syncthreads();
    token = (int)digit_search<kVerifyThreads, true>(
        count, bits_of((uint32_t)(V - 1)), [&](int i) { return (uint32_t)id[i]; },
        [&](int i) { return (unsigned long long)__double_as_longlong(mass[i]); },
        (double)u * (double)total, bucket, before, inside);
  }
  if (threadIdx.x == 0) A.out_tokens[row0 + a] = token;
}

// The new tokens of the sequences whose row a has no list (no filter, or a
// nucleus of thousands): the residual's and p's mass of every tile of the row,
// one workgroup per tile over all CUs; the one that finishes a sequence's last
// tile finds the token.
template <typename LT, bool QL>
__global__ __launch_bounds__(kVerifyThreads) void residual_kernel(FilteredVerifyLaunch A) {
  constexpr int WAVES = kVerifyThreads / kWave, OCTS = kRowTile / kTile / WAVES;
  __shared__ ExpEntry table[kExpTable];
  __shared__ double red[WAVES], red2[WAVES];
  __shared__ int redi[WAVES];
  __shared__ double mass[kRowTiles];
  __shared__ int sh_last;
  const int pending = A.pending[0];
  const int K = A.K, V = A.V;
  const int tiles = (V + kRowTile - 1) / kRowTile;
  if ((long)blockIdx.x >= (long)pending * tiles) return;
  fill_exp_table(table);
  __syncthreads();
  const int w = threadIdx.x / kWave, l = lane_id();
  for (long item = blockIdx.x; item < (long)pending * tiles; item += gridDim.x) {
    const int b = A.pending[1 + item / tiles];
    const long row0 = (long)b * (K + 1);
    const int a = A.out_num_accepted[b];
    const sv_filter_row f = A.rows[row0 + a];
    const LT* za = static_cast<const LT*>(A.logits) + (row0 + a) * A.row_stride;
    const bool residual = a < K;
    const DrafterQ<LT, QL> q(A, b, residual ? a : 0);
    double* rmass = A.tile_mass + (long)b * 2 * tiles;
    double* pmass = rmass + tiles;
    const auto p_at = [&](float z, int x) {
      z = clean_logit(z);
      return row_keeps(f, z, x) ? weight(z, f.max, f.scale, table) * f.inv_sum : 0.0;
    };
    const auto q_of = [&](float z, int x) {          // from the drafter's logit
      z = clean_logit(z);
      return row_keeps(q.row, z, x) ? weight(z, q.row.max, q.row.scale, table) * q.row.inv_sum
                                    : 0.0;
    };
    const auto q_at = [&](int x) {
      if constexpr (QL) {
        return q.logits ? q_of(logit_at(q.logits, x), x) : 0.0;
      } else {
        return (double)q.probs[x];
      }
    };
    const auto r_at = [&](int x) {
      const double p = p_at(logit_at(za, x), x);
      return p > 0.0 ? fmax(0.0, p - q_at(x)) : 0.0;
    };
    const int t = (int)(item % tiles);
    double rs = 0.0, ps = 0.0;
    // a lane's octets of the tile and of q together
    Raw<LT> rz[OCTS], rq[OCTS];
    float qf[OCTS][8];
    const int e0 = t * kRowTile + w * OCTS * kTile + 8 * l;
#pragma unroll
    for (int i = 0; i < OCTS; ++i) {
      const int e = e0 + i * kTile;
      if (e + 8 <= V) raw8(za + e, rz[i]);
      else raw8_end(za, e, V, rz[i]);
      if (residual) {
        if constexpr (QL) {
          if (q.logits) {
            if (e + 8 <= V) raw8(q.logits + e, rq[i]);
            else raw8_end(q.logits, e, V, rq[i]);
          }
        } else if (e + 8 <= V) {
          load8(q.probs + e, qf[i]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) qf[i][j] = e + j < V ? q.probs[e + j] : 0.f;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < OCTS; ++i) {
      const int e = e0 + i * kTile;
      float z[8], zq[8];
      unpack(rz[i], z);
      if constexpr (QL) unpack(rq[i], zq);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double p = e + j < V ? p_at(z[j], e + j) : 0.0;
        ps += p;
        if (residual && p > 0.0) {
          double x;
          if constexpr (QL) x = q.logits ? q_of(zq[j], e + j) : 0.0;
          else x = (double)qf[i][j];
          rs += fmax(0.0, p - x);
        }
      }
    }
    rs = wave_reduce(rs, OpAdd());
    ps = wave_reduce(ps, OpAdd());
    if (l == 0) { red[w] = rs; red2[w] = ps; }
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
      for (int i = 1; i < WAVES; ++i) { rs += red[i]; ps += red2[i]; }
      st_coherent(rmass + t, rs);
      st_coherent(pmass + t, ps);
      wait_stores_performed();
      sh_last = atomicAdd(&A.done[b], 1) == tiles - 1;
    }
    __syncthreads();
    if (sh_last) {                                   // uniform
      const float u = A.uniforms[row0 + K];
      double target, before = 0.0;
      int tile = -1;
      if (residual) {
        for (int i = threadIdx.x; i < tiles; i += kVerifyThreads) mass[i] = ld_coherent(rmass + i);
        __syncthreads();
        tile = find_tile(mass, tiles, u, target, before);
      }
      int token;
      if (tile >= 0) {
        token = find_in_tile<kVerifyThreads>(tile, V, before, target, red, redi, r_at);
      } else {                                       // a = K, or q covers p
        __syncthreads();
        for (int i = threadIdx.x; i < tiles; i += kVerifyThreads) mass[i] = ld_coherent(pmass + i);
        __syncthreads();
        tile = find_tile(mass, tiles, u, target, before);
        token = find_in_tile<kVerifyThreads>(tile, V, before, target, red, redi,
                                             [&](int x) { return p_at(logit_at(za, x), x); });
      }
      if (threadIdx.x == 0) A.out_tokens[row0 + a] = token;
    }
    __syncthreads();
  }
}

}  // namespace

namespace {

// Few rows take workgroups of 512 threads; where they are long, their stream
// gets a kernel of its own, spread over all CUs.  For rows of 151936 in bf16 and
// the one kind against the other: 513 rows 68 against 54 us under top-k, 85
// against 152 with top-p in half of them, 85 against 109 without a filter; 1024
// rows 111 against 79, 180 against 195, 144 against 146; 2048 rows 220 against 143,
// 347 against 249, 277 against 253.
bool few_rows(long rows) { return rows <= 512; }
bool streams_apart(long rows, int V) { return few_rows(rows) && V > 16 * kRowTile; }

// The parts of the workspace, in order; each starts at a multiple of 16 bytes.
struct FilterWorkspace {
  size_t rows = 0, counts = 0, lists = 0, pending = 0, done = 0, tile_mass = 0;
  size_t group_key = 0, tile_max = 0, tile_sum = 0, bytes = 0;
  FilterWorkspace(long n, int V, bool verify) {
    const size_t tiles = (V + kRowTile - 1) / kRowTile;
    size_t at = 0;
    const auto part = [&](size_t& where, size_t size) {
      where = at;
      at += (size + 15) / 16 * 16;
    };
    part(counts, n * sizeof(int32_t));
    if (verify) {
      part(rows, n * sizeof(sv_filter_row));
      part(lists, n * kCand * sizeof(int32_t));
      // no more sequences than rows
      part(pending, (n + 1) * sizeof(int32_t));
      part(done, n * sizeof(int32_t));
      part(tile_mass, n * 2 * tiles * sizeof(double));
    }
    if (streams_apart(n, V)) {
      part(group_key, n * tiles * (kRowTile / 8) / group_octets(V, kGroupsFew) * sizeof(uint16_t));
      part(tile_max, n * tiles * sizeof(float));
      part(tile_sum, n * tiles * sizeof(double));
    }
    bytes = at;
  }
};

// The LDS of a workgroup that takes rows, and its list's length: as much as 64 KB
// hold where it also does the general path.
template <int THREADS, bool GENERAL>
size_t row_lds(FilterLaunch& L) {
  const size_t tiles = (L.V + kRowTile - 1) / kRowTile;
  const size_t keys = tiles * (kRowTile / 8) / L.group_octets * sizeof(uint16_t);
  const size_t fixed = sizeof(RowShared<THREADS>) + keys, entry = sizeof(unsigned long long);
  L.list_cap = GENERAL ? (int)std::min((size_t)kCandFew, (65024 - fixed) / entry) : kCand;
  return std::max(fixed + L.list_cap * entry, GENERAL ? sizeof(FilterShared<THREADS>) : 0);
}
template <typename LT, int THREADS, bool PRE, bool GENERAL>
void launch_rows(FilterLaunch L, hipStream_t stream) {
  const size_t lds = row_lds<THREADS, GENERAL>(L);
  filter_rows_kernel<LT, THREADS, PRE, GENERAL>
      <<<dim3((unsigned)((long)L.B * L.per_seq)), THREADS, lds, stream>>>(L);
}

template <typename LT>
hipError_t launch_filter(FilterLaunch L, hipStream_t stream) {
  const long rows = (long)L.B * L.per_seq;
  const int tiles = (L.V + kRowTile - 1) / kRowTile;
  L.group_octets = group_octets(L.V, few_rows(rows) ? kGroupsFew : kGroups);
  if (streams_apart(rows, L.V)) {
    const int waves = kStreamThreads / kWave;
    trace_before(stream, SV_KERNEL_FILTER_ROWS);
    filter_stream_kernel<LT><<<dim3((unsigned)rows, (unsigned)((tiles + waves - 1) / waves)),
                               kStreamThreads, 0, stream>>>(L);
    trace_after(stream, SV_KERNEL_FILTER_ROWS);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  trace_before(stream, SV_KERNEL_FILTER_ROWS);
  if (streams_apart(rows, L.V)) launch_rows<LT, 512, true, true>(L, stream);
  else if (few_rows(rows)) launch_rows<LT, 512, false, true>(L, stream);
  else launch_rows<LT, 256, false, false>(L, stream);
  trace_after(stream, SV_KERNEL_FILTER_ROWS);
  hipError_t e = hipGetLastError();
  // every token of a short row fits the list
  if (e == hipSuccess && !few_rows(rows) && L.V > kCand) {
    trace_before(stream, SV_KERNEL_FILTER_ROWS);
    const size_t lds = row_lds<kLeftThreads, true>(L);
    filter_left_kernel<LT><<<dim3((unsigned)std::min(rows, 512L)), kLeftThreads, lds, stream>>>(L);
    trace_after(stream, SV_KERNEL_FILTER_ROWS);
    e = hipGetLastError();
  }
  return e;
}

template <typename LT, bool QL>
hipError_t launch_verify_tail(const FilteredVerifyLaunch& L, hipStream_t stream) {
  trace_before(stream, SV_KERNEL_FILTERED_VERIFY);
  filtered_verify_kernel<LT, QL><<<dim3((unsigned)L.B), kVerifyThreads, 0, stream>>>(L);
  trace_after(stream, SV_KERNEL_FILTERED_VERIFY);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && L.V > kCand) {              // a shorter row always has a list
    const long tiles = (L.V + kRowTile - 1) / kRowTile;
    trace_before(stream, SV_KERNEL_FILTERED_VERIFY);
    residual_kernel<LT, QL><<<dim3((unsigned)std::min(L.B * tiles, 2048L)), kVerifyThreads, 0,
                              stream>>>(L);
    trace_after(stream, SV_KERNEL_FILTERED_VERIFY);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

size_t filter_workspace_bytes(long n_rows, int V) {
  return FilterWorkspace(n_rows, V, true).bytes;
}

hipError_t launch_filter_rows(const FilterLaunch& L0, hipStream_t stream) {
  FilterLaunch L = L0;
  char* ws = static_cast<char*>(L.workspace);
  const FilterWorkspace at((long)L.B * L.per_seq, L.V, L.verify);
  if (L.verify) {
    L.out_rows = reinterpret_cast<sv_filter_row*>(ws + at.rows);
    L.lists = reinterpret_cast<int32_t*>(ws + at.lists);
    L.pending = reinterpret_cast<int32_t*>(ws + at.pending);
  }
  L.list_counts = reinterpret_cast<int32_t*>(ws + at.counts);
  L.group_key = reinterpret_cast<uint16_t*>(ws + at.group_key);
  L.tile_max = reinterpret_cast<float*>(ws + at.tile_max);
  L.tile_sum = reinterpret_cast<double*>(ws + at.tile_sum);
  return L.bf16 ? launch_filter<uint16_t>(L, stream) : launch_filter<float>(L, stream);
}

hipError_t launch_filtered_verify(const FilteredVerifyLaunch& L0, hipStream_t stream) {
  FilteredVerifyLaunch L = L0;
  const FilterWorkspace at((long)L.B * (L.K + 1), L.V, true);
  char* ws = static_cast<char*>(L.workspace);
  L.rows = reinterpret_cast<sv_filter_row*>(ws + at.rows);
  L.list_counts = reinterpret_cast<int32_t*>(ws + at.counts);
  L.lists = reinterpret_cast<int32_t*>(ws + at.lists);
  L.pending = reinterpret_cast<int32_t*>(ws + at.pending);
  L.done = reinterpret_cast<int32_t*>(ws + at.done);
  L.tile_mass = reinterpret_cast<double*>(ws + at.tile_mass);
  FilterLaunch F{};
  F.logits = L.logits;
  F.row_stride = L.row_stride;
  F.n_rows = (long)L.B * (L.K + 1);
  F.temperatures = L.temperatures;
  F.temperature = 1.f;
  F.top_ks = L.top_ks;
  F.top_ps = L.top_ps;
  F.min_ps = L.min_ps;
  F.B = L.B;
  F.per_seq = L.K + 1;
  F.V = L.V;
  F.bf16 = L.bf16;
  F.workspace = L.workspace;
  F.verify = 1;
  F.device_error = L.device_error;
  hipError_t e = launch_filter_rows(F, stream);
  if (e != hipSuccess) return e;
  return L.bf16 ? (L.lq ? launch_verify_tail<uint16_t, true>(L, stream)
                        : launch_verify_tail<uint16_t, false>(L, stream))
                : (L.lq ? launch_verify_tail<float, true>(L, stream)
                        : launch_verify_tail<float, false>(L, stream));
}

}  // namespace sv
