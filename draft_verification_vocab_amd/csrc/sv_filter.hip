// Filtered sampling and verification for gfx950: the token distribution of a
// logit row under temperature, top-k, top-p and min-p, drawn from (the
// sampler) or used as the target of rejection sampling (the verify).  The
// definitions are in sv_filter.h and include/spec_verify.h.
//
//   filter_rows_kernel   one workgroup per row: the row's kept set as a
//                        filter row (its last token, maximum and 1 / sum), and
//                        for the sampler the drawn token and the dense q;
//   filtered_verify_kernel  one workgroup per sequence: the accept scan from
//                        the filter rows, then the residual draw on the row
//                        of the first rejection.
#include "sv_filter.h"
#include "sv_internal.h"

namespace sv {

namespace {

constexpr int kFilterThreads = 512;
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
__device__ int block_draw(int V, float u, DrawShared& sh, F mass) {
  const int w = threadIdx.x / kWave, l = lane_id();
  const int tiles = (V + kDrawTile - 1) / kDrawTile;
  __syncthreads();
  for (int t = w; t < tiles; t += THREADS / kWave) {
    double s = 0.0;
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
__device__ int nth_tie(const LT* row, int V, uint32_t key, int t, FilterShared<THREADS>& sh) {
  const int tiles = (V + kDrawTile - 1) / kDrawTile;
  __syncthreads();
  for (int i = threadIdx.x; i < tiles; i += THREADS) sh.cnt[i] = 0;
  __syncthreads();
  each_logit<LT, THREADS>(row, V, [&](float z, int e) {
    if (logit_key(z) == key) atomicAdd(&sh.cnt[e / kDrawTile], 1u);
  });
  __syncthreads();
  if (threadIdx.x < kWave) {
    const int l = lane_id();
    int tile = 0, before = 0;
    for (; tile < tiles - 1; ++tile) {
      const int n = (int)sh.cnt[tile];
      if (before + n >= t) break;
      before += n;
    }
    int found = V - 1;
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
    if (l == 0) sh.bin = found;
  }
  __syncthreads();
  const int r = sh.bin;
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
__device__ uint32_t radix_cut(const LT* row, int V, const Cut& in, float m, double c,
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
__device__ sv_filter_row filter_row(const LT* row, int V, const FilterSettings& s,
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
    cut = Cut{key, keep >= ties ? V : nth_tie<LT, THREADS>(row, V, key, keep, sh)};
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
      cut = Cut{key, keep >= ties ? V : nth_tie<LT, THREADS>(row, V, key, keep, sh)};
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

// ---------------------------------------------------------------- kernels
template <typename LT>
__global__ __launch_bounds__(kFilterThreads) void filter_rows_kernel(FilterLaunch A) {
  __shared__ union {
    FilterShared<kFilterThreads> filter;
    DrawShared draw;
  } sh;
  const long r = blockIdx.x;
  const int b = (int)(r / A.per_seq);
  const int V = A.V;
  int errors = 0;
  const FilterSettings s = filter_settings(A.temperatures, A.temperature, A.top_ks, A.top_ps,
                                           A.min_ps, b, V, errors);
  const long ri = A.row_index ? (long)A.row_index[r] : r;
  const bool there = ri >= 0 && ri < A.n_rows;
  sv_filter_row f{0.0, 0.0, -INFINITY, INFINITY, -1, 0};
  const LT* row = static_cast<const LT*>(A.logits) + (there ? ri : 0) * A.row_stride;
  if (there) f = filter_row<LT, kFilterThreads>(row, V, s, sh.filter);
  if (!there) errors |= SV_DEVERR_ROW_INDEX;
  else if (f.n_kept == 0) errors |= SV_DEVERR_EMPTY_ROW;
  if (threadIdx.x == 0) {
    if (errors) flag_error(A.device_error, errors);
    if (A.out_rows) A.out_rows[r] = f;
  }
  if (A.out_tokens) {
    int token = there ? 0 : -1;
    if (f.n_kept > 0) {
      token = s.c == 0.0 ? f.last
                         : block_draw<kFilterThreads>(V, A.uniforms[r], sh.draw, [&](int e) {
                             const float z = clean_logit(logit_at(row, e));
                             return row_keeps(f, z, e) ? weight(z, f.max, f.scale) : 0.0;
                           });
    }
    if (threadIdx.x == 0) A.out_tokens[r] = token;
  }
  if (A.out_probs) {
    float* q = A.out_probs + r * V;
    for (int e = threadIdx.x; e < V; e += kFilterThreads)
      __builtin_nontemporal_store(f.n_kept ? (float)row_prob(f, logit_at(row, e), e) : 0.f, q + e);
  }
}

template <typename LT, bool QL>
__global__ __launch_bounds__(kVerifyThreads) void filtered_verify_kernel(FilteredVerifyLaunch A) {
  __shared__ DrawShared draw;
  __shared__ int sh_a;
  const int b = blockIdx.x, K = A.K, V = A.V;
  const int l = lane_id();
  const long row0 = (long)b * (K + 1);
  const LT* z0 = static_cast<const LT*>(A.logits) + row0 * A.row_stride;
  // q of draft k at token x
  const auto q_at = [&](int k, long dr, const sv_filter_row& f, int x) -> double {
    if constexpr (QL) {
      if (dr < 0) return 0.0;
      return row_prob(f, logit_at(static_cast<const LT*>(A.dlogits) + dr * A.d_stride, x), x);
    } else {
      return (double)A.draft_probs[((long)b * K + k) * V + x];
    }
  };
  const auto drafter_row = [&](int k) -> long {
    if constexpr (!QL) return 0;
    const long i = (long)b * K + k;
    const long dr = A.drows ? (long)A.drows[i] : i;
    return dr >= 0 && dr < A.d_rows ? dr : -1;
  };
  int errors = 0;
  if (threadIdx.x < kWave) {
    bool accepted = false;
    if (l < K) {
      const sv_filter_row f = A.rows[row0 + l];
      const bool greedy = f.scale == 0.0;
      const int x = A.draft_tokens[(long)b * K + l];
      double p = 0.0;
      if (x >= 0 && x < V) {
        p = row_prob(f, logit_at(z0 + l * A.row_stride, x), x);
        if (greedy) {
          accepted = x == f.last;
        } else if (p > 0.0) {
          const long dr = drafter_row(l);
          if (dr < 0) errors |= SV_DEVERR_ROW_INDEX;
          sv_filter_row fq{};
          if constexpr (QL) fq = A.ddesc[(long)b * K + l];
          accepted = (double)A.uniforms[row0 + l] * q_at(l, dr, fq, x) < p;
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
  int token = 0;
  if (f.n_kept == 0) {
    token = 0;
  } else if (f.scale == 0.0) {
    token = f.last;
  } else {
    const float u = A.uniforms[row0 + K];
    token = -1;
    if (a < K) {
      const long dr = drafter_row(a);
      sv_filter_row fq{};
      if constexpr (QL) fq = A.ddesc[(long)b * K + a];
      token = block_draw<kVerifyThreads>(V, u, draw, [&](int e) {
        const double p = row_prob(f, logit_at(za, e), e);
        return p > 0.0 ? fmax(0.0, p - q_at(a, dr, fq, e)) : 0.0;
      });
    }
    if (token < 0)
      token = block_draw<kVerifyThreads>(V, u, draw,
                                         [&](int e) { return row_prob(f, logit_at(za, e), e); });
  }
  if (threadIdx.x == 0) A.out_tokens[row0 + a] = token;
}

}  // namespace

size_t filter_workspace_bytes(long n_rows, int V) {
  (void)V;
  return (size_t)n_rows * sizeof(sv_filter_row);
}

hipError_t launch_filter_rows(const FilterLaunch& L, hipStream_t stream) {
  const dim3 grid((unsigned)((long)L.B * L.per_seq));
  trace_before(stream, SV_KERNEL_FILTER_ROWS);
  if (L.bf16) filter_rows_kernel<uint16_t><<<grid, kFilterThreads, 0, stream>>>(L);
  else filter_rows_kernel<float><<<grid, kFilterThreads, 0, stream>>>(L);
  trace_after(stream, SV_KERNEL_FILTER_ROWS);
  return hipGetLastError();
}

hipError_t launch_filtered_verify(const FilteredVerifyLaunch& L0, hipStream_t stream) {
  FilteredVerifyLaunch L = L0;
  L.rows = static_cast<sv_filter_row*>(L.workspace);
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
  F.out_rows = L.rows;
  F.device_error = L.device_error;
  hipError_t e = launch_filter_rows(F, stream);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)L.B);
  trace_before(stream, SV_KERNEL_FILTERED_VERIFY);
  if (L.bf16) {
    if (L.lq) filtered_verify_kernel<uint16_t, true><<<grid, kVerifyThreads, 0, stream>>>(L);
    else filtered_verify_kernel<uint16_t, false><<<grid, kVerifyThreads, 0, stream>>>(L);
  } else {
    if (L.lq) filtered_verify_kernel<float, true><<<grid, kVerifyThreads, 0, stream>>>(L);
    else filtered_verify_kernel<float, false><<<grid, kVerifyThreads, 0, stream>>>(L);
  }
  trace_after(stream, SV_KERNEL_FILTERED_VERIFY);
  return hipGetLastError();
}

}  // namespace sv
