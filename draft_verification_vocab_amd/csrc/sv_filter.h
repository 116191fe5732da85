// Filtered distributions (temperature, top-k, top-p, min-p) of logit rows, for
// the filtered sampler and the filtered verify (gfx950, wave64).
//
// A row z[V] at temperature T has weights w(x) = 2^((z(x) - m) c), m = max z,
// c = log2(e) / T.  Its tokens are ordered by logit, the largest first, equal
// logits by index; -inf and NaN logits are never kept.  Every filter keeps a
// prefix of that order, so a kept set is described by its last token alone:
// token x is kept iff z(x) > z_last, or z(x) = z_last and x <= last.
//
// Weights and their sums are fp64: top-p cuts between two neighbouring
// running sums, which differ by one token's share (1e-5 of the total and less
// in a flat row of 150k tokens) and which fp32 exponentials (1e-7 each) do not
// tell apart reliably.
#pragma once

#include <math.h>

#include "../../include/spec_verify.h"
#include "sv_device.h"
#include "sv_rowstats.h"

namespace sv {

// ---------------------------------------------------------------- keys
// Unsigned key of a logit that grows with it: -0 and +0 share one, NaN counts
// as -inf.  Every finite logit's key is greater than kKeyNegInf.
constexpr uint32_t kKeyNegInf = 0x007fffffu;
__device__ __forceinline__ float clean_logit(float z) {
  return z > -INFINITY ? z + 0.f : -INFINITY;
}
__device__ __forceinline__ uint32_t logit_key(float z) {       // z cleaned
  const uint32_t b = __float_as_uint(z);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float(k ^ ((uint32_t)((int32_t)~k >> 31) | 0x80000000u));
}

// ---------------------------------------------------------------- weights
// 2^x in fp64 for x <= 0: x = n + f, |f| <= 1/2, the exponential series of
// f ln 2 up to its 12th power (the 13th is below 2e-16).
__device__ __forceinline__ double exp2_f64(double x) {
  x = fmax(x, -1100.0);                     // 0 after the scaling; also -inf and NaN
  const double n = rint(x);
  const double f = x - n;
  double p = 2.5678435993488196e-11;        // (ln 2)^k / k!, k = 12 .. 0
  p = fma(p, f, 4.4455382718708101e-10);
  p = fma(p, f, 7.0549116208011209e-09);
  p = fma(p, f, 1.0178086009239696e-07);
  p = fma(p, f, 1.3215486790144305e-06);
  p = fma(p, f, 1.5252733804059838e-05);
  p = fma(p, f, 1.5403530393381606e-04);
  p = fma(p, f, 1.3333558146428441e-03);
  p = fma(p, f, 9.6181291076284769e-03);
  p = fma(p, f, 5.5504108664821576e-02);
  p = fma(p, f, 2.4022650695910069e-01);
  p = fma(p, f, 6.9314718055994529e-01);
  p = fma(p, f, 1.0);
  return ldexp(p, (int)n);
}

// 2^x for -1000 <= x <= 0 with a table: x = k/64 + r with |r| <= 1/128, 2^(k/64)
// from the table and 2^r by the exponential series up to r^5, exact to 1e-15.
// Adding 1.5 * 2^46 rounds x to a multiple of 1/64 and leaves k in the sum's low
// word.  The table is 64 doubles, two for each pair of LDS banks, so that lanes
// reading different entries hardly wait for each other.  Entry j is kept less
// j << 46: adding k << 14 to its high word puts in the whole part of k/64.
constexpr int kExpTable = 64;
struct ExpTable {
  unsigned long long v[kExpTable];
  constexpr ExpTable() : v() {
    for (int i = 0; i < kExpTable; ++i) {
      // 2^(i/64) as the square of the exponential series of half its logarithm
      const double y = 0.69314718055994530942 * i / (2.0 * kExpTable);
      double term = 1.0, sum = 0.0;
      for (int k = 24; k >= 0; --k) {               // smallest terms first
        term = 1.0;
        for (int j = 1; j <= k; ++j) term *= y / j;
        sum += term;
      }
      v[i] = __builtin_bit_cast(unsigned long long, sum * sum) - ((unsigned long long)i << 46);
    }
  }
};
__device__ constexpr ExpTable kExp2Table;
typedef unsigned long long ExpEntry;
__device__ __forceinline__ void fill_exp_table(ExpEntry* table) {
  if (threadIdx.x < kExpTable) table[threadIdx.x] = kExp2Table.v[threadIdx.x];
}
constexpr double kExpRound = 0x1.8p46;
// 2^(k/64), k the low word of kExpRound + k/64.
__device__ __forceinline__ double table_entry(double y, const ExpEntry* table) {
  const uint32_t k = (uint32_t)__double_as_longlong(y);
  const ExpEntry t = table[k % kExpTable];
  return __longlong_as_double((ExpEntry)((uint32_t)(t >> 32) + (k << 14)) << 32 | (uint32_t)t);
}
__device__ __forceinline__ double exp2_table(double x, const ExpEntry* table) {
  const double y = x + kExpRound, r = x - (y - kExpRound);
  const double T = table_entry(y, table);
  const double q = fma(r, fma(r, fma(r, fma(r, 1.3333558146428443e-03, 9.6181291076284770e-03),
                                     5.5504108664821580e-02), 2.4022650695910071e-01),
                       6.9314718055994531e-01);
  return fma(T, r * q, T);
}
// 2^r for the long sums: the series up to r^4 with r^4 replaced by the polynomial
// h^2 r^2 - h^4/8 that comes nearest to it on |r| <= h = 1/128: exact to 5e-12.
struct TwoTo {
  // The coefficients are taken up where the object stands: hoisted out of the
  // caller's outer loops they would take the registers that are short there.
  double c[4] = {0.99999999999552125, 0.69314718055994529, 0.24022709400311362,
                 0.055504108664821576};
  __device__ __forceinline__ TwoTo() {
#pragma unroll
    for (int i = 0; i < 4; ++i) asm volatile("" : "+s"(c[i]));
  }
  __device__ __forceinline__ double operator()(double r) const {
    return fma(r, fma(r, fma(r, c[3], c[2]), c[1]), c[0]);
  }
};

// The weight of logit z in a row of maximum m: 1 at the maximum (also where
// that is +inf), 0 at -inf.
__device__ __forceinline__ double weight(float z, float m, double c) {
  if (z == m) return 1.0;
  return z > -INFINITY ? exp2_f64(((double)z - (double)m) * c) : 0.0;
}

// The same with a table, to 1e-14 (0 below 2^-1000).
__device__ __forceinline__ double weight(float z, float m, double c, const ExpEntry* table) {
  if (z == m) return 1.0;
  const double x = ((double)z - (double)m) * c;
  return z > -INFINITY && x > -1000.0 ? exp2_table(x, table) : 0.0;
}

// Whether a filter row keeps token x of logit z (cleaned).
__device__ __forceinline__ bool row_keeps(const sv_filter_row& f, float z, long x) {
  return z > f.min_kept || (z == f.min_kept && x <= (long)f.last);
}
// The probability a filter row gives token x of logit z.
__device__ __forceinline__ double row_prob(const sv_filter_row& f, float z, long x) {
  z = clean_logit(z);
  return row_keeps(f, z, x) ? weight(z, f.max, f.scale) * f.inv_sum : 0.0;
}

// ---------------------------------------------------------------- settings
struct FilterSettings {
  double c;      // log2(e) / T; 0: greedy
  int k;         // 1 .. V (V: off)
  float p;       // >= 1: off
  float mp;      // <= 0: off
  bool off;      // no filter at all
};

// The settings of sequence b.  Bad values are flagged and switched off (a bad
// temperature is greedy, as everywhere else).
__device__ __forceinline__ FilterSettings filter_settings(const float* temperatures,
                                                          float temperature, const int32_t* top_ks,
                                                          const float* top_ps, const float* min_ps,
                                                          int b, int V, int& errors) {
  FilterSettings s;
  bool bad;
  const float T = temperatures ? temperatures[b] : temperature;
  const float c32 = seq_scale(T, bad);
  if (bad) errors |= SV_DEVERR_TEMPERATURE;
  s.c = c32 == 0.f ? 0.0 : 1.4426950408889634 / (double)T;
  int k = top_ks ? top_ks[b] : 0;
  float p = top_ps ? top_ps[b] : 1.f;
  float mp = min_ps ? min_ps[b] : 0.f;
  if (k < 0) { errors |= SV_DEVERR_FILTER; k = 0; }
  if (!(p > 0.f && p <= 1.f)) { errors |= SV_DEVERR_FILTER; p = 1.f; }
  if (!(mp >= 0.f && mp <= 1.f)) { errors |= SV_DEVERR_FILTER; mp = 0.f; }
  if (c32 == 0.f) { k = 1; p = 1.f; mp = 0.f; }
  s.k = k == 0 || k > V ? V : k;
  s.p = p;
  s.mp = mp;
  s.off = s.k == V && s.p >= 1.0 && s.mp <= 0.0 && c32 != 0.f;
  return s;
}

// ---------------------------------------------------------------- workgroup reductions
// A value that all lanes hold, in scalar registers.
template <typename T>
__device__ __forceinline__ T uniform(T x) {
  static_assert(sizeof(T) == 4 || sizeof(T) == 8, "one or two registers");
  int w[sizeof(T) / 4];
  __builtin_memcpy(w, &x, sizeof(T));
#pragma unroll
  for (unsigned i = 0; i < sizeof(T) / 4; ++i) w[i] = __builtin_amdgcn_readfirstlane(w[i]);
  __builtin_memcpy(&x, w, sizeof(T));
  return x;
}

// x of the lane that a DPP control names, `old` in lanes without one.
template <int CTRL, int ROWS = 0xf, typename T>
__device__ __forceinline__ T dpp(T x, T old) {
  static_assert(sizeof(T) == 4 || sizeof(T) == 8, "one or two registers");
  int w[sizeof(T) / 4], o[sizeof(T) / 4];
  __builtin_memcpy(w, &x, sizeof(T));
  __builtin_memcpy(o, &old, sizeof(T));
#pragma unroll
  for (unsigned i = 0; i < sizeof(T) / 4; ++i)
    w[i] = __builtin_amdgcn_update_dpp(o[i], w[i], CTRL, ROWS, 0xf, false);
  __builtin_memcpy(&x, w, sizeof(T));
  return x;
}
template <typename T>
__device__ __forceinline__ T of_lane(T x, int lane) {
  int w[sizeof(T) / 4];
  __builtin_memcpy(w, &x, sizeof(T));
#pragma unroll
  for (unsigned i = 0; i < sizeof(T) / 4; ++i) w[i] = __builtin_amdgcn_readlane(w[i], lane);
  __builtin_memcpy(&x, w, sizeof(T));
  return x;
}
// Over a wave: rotations within its rows of 16 lanes, then the four rows'
// results by readlane.  A step is a few instructions, where a shuffle through
// LDS takes over 100 cycles.  The result is uniform.
template <typename T, typename OP>
__device__ __forceinline__ T wave_reduce(T x, OP op) {
  x = op(x, dpp<0x128>(x, x));          // row_ror 8, 4, 2, 1
  x = op(x, dpp<0x124>(x, x));
  x = op(x, dpp<0x122>(x, x));
  x = op(x, dpp<0x121>(x, x));
  return op(op(of_lane(x, 0), of_lane(x, 16)), op(of_lane(x, 32), of_lane(x, 48)));
}
// Inclusive running totals over a wave's lanes: shifts within the rows, then
// the last lanes of row 0 and 2 to the next rows, and of row 1 to the upper half.
template <typename T>
__device__ __forceinline__ T wave_prefix(T x) {
  x += dpp<0x111>(x, T(0));             // row_shr 1, 2, 4, 8
  x += dpp<0x112>(x, T(0));
  x += dpp<0x114>(x, T(0));
  x += dpp<0x118>(x, T(0));
  x += dpp<0x142, 0xa>(x, T(0));        // row_bcast 15
  x += dpp<0x143, 0xc>(x, T(0));        // row_bcast 31
  return x;
}

// Over the workgroup; sm holds one entry per wave.
template <int THREADS, typename T, typename OP>
__device__ __forceinline__ T block_reduce(T x, T* sm, OP op) {
  x = wave_reduce(x, op);
  __syncthreads();                      // sm may still be read from before
  if (lane_id() == 0) sm[threadIdx.x / kWave] = x;
  __syncthreads();
  x = sm[0];
#pragma unroll
  for (int i = 1; i < THREADS / kWave; ++i) x = op(x, sm[i]);
  return uniform(x);
}
struct OpAdd { template <typename T> __device__ T operator()(T a, T b) const { return a + b; } };
struct OpMax { template <typename T> __device__ T operator()(T a, T b) const { return a > b ? a : b; } };
struct OpMin { template <typename T> __device__ T operator()(T a, T b) const { return a < b ? a : b; } };

// ---------------------------------------------------------------- loads
// Eight consecutive logits from element e on, whatever the row's alignment: a
// row of odd length, or one inside a padded buffer, starts at any multiple of
// its element size, and gfx950 loads 16 bytes from any such address.
struct __attribute__((packed, aligned(2))) OctBf16 { u32x4 w; };
struct __attribute__((packed, aligned(4))) OctF32 { u32x4 a, b; };
__device__ __forceinline__ void raw8(const uint16_t* p, Raw<uint16_t>& r) {
  r.w = reinterpret_cast<const OctBf16*>(p)->w;
}
__device__ __forceinline__ void raw8(const float* p, Raw<float>& r) {
  const OctF32 v = *reinterpret_cast<const OctF32*>(p);
  r.a = v.a;
  r.b = v.b;
}
template <typename LT>
__device__ __forceinline__ void load8(const LT* p, float z[8]) {
  Raw<LT> r;
  raw8(p, r);
  unpack(r, z);
}
// Octets that reach past the row's end: the rest reads as -inf.
__device__ __forceinline__ void raw8_end(const uint16_t* row, int e, int V, Raw<uint16_t>& r) {
  uint32_t x[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    x[j] = (e + 2 * j < V ? row[e + 2 * j] : 0xff80u) |
           ((e + 2 * j + 1 < V ? row[e + 2 * j + 1] : 0xff80u) << 16);
  r.w = u32x4{x[0], x[1], x[2], x[3]};
}
__device__ __forceinline__ void raw8_end(const float* row, int e, int V, Raw<float>& r) {
  uint32_t x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = e + j < V ? __float_as_uint(row[e + j]) : 0xff800000u;
  r.a = u32x4{x[0], x[1], x[2], x[3]};
  r.b = u32x4{x[4], x[5], x[6], x[7]};
}
// An empty statement that claims to change a loaded octet, so that the
// compiler unpacks it again instead of holding the unpacked values.
__device__ __forceinline__ void keep_raw(Raw<uint16_t>& r) { asm volatile("" : "+v"(r.w)); }
__device__ __forceinline__ void keep_raw(Raw<float>& r) { asm volatile("" : "+v"(r.a), "+v"(r.b)); }

// Every element of a row by the whole workgroup: f(z cleaned, index).
template <typename LT, int THREADS, typename F>
__device__ __forceinline__ void each_logit(const LT* row, int V, F f) {
  const int full = V / 8;
#pragma unroll 1
  for (int o = threadIdx.x; o < full; o += THREADS) {
    float z[8];
    load8(row + o * 8, z);
#pragma unroll
    for (int j = 0; j < 8; ++j) f(clean_logit(z[j]), o * 8 + j);
  }
  const int e = full * 8 + threadIdx.x;
  if (e < V) f(clean_logit(logit_at(row, e)), e);
}

}  // namespace sv
