// Appending a drafter batch's keys and values to a paged cache for gfx950,
// with the rotary position embedding of keys (and queries) applied on the way
// (peagle_append_kv in include/spec_verify.h).
//
// A copy with three flops an element, bounded by HBM: 1024 drafts of 14 rows (32
// query heads, 4 key heads of 128, bf16 into e4m3; 279 MB) take 53 us, 5.2 TB/s, the
// rate of a plain copy; one row takes 3.3 us.  Every workgroup takes a
// few rows: it first computes the cosine and sine of each row's rot / 2 angles
// once (they are shared by all heads) into LDS, then its threads stream the
// rows' query, key and value heads, up to 16 bytes of the source type per load.
//
// Angles: position * inv_freq is exact in fp64 for positions below 2^29 (29 +
// 24 bits), so the angle is reduced to a fraction of a turn in fp64 and only
// the reduced angle goes through fp32 sine and cosine; a far position is as
// exact as a near one.
#include <hip/hip_bf16.h>

#include <algorithm>

#include "sv_device.h"
#include "sv_internal.h"

namespace sv {

namespace {

constexpr int kAppendThreads = 256;
// (cos, sin) pairs per workgroup: 16 KB, so that eight workgroups fit a CU (with
// 32 KB five do: 66 against 56 us for 1024 drafts of 14 rows of 32 heads, keys and values into
// e4m3)
constexpr int kAppendLds = 2048;
constexpr int kAppendRows = 16;       // most rows of a workgroup

// n / d for n * d < 2^32 with magic = ceil(2^32 / d).
__device__ __forceinline__ unsigned div_magic(unsigned n, unsigned magic, unsigned d) {
  return d == 1 ? n : __umulhi(n, magic);
}

template <typename T> __device__ __forceinline__ float to_f32(T x);
template <> __device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ float to_f32<__hip_bfloat16>(__hip_bfloat16 x) {
  return __bfloat162float(x);
}
template <> __device__ __forceinline__ float to_f32<_Float16>(_Float16 x) { return (float)x; }
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __hip_bfloat16 from_f32<__hip_bfloat16>(float x) {
  return __float2bfloat16(x);
}
template <> __device__ __forceinline__ _Float16 from_f32<_Float16>(float x) { return (_Float16)x; }

// N elements, aligned as one element: gfx950 loads and stores up to 16 bytes
// at any such address, so views into a packed projection and odd head sizes
// take the same path.
template <typename T, int N> struct __attribute__((packed, aligned(sizeof(T)))) Vec { T v[N]; };

template <typename T, int N>
__device__ __forceinline__ void load_n(const T* p, float (&x)[N]) {
  const Vec<T, N> r = *reinterpret_cast<const Vec<T, N>*>(p);
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = to_f32<T>(r.v[i]);
}
template <typename T, int N>
__device__ __forceinline__ void store_n(T* p, const float (&x)[N]) {
  Vec<T, N> r;
#pragma unroll
  for (int i = 0; i < N; ++i) r.v[i] = from_f32<T>(x[i]);
  *reinterpret_cast<Vec<T, N>*>(p) = r;
}

// x / scale as e4m3 bits, to nearest, limited to the largest finite value
// (448); NaN stays NaN.
__device__ __forceinline__ float e4m3_range(float x, float scale) {
  x = x / scale;
  return x != x ? x : fminf(fmaxf(x, -448.f), 448.f);
}
template <int N>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float (&x)[N], float scale) {
  Vec<uint8_t, N> r;
  if constexpr (N == 1) {
    const float a = e4m3_range(x[0], scale);
    r.v[0] = (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(a, a, 0, false) & 255);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const int w = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_range(x[i], scale),
                                                    e4m3_range(x[i + 1], scale), 0, false);
      r.v[i] = (uint8_t)(w & 255);
      r.v[i + 1] = (uint8_t)((w >> 8) & 255);
    }
  }
  *reinterpret_cast<Vec<uint8_t, N>*>(p) = r;
}

// N elements to a cache: the source type, or e4m3.
template <typename T, bool FP8, int N>
__device__ __forceinline__ void store_cache(void* cache, long at, const float (&x)[N], float scale) {
  if constexpr (FP8) store_e4m3<N>(static_cast<uint8_t*>(cache) + at, x, scale);
  else store_n<T, N>(static_cast<T*>(cache) + at, x);
}

// The work of a row is its heads' items: queries, keys, then values.  An item
// is one N-vector, except in the rotated part of a head whose pairs are rot / 2
// apart, where it is the two N-vectors of N pairs (and single pairs of
// neighbours when N = 1).
template <typename T, bool FP8, bool INTER, int N>
__global__ __launch_bounds__(kAppendThreads) void append_kv_kernel(AppendLaunch A) {
  __shared__ float2 turn[kAppendLds];
  __shared__ long slots[kAppendRows];
  const long r0 = (long)blockIdx.x * A.rows_per_block;
  const int nr = (int)min((long)A.rows_per_block, A.R - r0);
  const int half = A.rot / 2;
  for (int i = threadIdx.x; i < nr * half; i += kAppendThreads) {
    const int r = i / half, j = i - r * half;
    const double t = (double)A.positions[r0 + r] * (double)A.inv_freq[j] * 0.15915494309189535;
    float s, c;
    sincospif((float)(2.0 * (t - rint(t))), &s, &c);
    turn[i] = float2{c * A.rotary_scale, s * A.rotary_scale};
  }
  if ((int)threadIdx.x < nr) {
    const long slot = A.slots[r0 + threadIdx.x];
    const bool in = slot >= 0 && slot < A.num_slots;
    if (!in && slot != SV_PADDING_SLOT_ID) flag_error(A.device_error, SV_DEVERR_SLOT);
    slots[threadIdx.x] = in ? slot : -1;
  }
  __syncthreads();

  const int D = A.head_dim, items = A.items, vitems = D / N;
  const int turned = half / N;                         // pair items of a head
  const int q_items = A.q_heads * items, k_items = A.kv_heads * items;
  const int row_items = q_items + k_items + A.kv_heads * vitems;
  for (int i = threadIdx.x; i < nr * row_items; i += kAppendThreads) {
    const int r = nr == 1 ? 0 : (int)div_magic(i, A.row_magic, row_items);
    int w = i - r * row_items;
    const long row = r0 + r, slot = slots[r];
    long at = 0;                                       // the slot's place in the caches
    if (w >= q_items) {
      if (slot < 0) continue;
      const long blk = slot / A.block_size;
      at = blk * A.block_stride + (slot - blk * A.block_size) * A.slot_stride;
    }
    if (w >= q_items + k_items) {                      // values: copied
      w -= q_items + k_items;
      const int h = (int)div_magic(w, A.vitem_magic, vitems), e = (w - h * vitems) * N;
      float x[N];
      load_n<T, N>(static_cast<const T*>(A.value) + row * A.v_stride + h * D + e, x);
      store_cache<T, FP8, N>(A.value_cache, at + h * A.head_stride + e, x,
                             FP8 && A.v_scales ? A.v_scales[h] : 1.f);
      continue;
    }
    const bool is_q = w < q_items;
    if (!is_q) w -= q_items;
    const int h = (int)div_magic(w, A.item_magic, items), j = w - h * items;
    const T* src = is_q ? static_cast<const T*>(A.query) + row * A.q_stride + h * D
                        : static_cast<const T*>(A.key) + row * A.k_stride + h * D;
    const long dst = is_q ? row * A.out_q_stride + h * D : at + h * A.head_stride;
    const float scale = FP8 && !is_q && A.k_scales ? A.k_scales[h] : 1.f;
    const auto put = [&](int e, const float (&x)[N]) {
      if (is_q) store_n<T, N>(static_cast<T*>(A.out_query) + dst + e, x);
      else store_cache<T, FP8, N>(A.key_cache, dst + e, x, scale);
    };
    if (INTER && N > 1) {                              // neighbours: within one vector
      const int e = j * N;
      float x[N];
      load_n<T, N>(src + e, x);
      if (e < A.rot) {
        const float2* cs = turn + r * half + e / 2;
#pragma unroll
        for (int i = 0; i + 1 < N; i += 2) {
          const float2 t = cs[i / 2];
          const float x0 = x[i], x1 = x[i + 1];
          x[i] = x0 * t.x - x1 * t.y;
          x[i + 1] = x1 * t.x + x0 * t.y;
        }
      }
      put(e, x);
    } else if (j < turned) {
      const float2* cs = turn + r * half + j * N;      // pairs j N .. j N + N - 1
      const int e0 = INTER ? 2 * j : j * N, e1 = INTER ? e0 + 1 : half + j * N;
      float x0[N], x1[N];
      load_n<T, N>(src + e0, x0);
      load_n<T, N>(src + e1, x1);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float2 t = cs[i];
        const float a = x0[i], b = x1[i];
        x0[i] = a * t.x - b * t.y;
        x1[i] = b * t.x + a * t.y;
      }
      put(e0, x0);
      put(e1, x1);
    } else {                                           // past the rotated part: copied
      const int e = A.rot + (j - turned) * N;
      float x[N];
      load_n<T, N>(src + e, x);
      put(e, x);
    }
  }
}

template <typename T, bool FP8, int N>
void launch_append_n(const AppendLaunch& L, dim3 grid, hipStream_t stream) {
  if (L.interleaved) append_kv_kernel<T, FP8, true, N><<<grid, kAppendThreads, 0, stream>>>(L);
  else append_kv_kernel<T, FP8, false, N><<<grid, kAppendThreads, 0, stream>>>(L);
}

template <typename T, int MAXN>
void launch_append_t(const AppendLaunch& L, int N, dim3 grid, hipStream_t stream) {
  switch (L.fp8 ? -N : N) {
    case 8: launch_append_n<T, false, MAXN>(L, grid, stream); break;
    case 4: launch_append_n<T, false, 4>(L, grid, stream); break;
    case 2: launch_append_n<T, false, 2>(L, grid, stream); break;
    case 1: launch_append_n<T, false, 1>(L, grid, stream); break;
    case -8: launch_append_n<T, true, MAXN>(L, grid, stream); break;
    case -4: launch_append_n<T, true, 4>(L, grid, stream); break;
    case -2: launch_append_n<T, true, 2>(L, grid, stream); break;
    default: launch_append_n<T, true, 1>(L, grid, stream); break;
  }
}

unsigned magic_of(unsigned d) { return (unsigned)(((1ull << 32) + d - 1) / d); }

}  // namespace

hipError_t launch_append(const AppendLaunch& L0, hipStream_t stream) {
  AppendLaunch L = L0;
  // the widest vector, up to 16 bytes, that divides the head and its rotated parts
  int N = L.dtype == SV_F32 ? 4 : 8;
  while (N > 1 && (L.head_dim % N || (L.interleaved ? L.rot : L.rot / 2) % N ||
                   (L.head_dim - L.rot) % N))
    N /= 2;
  L.items = L.interleaved && N > 1 ? L.head_dim / N : L.rot / 2 / N + (L.head_dim - L.rot) / N;
  const long row_items =
      (long)(L.q_heads + L.kv_heads) * L.items + (long)L.kv_heads * (L.head_dim / N);
  // rows per workgroup: about four items a thread, while the grid still covers
  // the chip twice.  More than one row only below 1024 items a row, so that
  // the division of an item number by them stays exact.
  long rows = row_items < 4 * kAppendThreads ? 4 * kAppendThreads / row_items : 1;
  rows = std::min(rows, std::max(1L, L.R / 512));
  rows = std::max(1L, std::min(rows, (long)kAppendRows));
  if (L.rot > 0) rows = std::min(rows, (long)(kAppendLds / (L.rot / 2)));
  L.rows_per_block = (int)rows;
  L.row_magic = magic_of((unsigned)row_items);
  L.item_magic = magic_of((unsigned)std::max(1, L.items));
  L.vitem_magic = magic_of((unsigned)(L.head_dim / N));
  const dim3 grid((unsigned)((L.R + rows - 1) / rows));
  trace_before(stream, SV_KERNEL_APPEND_KV);
  if (L.dtype == SV_F32) launch_append_t<float, 4>(L, N, grid, stream);
  else if (L.dtype == SV_BF16) launch_append_t<__hip_bfloat16, 8>(L, N, grid, stream);
  else launch_append_t<_Float16, 8>(L, N, grid, stream);
  const hipError_t err = hipGetLastError();
  trace_after(stream, SV_KERNEL_APPEND_KV);
  return err;
}

}  // namespace sv
