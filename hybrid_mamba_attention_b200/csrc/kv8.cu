// Writing tokens into the 8-bit paged KV cache and reading them back (hspec_kv8_write,
// hspec_kv8_read).
//
// Work unit: one page that a request's token range touches, of one kv head, K or V -- one
// warp.  The touched pages of all requests are numbered without a pass over the lengths:
// request c owns the slots [cu[c] / page + 2c, cu[c+1] / page + 2(c + 1)), at least
// floor(n / page) + 2 of them for its n tokens, and n tokens touch at most
// floor((n - 1) / page) + 2 pages, so the slots suffice wherever the range starts; a warp
// finds its request by a 32-way search over c and leaves when its slot has no page.  The
// host knows the number of slots from T and C alone: one launch, no workspace.
//
// Both directions are bound by HBM: the new rows once (2 or 4 bytes an element) and the
// codes once (1 byte).  A unit of up to 32 lanes x 4 chunks of 16 elements (a page of 16
// tokens of 128 dims) stays in registers between the search for its largest magnitude and the
// quantisation; a larger one is read a second time, out of L2.  At 8 kv heads of 128 dims,
// bf16, pages of 16: 16 prefixes of 512 .. 8192 tokens are read in 78 us (5.5 TB/s of the 6.56
// that a copy reaches), 8 prompts of 512 .. 16384 written in 88 us (4.7 TB/s: one warp waits
// for its page's rows, finds their maximum and only then stores), a token of each of 128
// requests in 7.2 us, a launch and four loads one after the other; fp32: 154, 129 and 7.8 us.
#include <type_traits>

#include "../../include/hspec.h"
#include "common.cuh"
#include "kernels.cuh"
#include "kv8.cuh"

namespace hspec {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kHeld = 4;  // chunks per lane that stay in registers

// The page of slot u: tokens [t0, t0 + n) of the request, slots [slot0, slot0 + n) of
// page `pg`, rows from `row` on.  n = 0: nothing (pg < 0 with n > 0: a bad page id).
struct Unit {
  int n, slot0, pg;
  long row;
};

__device__ __forceinline__ Unit find_unit(const Kv8MoveArgs& a, int u) {
  const int page = a.kv.page_size, lane = threadIdx.x & 31;
  Unit r = {0, 0, -1, 0};
  // the last request whose slots start at or before u (with offsets that fall, the starts are not
  // in order and the search may miss it: the slot's page is then left alone)
  int c = 0;
  for (int n = a.C; n > 1;) {
    const int step = (n + 31) / 32, i = lane * step;
    const bool at = i < n && a.cu[c + i] / page + 2 * (c + i) <= u;
    const int hits = __popc(__ballot_sync(0xffffffffu, at));
    if (hits == 0) return r;
    c += (hits - 1) * step;
    n = min(step, n - (hits - 1) * step);
  }
  if (c >= a.C) return r;  // (only with offsets out of order)
  const int b = a.cu[c], e = a.cu[c + 1];
  const int f = a.first ? a.first[c] : 0;
  // a range that is out of order, outside the rows or past the table is left alone
  if (b < 0 || e < b || e > a.T || f < 0 || (long)f + (e - b) > (long)a.kv.max_pages * page) return r;
  const int i = u - (b / page + 2 * c);
  const int p0 = f / page, p = p0 + i;
  if (i < 0 || b == e || p > (f + (e - b) - 1) / page) return r;
  const int t0 = max(f, p * page), t1 = min(f + (e - b), (p + 1) * page);
  r.n = t1 - t0;
  r.slot0 = t0 - p * page;
  r.row = b + (t0 - f);
  const int pg = a.kv.table[(size_t)c * a.kv.max_pages + p];
  r.pg = pg >= 0 && pg < a.kv.num_pages ? pg : -1;
  return r;
}

// Reports bad ranges: the first warp of CTA u < C looks at request u.
__device__ __forceinline__ void check_request(const Kv8MoveArgs& a, int c) {
  const int b = a.cu[c], e = a.cu[c + 1], f = a.first ? a.first[c] : 0;
  if (b < 0 || e < b || e > a.T || f < 0 || (long)f + ((long)e - b) > (long)a.kv.max_pages * a.kv.page_size)
    flag_error(a.err, kErrCtxOOB);
}

// V consecutive elements of a row as they lie in memory; 16-byte accesses for V = 16.
template <typename T, int V>
struct Raw {
  static constexpr int W = sizeof(T) * V / 16;
  uint4 w[W];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = __ldcs((const uint4*)p + i);
  }
  __device__ __forceinline__ void get(float (&v)[V]) const {
    const uint32_t* x = &w[0].x;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        v[2 * i] = __uint_as_float(x[i] << 16);
        v[2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = __uint_as_float(x[i]);
    }
  }
};
template <typename T>
struct Raw<T, 1> {
  T w;
  __device__ __forceinline__ void load(const T* p) { w = *p; }
  __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = to_f(w); }
};

template <int V>
__device__ __forceinline__ void store_row(float* p, const float (&v)[V]) {
  if constexpr (V == 16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) __stcs((float4*)p + i, make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
  } else {
    *p = v[0];
  }
}
template <int V>
__device__ __forceinline__ void store_row(bf16* p, const float (&v)[V]) {
  if constexpr (V == 16) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    __stcs((uint4*)p, make_uint4(w[0], w[1], w[2], w[3]));
    __stcs((uint4*)p + 1, make_uint4(w[4], w[5], w[6], w[7]));
  } else {
    *p = from_f<bf16>(v[0]);
  }
}

// Codes of V values times inv.
template <int V>
__device__ __forceinline__ void store_codes(uint8_t* o, const float (&v)[V], float inv) {
  if constexpr (V == 16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = e4m3x4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
    *(uint4*)o = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    *o = (uint8_t)e4m3x2(v[0] * inv, 0.f);
  }
}

template <int V>
__device__ __forceinline__ float largest(const float (&v)[V], float m) {
#pragma unroll
  for (int k = 0; k < V; ++k) m = fmaxf(m, kv8_mag(v[k]));
  return m;
}

// Row and first element of chunk i; `shift` = log2 of a row's chunks, or -1.
__device__ __forceinline__ void chunk_at(int i, int per_row, int shift, int& row, int& col) {
  row = shift >= 0 ? i >> shift : i / per_row;
  col = i - row * per_row;
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) kv8_write_kernel(const Kv8MoveArgs a, int shift) {
  const int lane = threadIdx.x & 31, y = blockIdx.y * kWarps + (threadIdx.x >> 5);
  if (blockIdx.y == 0 && threadIdx.x == 0 && blockIdx.x < (unsigned)a.C) check_request(a, blockIdx.x);
  const int g = y >> 1;
  const bool is_v = y & 1;
  if (g >= a.kv.Hkv) return;
  const Unit u = find_unit(a, blockIdx.x);
  if (u.n == 0) return;
  if (u.pg < 0) {
    if (lane == 0) flag_error(a.err, kErrPageOOB);
    return;
  }
  const int D = a.kv.D, per_row = D / V, total = u.n * per_row;
  const T* src = (const T*)(is_v ? a.v : a.k) + u.row * a.rs + (long)g * D;
  const size_t page_head = (size_t)u.pg * a.kv.Hkv + g;
  uint8_t* dst = (is_v ? a.kv.v : a.kv.k) + page_head * a.kv.page_size * D;
  float* scale = (is_v ? a.kv.vs : a.kv.ks) + page_head;
  const float old = u.slot0 > 0 ? *scale : 0.f;

  Raw<T, V> held[kHeld];
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    int row, col;
    chunk_at(lane + 32 * j, per_row, shift, row, col);
    if (lane + 32 * j < total) held[j].load(src + row * a.rs + col * V);
  }
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    float v[V];
    held[j].get(v);
    if (lane + 32 * j < total) amax = largest<V>(v, amax);
  }
  for (int i = lane + 32 * kHeld; i < total; i += 32) {
    int row, col;
    chunk_at(i, per_row, shift, row, col);
    Raw<T, V> x;
    float v[V];
    x.load(src + row * a.rs + col * V);
    x.get(v);
    amax = largest<V>(v, amax);
  }
  amax = warp_max(amax);
  const float mine = kv8_scale_of(amax);
  // (a NaN among the old scales loses against a number)
  const float now = u.slot0 > 0 ? fmaxf(old, mine) : mine;
  __syncwarp();  // every lane has read the old scale
  if (lane == 0) *scale = now;
  // an old scale that is no power of two of this call's making is divided by as it is
  const float inv = now == mine ? kv8_inverse(now) : fminf(1.f / now, 3.402823466e38f);
  uint8_t* out = dst + (size_t)u.slot0 * D;
#pragma unroll
  for (int j = 0; j < kHeld; ++j)
    if (lane + 32 * j < total) {
      float v[V];
      held[j].get(v);
      store_codes<V>(out + (size_t)(lane + 32 * j) * V, v, inv);
    }
  for (int i = lane + 32 * kHeld; i < total; i += 32) {
    int row, col;
    chunk_at(i, per_row, shift, row, col);
    Raw<T, V> x;
    float v[V];
    x.load(src + row * a.rs + col * V);
    x.get(v);
    store_codes<V>(out + (size_t)i * V, v, inv);
  }
  if (u.slot0 > 0 && now != old) {
    // the earlier tokens of the page under the new scale
    const float ratio = now > 0.f ? old / now : 0.f;
    for (int i = lane; i < u.slot0 * per_row; i += 32) {
      uint8_t* o = dst + (size_t)i * V;
      float v[V];
      if constexpr (V == 16) {
        const uint4 w = *(const uint4*)o;
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 x = e4m3x2_to_f2(ws[k >> 1] >> (16 * (k & 1)));
          v[2 * k] = x.x, v[2 * k + 1] = x.y;
        }
      } else {
        v[0] = e4m3_to_f(*o);
      }
      store_codes<V>(o, v, ratio);
    }
  }
}

// code * scale.  The product of 4 and 24 bits is exact in fp32 unless the scale
// uses its last four bits or the product leaves the normal range (never for the write's scales);
// ODD: it may, and is then rounded to odd, so that a store to bf16 rounds as if from the product
// itself.
template <bool ODD>
__device__ __forceinline__ float scaled(float x, float s) {
  if constexpr (!ODD) return x * s;
  const int p = __float_as_int(__fmul_rz(x, s));
  return __int_as_float(__fmul_rd(x, s) != __fmul_ru(x, s) ? p | 1 : p);
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) kv8_read_kernel(const Kv8MoveArgs a, int shift) {
  const int lane = threadIdx.x & 31, y = blockIdx.y * kWarps + (threadIdx.x >> 5);
  if (blockIdx.y == 0 && threadIdx.x == 0 && blockIdx.x < (unsigned)a.C) check_request(a, blockIdx.x);
  const int g = y >> 1;
  const bool is_v = y & 1;
  if (g >= a.kv.Hkv) return;
  const Unit u = find_unit(a, blockIdx.x);
  if (u.n == 0) return;
  if (u.pg < 0 && lane == 0) flag_error(a.err, kErrPageOOB);
  const int D = a.kv.D, per_row = D / V, total = u.n * per_row;
  T* dst = (T*)(is_v ? a.v : a.k) + u.row * a.rs + (long)g * D;
  const size_t page_head = (size_t)max(u.pg, 0) * a.kv.Hkv + g;
  const uint8_t* src = (is_v ? a.kv.v : a.kv.k) + (page_head * a.kv.page_size + u.slot0) * D;
  const float scale = (is_v ? a.kv.vs : a.kv.ks)[page_head];
  const bool zero = u.pg < 0;  // a bad page reads as zeros
  auto copy = [&](auto odd) {
    for (int i0 = lane; i0 < total; i0 += 32 * kHeld) {
      uint4 w[kHeld];
#pragma unroll
      for (int j = 0; j < kHeld; ++j) {
        const int i = i0 + 32 * j;
        if (i < total) {
          if constexpr (V == 16) w[j] = __ldcs((const uint4*)(src + (size_t)i * V));
          else w[j].x = src[i];
        }
      }
#pragma unroll
      for (int j = 0; j < kHeld; ++j) {
        const int i = i0 + 32 * j;
        if (i >= total) break;
        float v[V];
        const uint32_t* ws = &w[j].x;
        if constexpr (V == 16) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float2 x = e4m3x2_to_f2(ws[k >> 1] >> (16 * (k & 1)));
            v[2 * k] = scaled<odd.value>(x.x, scale), v[2 * k + 1] = scaled<odd.value>(x.y, scale);
          }
        } else {
          v[0] = scaled<odd.value>(e4m3_to_f((uint8_t)ws[0]), scale);
        }
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = zero ? 0.f : v[k];
        int row, col;
        chunk_at(i, per_row, shift, row, col);
        store_row<V>(dst + row * a.rs + col * V, v);
      }
    }
  };
  // (2^-117: a code is 2^-9 at least.  Branching here, not at each chunk: 16 prefixes 79 us, 82)
  if (sizeof(T) == 2 && ((__float_as_int(scale) & 15) != 0 || scale < 6.1e-36f)) copy(std::true_type());
  else copy(std::false_type());
}

// Sixteen elements at a time need D in multiples of sixteen, the row stride in multiples of
// 16 bytes and the rows 16-byte aligned (the codes are, by the entry points' check).
template <typename T>
bool wide(const Kv8MoveArgs& a) {
  return a.kv.D % 16 == 0 && a.rs * sizeof(T) % 16 == 0 && (((uintptr_t)a.k | (uintptr_t)a.v) & 15) == 0;
}

template <typename T>
void launch_move(bool write, const Kv8MoveArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)(a.T / a.kv.page_size + 2 * a.C), (unsigned)cdiv(2 * a.kv.Hkv, kWarps));
  const bool w = wide<T>(a);
  const int per_row = a.kv.D / (w ? 16 : 1);
  int shift = 0;
  while ((1 << shift) < per_row) ++shift;
  if ((1 << shift) != per_row) shift = -1;
  if (write) {
    if (w) kv8_write_kernel<T, 16><<<grid, kThreads, 0, s>>>(a, shift);
    else kv8_write_kernel<T, 1><<<grid, kThreads, 0, s>>>(a, shift);
  } else {
    if (w) kv8_read_kernel<T, 16><<<grid, kThreads, 0, s>>>(a, shift);
    else kv8_read_kernel<T, 1><<<grid, kThreads, 0, s>>>(a, shift);
  }
  note_launch();
}

}  // namespace

void kv8_write(int dtype, const Kv8MoveArgs& a, cudaStream_t s) {
  if (dtype == HSPEC_DTYPE_BF16) launch_move<bf16>(true, a, s);
  else launch_move<float>(true, a, s);
}

void kv8_read(int dtype, const Kv8MoveArgs& a, cudaStream_t s) {
  if (dtype == HSPEC_DTYPE_BF16) launch_move<bf16>(false, a, s);
  else launch_move<float>(false, a, s);
}

}  // namespace hspec
