// Writing tokens into the 8-bit paged KV cache and reading them back (hspec_kv8_write,
// hspec_kv8_read).
//
// Work unit: one page that a request's token range touches, of one kv head, K or V.  The
// touched pages of all requests are numbered without a pass over the lengths: request c
// owns the slots [cu[c] / page + 2c, cu[c+1] / page + 2(c + 1)), at least
// floor(n / page) + 2 of them for its n tokens, and n tokens touch at most
// floor((n - 1) / page) + 2 pages, so the slots suffice wherever the range starts; a CTA
// finds its request by bisection over c and leaves when its slot has no page.  The host
// knows the number of slots from T and C alone.
//
// Both directions are bound by HBM: the new rows once (2 or 4 bytes an element) and the
// codes once (1 byte).
#include "../../include/hspec.h"
#include "common.cuh"
#include "kernels.cuh"
#include "kv8.cuh"

namespace hspec {
namespace {

constexpr int kThreads = 128;

// The page of slot u: tokens [t0, t0 + n) of the request, slots [slot0, slot0 + n) of
// page `pg`, rows from `row` on.  n = 0: nothing (pg < 0 with n > 0: a bad page id).
struct Unit {
  int n, slot0, pg;
  long row;
};

__device__ __forceinline__ Unit find_unit(const Kv8MoveArgs& a, int u) {
  const int page = a.kv.page_size;
  Unit r = {0, 0, -1, 0};
  // the last request whose slots start at or before u
  int lo = 0, hi = a.C - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.cu[mid] / page + 2 * mid <= u) lo = mid;
    else hi = mid - 1;
  }
  const int c = lo, b = a.cu[c], e = a.cu[c + 1];
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

// Reports bad ranges: CTA u < C of the first head looks at request u.
__device__ __forceinline__ void check_request(const Kv8MoveArgs& a, int c) {
  const int b = a.cu[c], e = a.cu[c + 1], f = a.first ? a.first[c] : 0;
  if (b < 0 || e < b || e > a.T || f < 0 || (long)f + ((long)e - b) > (long)a.kv.max_pages * a.kv.page_size)
    flag_error(a.err, kErrCtxOOB);
}

// V consecutive elements as floats: 16-byte loads for V = 8, else one element.
template <int V>
__device__ __forceinline__ void load_row(const float* p, float (&v)[V]) {
  if constexpr (V == 8) {
    const float4 x = ((const float4*)p)[0], y = ((const float4*)p)[1];
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
  } else {
    v[0] = *p;
  }
}
template <int V>
__device__ __forceinline__ void load_row(const bf16* p, float (&v)[V]) {
  if constexpr (V == 8) {
    const uint4 x = *(const uint4*)p;
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    v[0] = to_f(*p);
  }
}
template <int V>
__device__ __forceinline__ void store_row(float* p, const float (&v)[V]) {
  if constexpr (V == 8) {
    ((float4*)p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    ((float4*)p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *p = v[0];
  }
}
template <int V>
__device__ __forceinline__ void store_row(bf16* p, const float (&v)[V]) {
  if constexpr (V == 8) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *(uint4*)p = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    *p = from_f<bf16>(v[0]);
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) kv8_write_kernel(const Kv8MoveArgs a) {
  __shared__ float red[32];
  const int g = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  if (blockIdx.y == 0 && threadIdx.x == 0 && blockIdx.x < (unsigned)a.C) check_request(a, blockIdx.x);
  const Unit u = find_unit(a, blockIdx.x);
  if (u.n == 0) return;
  if (u.pg < 0) {
    if (threadIdx.x == 0) flag_error(a.err, kErrPageOOB);
    return;
  }
  const int D = a.kv.D, per_row = D / V, total = u.n * per_row;
  const T* src = (const T*)(is_v ? a.v : a.k) + u.row * a.rs + (long)g * D;
  const size_t page_head = (size_t)u.pg * a.kv.Hkv + g;
  uint8_t* dst = (is_v ? a.kv.v : a.kv.k) + page_head * a.kv.page_size * D;
  float* scale = (is_v ? a.kv.vs : a.kv.ks) + page_head;
  const float old = u.slot0 > 0 ? *scale : 0.f;

  float amax = 0.f;
  for (int i = threadIdx.x; i < total; i += kThreads) {
    float v[V];
    load_row<V>(src + (i / per_row) * a.rs + (i % per_row) * V, v);
#pragma unroll
    for (int k = 0; k < V; ++k) amax = fmaxf(amax, kv8_mag(v[k]));
  }
  amax = warp_max(amax);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  __syncthreads();  // every thread has read the old scale, too
  amax = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  // (a NaN among the old scales loses against a number)
  const float now = u.slot0 > 0 ? fmaxf(old, kv8_scale_of(amax)) : kv8_scale_of(amax);
  if (threadIdx.x == 0) *scale = now;
  // an old scale that is no power of two of this call's making is divided by as it is
  const float inv = now == kv8_scale_of(amax) ? kv8_inverse(now) : now > 0.f ? fminf(1.f / now, 3.402823466e38f) : 0.f;
  for (int i = threadIdx.x; i < total; i += kThreads) {
    float v[V];
    load_row<V>(src + (i / per_row) * a.rs + (i % per_row) * V, v);
    uint8_t* o = dst + (u.slot0 + i / per_row) * D + (i % per_row) * V;
    if constexpr (V == 8) {
      *(uint2*)o = make_uint2(e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                              e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
    } else {
      *o = (uint8_t)e4m3x2(v[0] * inv, 0.f);
    }
  }
  if (u.slot0 > 0 && now != old) {
    // the earlier tokens of the page under the new scale
    const float ratio = now > 0.f ? old / now : 0.f;
    for (int i = threadIdx.x; i < u.slot0 * per_row; i += kThreads) {
      uint8_t* o = dst + (size_t)i * V;
      if constexpr (V == 8) {
        uint2 w = *(const uint2*)o;
        uint32_t* ws = &w.x;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float2 x = e4m3x2_to_f2(ws[k]), y = e4m3x2_to_f2(ws[k] >> 16);
          ws[k] = e4m3x4(x.x * ratio, x.y * ratio, y.x * ratio, y.y * ratio);
        }
        *(uint2*)o = w;
      } else {
        *o = (uint8_t)e4m3x2(e4m3_to_f(*o) * ratio, 0.f);
      }
    }
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) kv8_read_kernel(const Kv8MoveArgs a) {
  const int g = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  if (blockIdx.y == 0 && threadIdx.x == 0 && blockIdx.x < (unsigned)a.C) check_request(a, blockIdx.x);
  const Unit u = find_unit(a, blockIdx.x);
  if (u.n == 0) return;
  if (u.pg < 0 && threadIdx.x == 0) flag_error(a.err, kErrPageOOB);
  const int D = a.kv.D, per_row = D / V, total = u.n * per_row;
  T* dst = (T*)(is_v ? a.v : a.k) + u.row * a.rs + (long)g * D;
  const size_t page_head = (size_t)max(u.pg, 0) * a.kv.Hkv + g;
  const uint8_t* src = (is_v ? a.kv.v : a.kv.k) + (page_head * a.kv.page_size + u.slot0) * D;
  const float scale = (is_v ? a.kv.vs : a.kv.ks)[page_head];
  for (int i = threadIdx.x; i < total; i += kThreads) {
    float v[V];
    if constexpr (V == 8) {
      const uint2 w = *(const uint2*)(src + (size_t)i * 8);
      const uint32_t ws[2] = {w.x, w.y};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 x = e4m3x2_to_f2(ws[k >> 1] >> (16 * (k & 1)));
        v[2 * k] = x.x * scale, v[2 * k + 1] = x.y * scale;
      }
    } else {
      v[0] = e4m3_to_f(src[i]) * scale;
    }
    if (u.pg < 0)
#pragma unroll
      for (int k = 0; k < V; ++k) v[k] = 0.f;
    store_row<V>(dst + (i / per_row) * a.rs + (i % per_row) * V, v);
  }
}

// 16-byte rows: eight elements at a time need D and the row stride in multiples of
// eight and the rows 16-byte aligned (the codes are, by the entry points' check).
bool wide(const Kv8MoveArgs& a) {
  return a.kv.D % 8 == 0 && a.rs % 8 == 0 && (((uintptr_t)a.k | (uintptr_t)a.v) & 15) == 0;
}

template <typename T>
void launch_move(bool write, const Kv8MoveArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)(a.T / a.kv.page_size + 2 * a.C), (unsigned)(2 * a.kv.Hkv));
  if (write) {
    if (wide(a)) kv8_write_kernel<T, 8><<<grid, kThreads, 0, s>>>(a);
    else kv8_write_kernel<T, 1><<<grid, kThreads, 0, s>>>(a);
  } else {
    if (wide(a)) kv8_read_kernel<T, 8><<<grid, kThreads, 0, s>>>(a);
    else kv8_read_kernel<T, 1><<<grid, kThreads, 0, s>>>(a);
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
