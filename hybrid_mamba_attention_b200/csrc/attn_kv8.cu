// Paged block attention over the 8-bit KV cache (hspec_attn_paged_block_kv8): the
// CUDA-core split kernel for any shape, the split policy, and the merge of the partials.
//
// attn_kv8_split_kernel: one CTA per (split, kv head g and block of 32 or 64 query rows,
// request c).  Its rows are (position j, query head g*G + i) pairs, all reading kv head
// g.  Keys and values pass through shared memory in tiles of 32, dequantised to fp32
// (code * scale is exact there for the write's powers of two); a warp owns four rows or eight: lane t computes their dot
// products with key t, the online softmax (exp2 domain) reduces over the lanes, and for
// the product with V a lane owns the dims t, t + 32, ...  Hidden keys are skipped, not
// multiplied by zero, so that a NaN in one reaches no row that does not see it.
//
// attn_kv8_merge_kernel: W = 1, 2, 4 or 8 warps per output row combine its partials,
// o = sum_s 2^(m_s - M) acc_s / sum_s 2^(m_s - M) l_s, in a fixed order.
#include "../../include/hspec.h"
#include "common.cuh"
#include "kernels.cuh"
#include "kv8.cuh"

namespace hspec {

int* device_error_word();

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 32;              // keys per tile
constexpr int kKeys = kTile / kWarps;  // keys of a tile that a warp copies

// Query rows per warp, RW: each row more shares a key's loads from shared memory, eight cost
// registers that the widest heads have not got (8 requests of 512 .. 4096 tokens, 64 rows a kv
// head of 128 dims: 296 us with eight, 353 with four; 36 rows of 64 dims: 186 and 196).
__host__ __device__ inline int rows_per_warp(int R, int D) { return R > 4 * kWarps && D <= 128 ? 8 : 4; }
inline int row_blocks(int R, int D) { return cdiv(R, kWarps * rows_per_warp(R, D)); }

// Shared memory in floats: q [8 RW][Dp], k [32][Dp + 4] (a lane per key reads float4s: the
// four extra words put the lanes on different banks), v [32][Dp], p [8][32][RW].
__host__ __device__ inline int dim_pad(int D) { return (D + 3) & ~3; }
inline size_t split_smem(int D, int RW) {
  const int Dp = dim_pad(D), rows = kWarps * RW;
  return (size_t)(rows * Dp + kTile * (Dp + 4) + kTile * Dp + rows * kTile) * sizeof(float);
}

// E dims per lane: head_dim <= 32 E.
template <typename T, int E, int RW>
__global__ void __launch_bounds__(kThreads, 2) attn_kv8_split_kernel(const AttnKv8Args a, float scale_log2) {
  pdl_wait();  // the previous kernel on the stream is complete from here on
  pdl_trigger();
  constexpr int kRows = kWarps * RW;
  extern __shared__ float4 sm4[];
  float* sm = (float*)sm4;
  const int D = a.kv.D, Dp = dim_pad(D), Hkv = a.kv.Hkv, page = a.kv.page_size;
  float* sQ = sm;
  float* sK = sQ + kRows * Dp;
  float* sV = sK + kTile * (Dp + 4);
  float* sP = sV + kTile * Dp;
  const int split = blockIdx.x, g = blockIdx.y % Hkv, rb = blockIdx.y / Hkv, c = blockIdx.z;
  const int G = a.Hq / Hkv, R = a.K * G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ctx = a.ctx_lens[c];
  if (ctx < 0 || ctx > (long)a.kv.max_pages * page) {
    if (threadIdx.x == 0) flag_error(a.err, kErrCtxOOB);
    return;
  }
  const int total = ctx + (a.kb ? a.K : 0);
  const int t_begin = split * a.split_tokens;
  if (t_begin >= total) return;  // the merge reads only the splits that hold tokens
  const int t_end = min(total, t_begin + a.split_tokens);

  // keys [0, vis) are seen by the row
  int vis[RW];
  float m[RW], l[RW], acc[RW][E];
#pragma unroll
  for (int r = 0; r < RW; ++r) {
    const int row = rb * kRows + warp * RW + r, j = row / G;
    const T* q = (const T*)a.q + (size_t)(c * a.K + j) * a.q_rs + (size_t)(g * G + row % G) * D;
    for (int e = lane; e < Dp; e += 32)  // read by this warp alone
      sQ[(warp * RW + r) * Dp + e] = row < R && e < D ? to_f(q[e]) * scale_log2 : 0.f;
    vis[r] = row >= R ? 0 : !a.causal ? total : a.kb ? ctx + j + 1 : ctx - (a.K - 1) + j;
    m[r] = -INFINITY, l[r] = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) acc[r][i] = 0.f;
  }
  const int32_t* table = a.kv.table + (size_t)c * a.kv.max_pages;

  // Lane t of each warp looks up the page and the scales of key t0 + t, so that the copies of
  // the codes that follow depend on nothing but registers.
  auto look_up = [&](int t0, long& off, float& ks, float& vs) {
    const int t = t0 + lane;
    off = -1, ks = vs = 0.f;  // a bad page's keys read as 0
    if (t >= min(t_end, ctx)) return;
    const int pg = table[t / page];
    if (pg >= 0 && pg < a.kv.num_pages) {
      const size_t ph = (size_t)pg * Hkv + g;
      off = (long)((ph * page + t % page) * D), ks = a.kv.ks[ph], vs = a.kv.vs[ph];
    } else {
      flag_error(a.err, kErrPageOOB);
    }
  };
  long off, off_next;
  float ks, vs, ks_next, vs_next;
  look_up(t_begin, off, ks, vs);
  for (int t0 = t_begin; t0 < t_end; t0 += kTile) {
    look_up(t0 + kTile, off_next, ks_next, vs_next);
    __syncthreads();
    // a warp copies four keys, a lane the dims lane, lane + 32, ...
    for (int e0 = 0; e0 < Dp; e0 += 32) {
      const int e = e0 + lane;
      float k[kKeys], v[kKeys];
#pragma unroll
      for (int i = 0; i < kKeys; ++i) {
        const int tt = warp * kKeys + i, t = t0 + tt;
        const long o = __shfl_sync(0xffffffffu, off, tt);
        const float kscale = __shfl_sync(0xffffffffu, ks, tt), vscale = __shfl_sync(0xffffffffu, vs, tt);
        k[i] = v[i] = 0.f;
        if (e < D && o >= 0) {
          k[i] = e4m3_to_f(a.kv.k[o + e]) * kscale;
          v[i] = e4m3_to_f(a.kv.v[o + e]) * vscale;
        } else if (e < D && t >= ctx && t < t_end) {
          const size_t row = (size_t)(c * a.K + (t - ctx));
          k[i] = to_f(((const T*)a.kb)[row * a.kb_rs + (size_t)g * D + e]);
          v[i] = to_f(((const T*)a.vb)[row * a.vb_rs + (size_t)g * D + e]);
        }
      }
      if (e < Dp) {
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
          sK[(warp * kKeys + i) * (Dp + 4) + e] = k[i];
          sV[(warp * kKeys + i) * Dp + e] = v[i];
        }
      }
    }
    off = off_next, ks = ks_next, vs = vs_next;
    __syncthreads();
    float s[RW];
#pragma unroll
    for (int r = 0; r < RW; ++r) s[r] = 0.f;
    for (int e = 0; e < Dp; e += 4) {
      const float4 k = *(const float4*)(sK + lane * (Dp + 4) + e);
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        const float4 q = *(const float4*)(sQ + (warp * RW + r) * Dp + e);
        s[r] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, s[r]))));
      }
    }
    int nv[RW];
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      nv[r] = min(max(min(vis[r], t_end) - t0, 0), kTile);  // keys of the tile that the row sees
      const float sc = lane < nv[r] ? s[r] : -INFINITY;
      const float m_new = fmaxf(m[r], warp_max(sc));
      // with nothing visible yet (or NaN alone) subtract 0: a masked weight is 0, not NaN
      const float base = m_new == -INFINITY ? 0.f : m_new;
      const float p = lane < nv[r] ? exp2f(sc - base) : 0.f;
      const float alpha = m[r] == -INFINITY ? (l[r] == 0.f ? 0.f : 1.f) : exp2f(m[r] - m_new);
      l[r] = l[r] * alpha + warp_sum(p);
      m[r] = m_new;
#pragma unroll
      for (int i = 0; i < E; ++i) acc[r][i] *= alpha;
      sP[(warp * kTile + lane) * RW + r] = p;
    }
    __syncwarp();
    // Keys that all the warp's rows see, without a test; then those that some do.  A lane's dims
    // from D on add up what follows in shared memory (a row's end reads at most 256 floats on, into
    // p), and are never stored.
    static_assert(RW % 4 == 0, "a key's weights are read as float4s");
    int all = nv[0], any = nv[0];
#pragma unroll
    for (int r = 1; r < RW; ++r) all = min(all, nv[r]), any = max(any, nv[r]);
    const float4* p4 = (const float4*)(sP + warp * kTile * RW);
    const float* v1 = sV + lane;
#pragma unroll 4
    for (int t = 0; t < all; ++t) {
      float v[E];
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = v1[t * Dp + 32 * i];
#pragma unroll
      for (int r = 0; r < RW; r += 4) {
        const float4 p = p4[(t * RW + r) / 4];
#pragma unroll
        for (int i = 0; i < E; ++i) {
          acc[r][i] = fmaf(p.x, v[i], acc[r][i]);
          acc[r + 1][i] = fmaf(p.y, v[i], acc[r + 1][i]);
          acc[r + 2][i] = fmaf(p.z, v[i], acc[r + 2][i]);
          acc[r + 3][i] = fmaf(p.w, v[i], acc[r + 3][i]);
        }
      }
    }
    for (int t = all; t < any; ++t) {
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        if (t >= nv[r]) continue;
#pragma unroll
        for (int i = 0; i < E; ++i)
          acc[r][i] = fmaf(sP[(warp * kTile + t) * RW + r], v1[t * Dp + 32 * i], acc[r][i]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < RW; ++r) {
    const int row = rb * kRows + warp * RW + r;
    if (row >= R) break;
    const size_t base = (((size_t)c * Hkv + g) * a.n_splits + split) * R + row;
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (lane + 32 * i < D) a.ws_acc[base * D + lane + 32 * i] = acc[r][i];
    if (lane == 0) {
      a.ws_ml[base * 2] = m[r];
      a.ws_ml[base * 2 + 1] = l[r];
    }
  }
}

// W warps per row; lane t holds the dims t + 32 i, i < E.
template <typename T, int W, int E>
__global__ void __launch_bounds__(256) attn_kv8_merge_kernel(const AttnKv8Args a) {
  pdl_wait();  // the previous kernel on the stream is complete from here on
  pdl_trigger();
  constexpr int RPC = 8 / W;  // rows per CTA
  __shared__ float s_acc[W > 1 ? 8 : 1][32 * E];
  __shared__ float s_ml[8][2];
  const int D = a.kv.D, Hkv = a.kv.Hkv;
  const int wib = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wq = wib % W, rl = wib / W;
  const int G = a.Hq / Hkv, R = a.K * G;
  const long rows = (long)a.C * a.K * a.Hq;
  const long row_id = (long)blockIdx.x * RPC + rl;
  const bool live = row_id < rows;
  const long rid = live ? row_id : 0;
  const int h = (int)(rid % a.Hq), j = (int)(rid / a.Hq % a.K), c = (int)(rid / a.Hq / a.K);
  const int g = h / G, row = j * G + h % G;
  const int ctx = a.ctx_lens[c];
  const bool valid = live && ctx >= 0 && ctx <= (long)a.kv.max_pages * a.kv.page_size;
  // The row's partials, one per split of (c, g).
  const int ns = valid ? (ctx + (a.kb ? a.K : 0) + a.split_tokens - 1) / a.split_tokens : 0;
  const size_t base0 = ((size_t)c * Hkv + g) * a.n_splits * R + row, stride = R;
  float M = -INFINITY, L = 0.f, o[E];
#pragma unroll
  for (int i = 0; i < E; ++i) o[i] = 0.f;
  auto fold = [&](float m, float l, auto acc_of) {
    if (l == 0.f) return;  // no key seen
    const float mn = fmaxf(M, m);
    const float sc = L == 0.f ? 0.f : exp2f(M - mn), w = exp2f(m - mn);
    L = L * sc + l * w;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = o[i] * sc + acc_of(i) * w;
    M = mn;
  };
  for (int q = wq; q < ns; q += W) {
    const size_t b = base0 + (size_t)q * stride;
    const float2 ml = *(const float2*)(a.ws_ml + b * 2);
    const float* acc = a.ws_acc + b * D;
    fold(ml.x, ml.y, [&](int i) { return lane + 32 * i < D ? acc[lane + 32 * i] : 0.f; });
  }
  if constexpr (W > 1) {
#pragma unroll
    for (int i = 0; i < E; ++i) s_acc[wib][lane + 32 * i] = o[i];
    if (lane == 0) s_ml[wib][0] = M, s_ml[wib][1] = L;
    __syncthreads();
    if (wq != 0) return;
    for (int w = 1; w < W; ++w)
      fold(s_ml[wib + w][0], s_ml[wib + w][1], [&](int i) { return s_acc[wib + w][lane + 32 * i]; });
  }
  if (!live) return;
  T* out = (T*)a.out + (size_t)(c * a.K + j) * a.o_rs + (size_t)h * D;
  const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (lane + 32 * i < D) out[lane + 32 * i] = from_f<T>(o[i] * inv);
}

template <typename T, int W>
void launch_merge_w(const AttnKv8Args& a, long rows, cudaStream_t s) {
  const int grid = (int)((rows + 8 / W - 1) / (8 / W));
  if (a.kv.D <= 128) launch_pdl(attn_kv8_merge_kernel<T, W, 4>, grid, 256, 0, s, a);
  else launch_pdl(attn_kv8_merge_kernel<T, W, 8>, grid, 256, 0, s, a);
  note_launch();
}

template <typename T>
void launch_merge(const AttnKv8Args& a, cudaStream_t s) {
  // warps per output row: enough warps in all for about 32 per SM
  const long rows = (long)a.C * a.K * a.Hq;
  int W = 1;
  while (W < 8 && rows * W < 148L * 32) W *= 2;
  switch (W) {
    case 1: launch_merge_w<T, 1>(a, rows, s); break;
    case 2: launch_merge_w<T, 2>(a, rows, s); break;
    case 4: launch_merge_w<T, 4>(a, rows, s); break;
    default: launch_merge_w<T, 8>(a, rows, s); break;
  }
}

template <typename T, int E, int RW>
bool launch_split_e(const AttnKv8Args& a, cudaStream_t s) {
  const size_t smem = split_smem(a.kv.D, RW);
  auto kernel = attn_kv8_split_kernel<T, E, RW>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) {
    set_error("cudaFuncSetAttribute(attn_kv8_split_kernel) failed");
    return false;
  }
  const int nrb = row_blocks(a.K * (a.Hq / a.kv.Hkv), a.kv.D);
  const float scale_log2 = 1.4426950408889634f / sqrtf((float)a.kv.D);
  launch_pdl(kernel, dim3(a.n_splits, a.kv.Hkv * nrb, a.C), kThreads, smem, s, a, scale_log2);
  note_launch();
  return true;
}

template <typename T>
bool launch_split(const AttnKv8Args& a, cudaStream_t s) {
  const bool eight = rows_per_warp(a.K * (a.Hq / a.kv.Hkv), a.kv.D) == 8;
  if (a.kv.D <= 64) return eight ? launch_split_e<T, 2, 8>(a, s) : launch_split_e<T, 2, 4>(a, s);
  if (a.kv.D <= 128) return eight ? launch_split_e<T, 4, 8>(a, s) : launch_split_e<T, 4, 4>(a, s);
  return launch_split_e<T, 8, 4>(a, s);
}

// CUDA-core path: tokens per split (a requested length, or about 16 CTAs per SM at the
// table's full width) and splits per sequence.
struct Split {
  int tokens, n;
  int most;  // the most splits that a table of this width or a narrower one gives
};
constexpr long kSplitCtas = 148L * 16;
Split split_of(int C, int K, int G, const Kv8& kv, int req) {
  const long max_keys = (long)kv.max_pages * kv.page_size + K;
  const long lines = (long)C * kv.Hkv * row_blocks(K * G, kv.D);
  long per = req > 0 ? req : (lines * max_keys + kSplitCtas - 1) / kSplitCtas;
  // A single tile where that gives every SM work enough (2 requests of 77 tokens: 9.9 us, 13.7
  // with two tiles); pairs of tiles otherwise (32 of 8192: 180 us in 256s, 194 in 224s).
  per = per <= kTile ? kTile : (per + 2 * kTile - 1) / (2 * kTile) * (2 * kTile);
  // the grid's x extent holds the splits: no limit in reach (2^31), so any length works
  const long n = (max_keys + per - 1) / per;
  // The length is rounded up in steps, so a wider table may have fewer splits than a narrower
  // one.  At any width a split has a tile at least and, unless its length is given, max_keys
  // lines / kSplitCtas keys: both counts only grow with max_keys.
  const long tiles = (max_keys + kTile - 1) / kTile, even = (kSplitCtas + lines - 1) / lines;
  return {(int)(per < max_keys ? per : max_keys), (int)n, (int)(req > 0 ? n : tiles < even ? tiles : even)};
}

}  // namespace

bool attn_kv8_supported(int dtype, int C, int K, int Hq, const Kv8& kv, int split_req, const char** why) {
  const long G = Hq / kv.Hkv;
  if (K < 1 || K > 64) return *why = "K must be in 1..64", false;
  if (kv.D > 256) return *why = "head_dim must be <= 256", false;
  if (K * G > 65536) return *why = "K * Hq / Hkv must be <= 65536", false;
  if (attn_kv8_tc_shape(dtype, kv.D, kv.page_size)) return attn_kv8_tc_fits(C, K, Hq, kv, split_req, why);
  // the grid's y and z extents
  if (C > 65535) return *why = "C must be <= 65535 off the tensor-core path", false;
  if (kv.Hkv * (long)row_blocks((int)(K * G), kv.D) > 65535)
    return *why = "more than 65535 kv heads times blocks of query rows", false;
  return true;
}

size_t attn_kv8_ws_bytes(int dtype, int C, int K, int Hq, const Kv8& kv, int split_req, bool narrower) {
  if (attn_kv8_tc_shape(dtype, kv.D, kv.page_size)) {
    AttnKv8Args a = {};
    a.kv = kv, a.C = C, a.K = K, a.Hq = Hq;
    return attn_kv8_tc_plan(a, split_req, nullptr);
  }
  const int G = Hq / kv.Hkv;
  const Split sp = split_of(C, K, G, kv, split_req);
  const size_t rows = (size_t)C * kv.Hkv * (narrower ? sp.most : sp.n) * K * G;
  return rows * (kv.D + 2) * sizeof(float);
}

bool attn_kv8(int dtype, AttnKv8Args& a, int split_req, void* ws, cudaStream_t s) {
  if (attn_kv8_tc_shape(dtype, a.kv.D, a.kv.page_size)) {
    attn_kv8_tc_plan(a, split_req, ws);
    return attn_kv8_tc_launch(a, s);
  }
  const int G = a.Hq / a.kv.Hkv;
  const Split sp = split_of(a.C, a.K, G, a.kv, split_req);
  a.split_tokens = sp.tokens, a.n_splits = sp.n;
  const size_t rows = (size_t)a.C * a.kv.Hkv * sp.n * a.K * G;
  a.ws_acc = (float*)ws;
  a.ws_ml = a.ws_acc + rows * a.kv.D;
  if (dtype == HSPEC_DTYPE_BF16) {
    if (!launch_split<bf16>(a, s)) return false;
    launch_merge<bf16>(a, s);
  } else {
    if (!launch_split<float>(a, s)) return false;
    launch_merge<float>(a, s);
  }
  return true;
}

}  // namespace hspec
