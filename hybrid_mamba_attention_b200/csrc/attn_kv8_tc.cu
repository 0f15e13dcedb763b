// Paged block attention over the 8-bit KV cache on the 5th-generation tensor cores (bf16
// queries, D = 64 or 128, page_size a multiple of 16).
//
// Both products run on the codes as they lie in the cache (kind::f8f6f4, e4m3), with the
// roles of keys and queries exchanged: a tile of 128 keys is the M side, the R query rows
// of a kv head the N side,
//     S^T [128 keys x R]  = K [128 x D] . Q^T           (K straight from the page, K-major)
//     O^T [D x R]        += V^T [D x 128 keys] . P^T    (V straight from the page, MN-major)
// so that a thread's TMEM lane is a key, whose page scales are one register each, and the
// tensor time falls with R (a decoded token has R = group size).  Nothing is dequantised:
// the K scale multiplies S^T, the V scale the weights P.
//
// Rounding.  A bf16 query row is scaled by a power of two and held as two e4m3 parts,
// hi + lo, which carry its 8 bits (down to 2^-17 of the row's largest element); both are
// multiplied with K into one fp32 accumulator.  The weights p = 2^(s - m) <= 2^5 enter as
// P = p * 2^3 * (V scale / largest V scale so far), hi = e4m3(P) and lo = e4m3(32 (P - hi))
// side by side in one N = 2R product, O = O_hi + O_lo / 32: 8 bits down to 2^-10 of the
// reference m, an absolute 2^-18 below.  Row sums use the unrounded fp32 weights.  The
// block's own bf16 keys and values are two e4m3 parts with a power-of-two scale per row, too.
//
// The reference m of a query starts as the first tile's maximum.  A tile's weights are
// computed under the references so far, then checked: only where one exceeds 2^5 (or a V
// scale the largest so far), which one barrier with an OR tells the group, the references
// rise to the maxima, O and the sums are rescaled and the tile is weighed again.  They come
// down, too, where they are looked at: weights far below the reference have few bits, and a key
// that outweighs all others (the first of a context does as a rule) would hide what follows.
// That is a piece's second item, every 32nd from there on, and behind a rise by more than 2^8
// the items 1, 5 and 21 on (a look costs about as much as an item: two more a piece, whatever
// the data, made 128 requests of 64 columns 7 % slower each).  So at most 31 items' keys, each
// below 2^-18, enter the sum and not O.
//
// Work partition: as the bf16 path's, the sequences (request, row block, kv head) lie end
// to end on a line of units, kAttn8SeqUnits for a start and one per 128-key tile; the line
// is cut into one chunk per SM, and a piece (one sequence's tiles in a chunk) writes one or
// two partials for the merge kernel.  The preparation kernel sums the line and, in its other
// CTAs, writes the queries' and the block's two-part images in their shared-memory layout,
// each then one bulk copy.
//
// Warp roles (one persistent CTA per SM; counts in Warps<NR>): producers, a warp for K and
// one for V (a tile's pages as TMA boxes of up to 128 rows and the pages' scales, a lane
// each); one warp that issues S^T, one that issues O^T; softmax groups of four warps, a
// thread per key, on two sides with an accumulator O^T each.  Up to 64 query rows the sides
// take the tiles in turn (one side's softmax runs under the other's products, two partials a
// piece); up to 128 rows each takes half of the rows of every tile, so that a tile's bytes
// serve both.
//
// What bounds it, at 32 query and 8 KV heads of 128 dims but for the first: few columns HBM,
// 2 D bytes a key and kv head (64 requests of 1024 .. 32768 tokens, 64 query heads, one
// position: 363 .. 390 us, 5.7 .. 6.1 TB/s of the 6.56 that a copy reaches); with more, the
// chain that turns S^T into P and its latency: 27 instructions issued a weight in all warps, about
// nine of them in weighing and three of those its split in two parts, 0.6 of the issue slots (128
// requests of 512 .. 16384 tokens, 16 positions: 800 us in a burst, 830 .. 890 back to back under
// the power cap, 2.7 TB/s; prepare 25 and merge 34 of them); single requests the three kernels' latencies (512 tokens: 16 us; prepare 4, this 9,
// merge 4).  Every wait gives up after a time bound and sets the device error word.
#include <stdint.h>

#include "../../include/hspec.h"
#include "common.cuh"
#include "kernels.cuh"
#include "kv8.cuh"
#include "tc_prims.cuh"

namespace hspec {
namespace {

constexpr int TT = kAttn8Tile;  // keys per tile
// Warps and registers by the width of the query side.  Two sides take the work in turn; CG groups
// of four warps share the columns of a side's item.
// Up to 16 columns one group holds an item whole: its fixed instructions (tests, barriers, the
// marks of the rows) are then paid once (64 requests of 8 columns a KV head: 380 us with one group,
// 411 with two).  With more columns two groups hide each other's latencies (128 requests of 64
// columns: 835 us with two, 945 with one and the registers of both; 32 columns: 296 and 309).
// Up to 32 columns a producer pair's instructions from tile to tile are the longest of the chain,
// so two pairs take turns; with more the softmax is, and its threads need the registers that a
// second pair would take (the 64 columns: 850 us with one pair, 967 with two).
// setmaxnreg moves registers inside what the launch gives, THREADS * LAUNCH: 256 * 72 + 256 * 184
// = 512 * 128, 256 * 64 + 512 * 88 = 768 * 80, 128 * 64 + 512 * 104 = 640 * 96.
template <int NR>
struct Warps {
  static constexpr int CG = NR <= 16 ? 1 : 2;
  static constexpr int NPW = NR <= 32 ? 4 : 2;       // producer warps: K's and V's, per pair
  static constexpr int SM_WARP0 = NR <= 32 ? 8 : 4;  // first softmax warp (a multiple of 4: warp % 4 is its TMEM quarter)
  static constexpr int THREADS = 32 * (SM_WARP0 + 8 * CG);
  static constexpr int kFewRegs = CG == 1 ? 72 : 64, kManyRegs = CG == 1 ? 184 : NR <= 32 ? 88 : 104;
};
constexpr float kPScale = 8.f;    // 2^3: weights enter P times this
constexpr float kOver = 32.f;     // 2^5: a weight may reach this before the reference rises (P: 2^8 of e4m3's 448)
constexpr float kSlack = 3.f;     // where it is looked at, a reference over a tile's maximum by more than 2^3
constexpr float kBelow = 60.f;    // comes down to that, though not below 2^-60 of the largest score so far
constexpr int kSettle = 32;       // looked at in a piece's second item, then every 32; and from a rise on by more
constexpr float kFar = 8.f;       // than 2^8 since the last look at gaps of 1, 4, 16, 32, ...
constexpr float kLoScale = 32.f;  // the low part of P is held times this (the rest of up to 2^8 is 2^3 at most)
constexpr int kMaxChunksAuto = 256, kMaxChunksExplicit = 2048;
constexpr int kBlkRows = 64;      // scales of a block's rows (K <= 64)

// Rows of a block's images: its K keys in whole 32-key steps of the product with V.
__host__ __device__ inline int blk_rows(int K) { return (K + 31) & ~31; }

// Byte offset of 16-byte chunk `ch` of row r in rows of W = 128, 64 or 32 bytes, swizzled over
// spans of that width.
template <int W>
__device__ __forceinline__ uint32_t swz(int r, int ch) {
  return (uint32_t)(r * W + ((W == 128 ? ch ^ (r & 7) : W == 64 ? ch ^ ((r >> 1) & 3) : ch ^ ((r >> 2) & 1)) << 4));
}

// Query image of a sequence: hi rows, lo rows (NR rows of D bytes each, swizzled), then
// the rows' scales (fp32).
__host__ __device__ inline size_t q_img_bytes(int NR, int D) { return (size_t)NR * (2 * D + 4); }

template <int D, int NR, bool PAIR>
struct Lay {
  static constexpr int ROWS = PAIR ? 2 * NR : NR;         // query rows of a sequence
  static constexpr int PN = NR == 16 ? 32 : NR == 32 ? 64 : 128;  // columns of O^T: hi from 0, lo from PN / 2
  static constexpr int Q_BYTES = ROWS * (2 * D + 4);
  static constexpr int Q_BUF = (Q_BYTES + 1023) & ~1023;
  static constexpr int KV = TT * D;                       // one operand of a stage
  static constexpr int STAGE = 2 * KV;
  static constexpr int P_BUF = TT * PN;                   // one byte an element
  static constexpr int OFF_Q = (2 * P_BUF + 1023) & ~1023;
  static constexpr int MISC = NR > 48 ? 6656 : 6144;
  // K/V ring stages beside nq query buffers
  static constexpr int stages(int nq) {
    const int room = (227 * 1024 - 1024 - MISC - OFF_Q - nq * Q_BUF) / STAGE;
    return room < 8 ? room : 8;
  }
  // Query buffers: the producers run ahead by as many pieces, which short contexts need (102
  // requests of 65 tokens, 32 kv heads: 148 us with four, 158 with two); up to 32 rows as many, up
  // to four, as cost no stage (more rows: two or three are alike).
  static constexpr int NQ = PAIR ? 1 : NR > 32 ? 2 : stages(4) == stages(2) ? 4 : stages(3) == stages(2) ? 3 : 2;
  static constexpr int NS = stages(NQ);
  static constexpr int OFF_KV = OFF_Q + NQ * Q_BUF;
  static constexpr int OFF_MISC = OFF_KV + NS * STAGE;
  static constexpr int SMEM = OFF_MISC + MISC + 1024;
  static constexpr uint32_t TMEM_COLS = 512;
  __host__ __device__ static constexpr uint32_t O_COL(int w) { return (uint32_t)(w * PN); }
  __host__ __device__ static constexpr uint32_t S_COL(int b) { return (uint32_t)(2 * PN + b * NR); }
  static_assert(NS >= 3, "ring");
  static_assert(2 * PN + 4 * NR <= (int)TMEM_COLS, "TMEM");
};

enum : int {  // TileMeta::flags
  kEnd = 1,       // no more work (nothing else is set)
  kFirst = 2,     // first tile of its piece
  kLast = 4,      // last tile of its piece
  kGroupFirst = 8, kGroupLast = 16,  // of its piece's tiles that the same side takes
  kBlock = 32,    // the block's own keys
  kMixed = 64,    // some key of the tile is hidden from some position
  kQPar = 128,    // parity of the load into the piece's query buffer,
  kQShift = 8,    // whose number is in bits 8 and 9
  kHalf = 1024,   // odd tile of its piece
};
struct alignas(16) TileMeta {  // written by producer warp 0 before the stage's barrier arrive
  int flags, cg, rb, slot;     // cg = request * Hkv + kv head; row block; the piece's slot
  int valid;                   // keys in the tile
  int joff;                    // key i of the tile is seen by the positions j >= joff + i
  int pad[2];
};

template <int NR>
struct Misc {
  uint64_t kv_full[8], kv_empty[8], s_full[4], s_free[4], p_full[2], pv_done[2], q_full[4], q_empty[4], drain[2];
  uint32_t tmem;
  int end_item;             // items from here on do not exist
  TileMeta meta[8];
  float scale[8][16];       // per stage: K scales of its eight 16-key groups, then V scales
  // per softmax group
  static constexpr int NG = 2 * Warps<NR>::CG, NC = NR / Warps<NR>::CG;  // groups, their columns
  alignas(16) float cq[NG][NC];       // the query rows' scales
  alignas(16) float nm[NG][NC];       // -reference (0 while there is none)
  alignas(16) float alpha[NG][NC];
  float m[NG][NC], top[NG][NC];       // the reference; the largest score so far
  float base[NG][NC];                 // the reference when it was last looked at
  float cmax[NG][4][NC];              // per warp: column maxima, later the rows' sums
  float svmax[NG][4];
  int pend_base[NG], pend_rows[NG];   // the partial that O^T still holds
  float pend_mul[NG];
  int look[NG], gap[NG];              // the item at which the references are looked at next; the gap before it
  uint4 v_nan[8];           // per stage: keys whose V row holds a NaN, as the groups find it
};

struct Maps {
  CUtensorMap k, v;
};

__device__ __forceinline__ int seq_units(int ctx, long max_ctx, int nbt) {
  const int tiles = ctx < 0 || ctx > max_ctx ? 0 : (ctx + TT - 1) / TT + nbt;
  return tiles > 0 ? kAttn8SeqUnits + tiles : 0;
}

// Two e4m3 parts of four values (NaN for a value that is not finite).
__device__ __forceinline__ void split4(const float (&x)[4], uint32_t& hi, uint32_t& lo) {
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = fabsf(x[i]) <= 3.402823466e38f ? x[i] : __int_as_float(0x7fffffff);
  hi = e4m3x4(v[0], v[1], v[2], v[3]);
  const float2 a = e4m3x2_to_f2(hi), b = e4m3x2_to_f2(hi >> 16);
  lo = e4m3x4(v[0] - a.x, v[1] - a.y, v[2] - b.x, v[3] - b.y);
}

// Power of two that takes a row of largest magnitude m to [128, 256), and its inverse.
__device__ __forceinline__ float row_factor(float m, float& inv) {
  const int e = max(__float_as_int(m) >> 23, 27);  // biased exponent; 2^-100 at least
  inv = __int_as_float((e - 7) << 23);
  return __int_as_float((254 + 7 - e) << 23);
}

// CTA 0: the line's offsets and the partition.  The others: two-part images, D / 8 lanes a
// row (16 bytes of it each), `passes` times 32 / (D / 8) rows a warp: query rows first, then
// the blocks' K and V rows.
template <int D>
__global__ void __launch_bounds__(256) attn_kv8_prep_kernel(const AttnKv8Args a, int grid, int passes) {
  pdl_wait();  // the previous kernel on the stream is complete from here on
  pdl_trigger();
  const int Hkv = a.kv.Hkv, G = a.Hq / Hkv, R = a.K * G, NR = a.row_block;
  if (blockIdx.x == 0) {
    __shared__ int part[256];
    const long max_ctx = (long)a.kv.max_pages * a.kv.page_size;
    const int nbt = a.kb ? 1 : 0, spr = Hkv * a.n_rb;
    int* off = a.sched + 64;
    const int per = (a.C + 255) / 256;
    const int c0 = min(a.C, (int)threadIdx.x * per), c1 = min(a.C, c0 + per);
    int sum = 0;
    for (int c = c0; c < c1; ++c) {
      const int ctx = a.ctx_lens[c];
      if (ctx < 0 || ctx > max_ctx) flag_error(a.err, kErrCtxOOB);
      sum += seq_units(ctx, max_ctx, nbt) * spr;
    }
    part[threadIdx.x] = sum;
    __syncthreads();
    for (int o = 1; o < 256; o <<= 1) {  // inclusive scan of the per-thread sums
      const int v = threadIdx.x >= (unsigned)o ? part[threadIdx.x - o] : 0;
      __syncthreads();
      part[threadIdx.x] += v;
      __syncthreads();
    }
    int run = threadIdx.x > 0 ? part[threadIdx.x - 1] : 0;
    for (int c = c0; c < c1; ++c) {
      off[c] = run;
      run += seq_units(a.ctx_lens[c], max_ctx, nbt) * spr;
    }
    if (threadIdx.x == 255) {
      const int T = part[255];
      int Z = a.chunk_units > 0 ? a.chunk_units : (T + grid - 1) / grid;
      Z = max(max(Z, (T + a.max_chunks - 1) / a.max_chunks), 1);
      off[a.C] = T;
      a.sched[1] = T;
      a.sched[2] = Z;
      a.sched[3] = (T + Z - 1) / Z;
    }
    return;
  }
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, part = lane % LPR;
  const int q_rows = a.C * Hkv * a.n_rb * NR, KP = blk_rows(a.K);
  const int rows = q_rows + (a.kb ? a.C * Hkv * 2 * KP : 0);
  const int w0 = ((blockIdx.x - 1) * 8 + (threadIdx.x >> 5)) * passes * RPW + lane / LPR;
  for (int p = 0; p < passes; ++p) {
    const int w = w0 + p * RPW;
    const bool live = w < rows;
    const bf16* src = nullptr;
    uint8_t* hi = nullptr;
    size_t lo_off = 0;
    float* scale = nullptr;
    int r = 0;
    if (w < q_rows) {
      const int seq = w / NR;  // (c * n_rb + rb) * Hkv + g
      r = w - seq * NR;
      const int cr = seq / Hkv, g = seq - cr * Hkv, c = cr / a.n_rb, rb = cr - c * a.n_rb;
      const int row = rb * NR + r, j = row / G;
      if (row < R) src = (const bf16*)a.q + (size_t)(c * a.K + j) * a.q_rs + (size_t)(g * G + row - j * G) * D;
      hi = a.q_img + (size_t)seq * q_img_bytes(NR, D);
      lo_off = (size_t)NR * D;
      scale = (float*)(hi + 2 * lo_off) + r;
    } else if (live) {
      const int b = w - q_rows, x = b / KP;  // x = (c * Hkv + g) * 2 + is_v
      r = b - x * KP;
      const int is_v = x & 1, cg = x >> 1, c = cg / Hkv, g = cg - c * Hkv;
      if (r < a.K)
        src = (const bf16*)(is_v ? a.vb : a.kb) + (size_t)(c * a.K + r) * (is_v ? a.vb_rs : a.kb_rs) + (size_t)g * D;
      hi = a.blk_img + (size_t)x * 2 * KP * D;
      lo_off = (size_t)KP * D;
      scale = a.blk_scale + x * kBlkRows + r;
    }
    uint4 v = make_uint4(0, 0, 0, 0);
    if (src) v = *(const uint4*)(src + part * 8);
    const uint32_t vs[4] = {v.x, v.y, v.z, v.w};
    float x[8], m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(vs[i] << 16), x[2 * i + 1] = __uint_as_float(vs[i] & 0xFFFF0000u);
      m = fmaxf(m, fmaxf(kv8_mag(x[2 * i]), kv8_mag(x[2 * i + 1])));
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float inv;
    const float f = row_factor(m, inv);
    uint32_t h[2], l[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float y[4] = {x[4 * i] * f, x[4 * i + 1] * f, x[4 * i + 2] * f, x[4 * i + 3] * f};
      split4(y, h[i], l[i]);
    }
    if (live) {
      const uint32_t o = swz<D>(r, part >> 1) + (part & 1) * 8;
      *(uint2*)(hi + o) = make_uint2(h[0], h[1]);
      *(uint2*)(hi + lo_off + o) = make_uint2(l[0], l[1]);
      if (part == 0) *scale = inv;
    }
  }
}

// Order-preserving integer of a float (NaN counts as -infinity) and back.
__device__ __forceinline__ int float_key(float v) {
  const int i = __float_as_int(v == v ? v : -INFINITY);
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float key_float(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7fffffff)); }

// Four weights (fp16: 11 bits, well below the two parts' error) as their e4m3 codes and the
// codes of what those leave, times kLoScale.
__device__ __forceinline__ void split_weights(__half2 p0, __half2 p1, uint32_t& hi, uint32_t& lo) {
  asm("{\n\t.reg .b16 a, b, c, d;\n\t.reg .b32 x, y;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 a, %2;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 b, %3;\n\t"
      "mov.b32 %0, {a, b};\n\t"
      "cvt.rn.f16x2.e4m3x2 x, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 y, b;\n\t"
      "sub.rn.f16x2 x, %2, x;\n\t"
      "sub.rn.f16x2 y, %3, y;\n\t"
      "mul.rn.f16x2 x, x, %4;\n\t"
      "mul.rn.f16x2 y, y, %4;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 c, x;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 d, y;\n\t"
      "mov.b32 %1, {c, d};\n\t}\n"
      : "=&r"(hi), "=&r"(lo)
      : "r"(*reinterpret_cast<uint32_t*>(&p0)), "r"(*reinterpret_cast<uint32_t*>(&p1)), "r"(0x50005000u));
}
static_assert(kLoScale == 32.f, "0x5000 is 32 in fp16");

// One lane of a converged warp (the tensor instructions are issued by it).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ TileMeta load_meta(const TileMeta* m) {
  TileMeta r;
  const uint32_t at = tc::smem_u32(m);
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.flags), "=r"(r.cg), "=r"(r.rb), "=r"(r.slot)
               : "r"(at)
               : "memory");
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.valid), "=r"(r.joff) : "r"(at + 16) : "memory");
  return r;
}

// An item is one tile's work for one side: item 2 n + w is the n-th of side w.
// PAIR = false (up to 64 query rows a sequence): the sides take the tiles in turn, item
// = tile.  PAIR = true (up to 128 rows): each takes one half of the rows of every tile,
// tile = item / 2, so that a tile's bytes serve both halves.
template <int D, int NR, bool PAIR>
__global__ void __launch_bounds__(Warps<NR>::THREADS, 1)
    attn_kv8_tc_kernel(const __grid_constant__ Maps maps, const AttnKv8Args a, float scale_log2, int box_shift) {
  using L = Lay<D, NR, PAIR>;
  constexpr int NS = L::NS, PN = L::PN, CG = Warps<NR>::CG, NC = NR / CG;
  constexpr int NPW = Warps<NR>::NPW, SM_WARP0 = Warps<NR>::SM_WARP0;
  constexpr int kFewRegs = Warps<NR>::kFewRegs, kManyRegs = Warps<NR>::kManyRegs;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = tc::smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023) & ~1023u) - raw);
  uint8_t* sP = smem;
  uint8_t* sQ = smem + L::OFF_Q;
  uint8_t* sKV = smem + L::OFF_KV;
  static_assert(sizeof(Misc<NR>) <= L::MISC, "misc area");
  Misc<NR>& ms = *(Misc<NR>*)(smem + L::OFF_MISC);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int Hkv = a.kv.Hkv, G = a.Hq / Hkv, R = a.K * G;
  const int RB = R < L::ROWS ? R : L::ROWS;  // rows of a partial
  int* const err = a.err;
  const uint64_t lim = a.wait_ns;  // pipeline waits (the launcher puts the default in)
  constexpr int QK_WARP = NPW, PV_WARP = NPW + 1;
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {  // for a whole warp
    return __all_sync(0xffffffffu, tc::mbar_wait_long(bar, parity, a.err, a.wait_ns));
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      tc::mbar_init(&ms.kv_full[s], 18);  // of K's and V's warp one lane and eight scale lanes each
      tc::mbar_init(&ms.kv_empty[s], 1);
    }
    for (int b = 0; b < 4; ++b) {
      tc::mbar_init(&ms.q_full[b], 1);
      tc::mbar_init(&ms.q_empty[b], 1);
      tc::mbar_init(&ms.s_full[b], 2);  // the product's commit and the issuer's own arrival
      tc::mbar_init(&ms.s_free[b], 4 * CG);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&ms.p_full[b], 4 * CG);
      tc::mbar_init(&ms.pv_done[b], 1);
      tc::mbar_init(&ms.drain[b], 1);
    }
    ms.end_item = 0x7fffffff;
    tc::fence_mbar_init();
  }
  if (warp == QK_WARP) tc::tmem_alloc(&ms.tmem, L::TMEM_COLS);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = ms.tmem;
  pdl_wait();  // the previous kernel on the stream is complete from here on
  pdl_trigger();

  if (warp < NPW) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    // ------------------------------------------------------------ producers
    // Warps 0 and 1 bring K and V (with four, of the even tiles, warps 2 and 3 of the odd): lane
    // x < 8 the tile's box x of 2^box_shift rows (within one page each), lane 8 + i the
    // scale of its 16-key group i.  All walk the same tiles; the K warp describes its tile,
    // warp 0 also loads the queries.
    const int pw = warp & 1, pair = warp >> 1;
    const int sub = lane < 8 ? lane << box_shift : 16 * (lane & 7);  // first key of the tile that concerns the lane
    const CUtensorMap* map = pw == 1 ? &maps.v : &maps.k;
    const float* scales = pw == 1 ? a.kv.vs : a.kv.ks;
    const uint32_t scale_at = tc::smem_u32(&ms.scale[0][8 * pw + (lane & 7)]);
    if (threadIdx.x == 0) {
      tc::tma_prefetch_desc(&maps.k);
      tc::tma_prefetch_desc(&maps.v);
    }
    const int spr = Hkv * a.n_rb;  // sequences per request
    const int page = a.kv.page_size;
    const int T = a.sched[1], Z = a.sched[2], n_chunks = a.sched[3];
    const int* off = a.sched + 64;
    // the request holding unit p of the line: the last c with off[c] <= p
    auto locate = [&](int p) -> int {
      int lo = 0, hi = a.C - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (off[mid] <= p) lo = mid;
        else hi = mid - 1;
      }
      return lo;
    };
    const uint64_t once = tc::l2_evict_first();  // the cache is read once
    int k = blockIdx.x;  // this CTA's chunk
    int pos = k < n_chunks ? k * Z : 0, end = k < n_chunks ? min(T, pos + Z) : 0;
    int c = pos < end ? locate(pos) : 0;
    // The next piece: tiles [lt0, lt0 + n) of sequence r of request c within the chunk (a
    // span that holds only a sequence's start units has no tiles and is passed over); n = 0
    // at the end.
    struct Piece {
      int c, r, k, lt0, n, ctx;
    };
    auto advance = [&]() -> Piece {
      Piece q = {0, 0, 0, 0, 0, 0};
      while (q.n == 0) {
        if (pos >= end) {  // the CTA's next chunk
          k += gridDim.x;
          if (k >= n_chunks) return q;
          pos = k * Z;
          end = min(T, pos + Z);
          c = locate(pos);
        }
        while (off[c + 1] <= pos) ++c;
        const int tw = (off[c + 1] - off[c]) / spr;
        const int rel = pos - off[c];
        q.r = rel / tw;
        const int u0 = rel - q.r * tw, u1 = min(tw, u0 + (end - pos));
        pos += u1 - u0;
        q.lt0 = max(u0 - kAttn8SeqUnits, 0);
        q.n = max(u1 - kAttn8SeqUnits - q.lt0, 0);
      }
      q.c = c, q.k = k, q.ctx = a.ctx_lens[c];
      return q;
    };
    const int pshift = (page & (page - 1)) == 0 ? __ffs(page) - 1 : -1;
    auto page_index = [&](int t) -> int { return pshift >= 0 ? t >> pshift : t / page; };
    // Page ids: one load brings the ids of a window of four tiles (at most 32 pages of 16 or
    // more keys), one per lane, a window ahead of its use; the index is clamped into the
    // request's row of the table (ids past the context's end are never used).
    auto window = [&](const Piece& q, int w) -> int {
      const int idx = page_index((q.lt0 + 4 * w) * TT) + lane;
      return a.kv.table[(size_t)q.c * a.kv.max_pages + min(idx, a.kv.max_pages - 1)];
    };
    int tile_i = 0;   // tiles this warp has armed (its arrival on their stage)
    int s = 0, s_par = 1;  // the tile's stage and the parity to wait for
    int q_last = -1;  // warp 0: the last piece whose queries it armed
    bool ok = true;
    // Every producer warp walks the same pieces and passes the same barriers: the loop
    // ends only at one, when the work is done or a producer has given up waiting.
    bool stopped = false;
    Piece next = {0, 0, 0, 0, 1, 0};  // (seq = -1: nothing but the look-ahead)
    int next_ids = 0;
    for (int seq = -1;; ++seq) {
      if (tc::bar_or<1, 32 * NPW>(!ok)) {
        stopped = true;
        break;
      }
      const Piece pc = next;
      if (pc.n == 0) break;
      const int g = pc.r % Hkv, rb = pc.r / Hkv;
      const int ctx = pc.ctx, n_tiles = pc.n;
      const int ct = (ctx + TT - 1) / TT;  // context tiles of the sequence
      const int qslot = seq % L::NQ, quse = seq / L::NQ;

      // the piece's queries into buffer `qslot` once the piece before in it is done
      if (warp == 0 && seq >= 0) {
        if (lane == 0) {
          ok = tc::mbar_wait_long(&ms.q_empty[qslot], (quse & 1) ^ 1, err, lim);
          if (ok) {
            q_last = seq;
            tc::mbar_arrive_expect_tx(&ms.q_full[qslot], (uint32_t)L::Q_BYTES);
            tc::bulk_load(sQ + qslot * L::Q_BUF, a.q_img + ((size_t)pc.c * spr + pc.r) * L::Q_BYTES,
                          (uint32_t)L::Q_BYTES, &ms.q_full[qslot]);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        q_last = __shfl_sync(0xffffffffu, q_last, 0);
      }

      int ids = next_ids, ids_ahead = n_tiles > 4 ? window(pc, 1) : 0, base = page_index(pc.lt0 * TT);
      for (int local = 0; local < n_tiles && ok; ++local) {
        if (local > 0 && (local & 3) == 0) {
          ids = ids_ahead;
          base = page_index((pc.lt0 + local) * TT);
          if (local + 4 < n_tiles) ids_ahead = window(pc, local / 4 + 1);
        }
        if ((NPW == 2 || (tile_i & 1) == pair) && seq >= 0) {  // a tile of this warp's
        const int st = pc.lt0 + local;  // tile of the sequence
        const int t0 = st * TT;
        const bool block = st >= ct;
        const int valid = block ? a.K : min(TT, ctx - t0);
        const int tk = t0 + sub, pidx = page_index(tk);
        int pid = __shfl_sync(0xffffffffu, ids, (pidx - base) & 31);
        const bool in = !block && sub < valid && lane < 16;
        const bool sound = (unsigned)pid < (unsigned)a.kv.num_pages;
        if (in && !sound) flag_error(err, kErrPageOOB);
        if (!sound) pid = 0;  // keep the copy in bounds (its scales are 0 here)
        const int row = pid * Hkv + g;
        ok = wait(&ms.kv_empty[s], s_par);
        if (!ok) break;
        uint8_t* dst = sKV + s * L::STAGE + pw * L::KV;
        if (lane >= 8 && lane < 16) {
          tc::cp_async4(scale_at + s * 64, scales + row, in && sound);
          tc::cp_async_arrive(&ms.kv_full[s]);
        }
        if (pw == 0 && lane == 0) {
          const int joff = !a.causal ? -TT : block ? 0 : a.kb ? -TT : max(t0 - ctx + a.K, -TT);
          constexpr int STEP = PAIR ? 1 : 2;  // tiles between those of one side
          TileMeta m;
          m.flags = (local == 0 ? kFirst : 0) | (local == n_tiles - 1 ? kLast : 0) | (local < STEP ? kGroupFirst : 0) |
                    (local >= n_tiles - STEP ? kGroupLast : 0) | (block ? kBlock : 0) |
                    (joff + valid - 1 > 0 ? kMixed : 0) | (quse & 1 ? kQPar : 0) | (qslot << kQShift) |
                    (local & 1 ? kHalf : 0);
          m.cg = pc.c * Hkv + g, m.rb = rb, m.slot = pc.c * spr + pc.r + pc.k, m.valid = valid, m.joff = joff;
          m.pad[0] = m.pad[1] = 0;
          ms.meta[s] = m;
          if (m.flags & kMixed) ms.v_nan[s] = make_uint4(0, 0, 0, 0);
        }
        if (block) {
          // the block's K or V image: hi rows, then lo rows
          const uint32_t bytes = (uint32_t)(2 * blk_rows(a.K) * D);
          if (lane == 0) {
            tc::mbar_arrive_expect_tx(&ms.kv_full[s], bytes);
            tc::bulk_load(dst, a.blk_img + ((size_t)(pc.c * Hkv + g) * 2 + pw) * bytes, bytes, &ms.kv_full[s]);
          }
        } else {
          const int boxes = (valid + (1 << box_shift) - 1) >> box_shift;
          if (lane == 0) tc::mbar_arrive_expect_tx(&ms.kv_full[s], (uint32_t)((boxes << box_shift) * D));
          __syncwarp();
          if (lane < boxes)
            tc::tma_load_3d_hint(dst + sub * D, map, &ms.kv_full[s], 0, tk - pidx * page, row, once);
        }
        __syncwarp();
        }
        if (seq >= 0) {
          ++tile_i;
          if (++s == NS) s = 0, s_par ^= 1;
        }
        if (local == 0) {  // look ahead while the ring is full
          next = advance();
          next_ids = next.n > 0 ? window(next, 0) : 0;
        }
      }
    }
    // No copy may land after the CTA has finished: wait, with the full limit, for the last
    // filling of every stage this warp armed, and warp 0 for its last query loads.  Before
    // the sentinel below, which completes the next phase of one of these stages.
    if (lane == 0) {
      for (int j = tile_i > NS ? tile_i - NS : 0; j < tile_i; ++j)
        tc::mbar_wait(&ms.kv_full[j % NS], (j / NS) & 1, err);
      for (int q = max(q_last - L::NQ + 1, 0); q <= q_last; ++q)
        tc::mbar_wait(&ms.q_full[q % L::NQ], (q / L::NQ) & 1, err);
    }
    __syncwarp();
    tc::bar_or<1, 32 * NPW>(false);  // (all have seen their stages' last fillings)
    // sentinel stage: no more work
    if (!stopped && pair == 0) {
      if (wait(&ms.kv_empty[s], s_par) && lane < 9) {  // as many arrivals as a tile's
        if (threadIdx.x == 0) ms.meta[s].flags = kEnd;
        tc::mbar_arrive(&ms.kv_full[s]);
      }
    }
  } else if (warp < SM_WARP0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    if (warp == QK_WARP) {
      // ---------------------------------------------------------- S^T issuer
      // S^T_b = K_i . Q^T into S buffer b = item % 4 once tile i has landed, the softmax has
      // read item - 4 out of S_b and the piece's queries are there.  Its own arrival on
      // s_full passes on what it has seen: the tile's description and scales, the queries.
      constexpr uint32_t idesc = tc::idesc_e4m3_f32(TT, NR, false, false);
      const uint32_t lo_part = (uint32_t)(blk_rows(a.K) * D);
      for (int i = 0;; ++i) {
        const int s = i % NS;
        if (!wait(&ms.kv_full[s], (i / NS) & 1)) break;
        const int flags = load_meta(&ms.meta[s]).flags;
        const int it0 = PAIR ? 2 * i : i;
        if (flags & kEnd) {
          // wake both sides: their next items are it0 and it0 + 1
          if (lane == 0) *(volatile int*)&ms.end_item = it0;
          __syncwarp();
          for (int it = it0; it < it0 + 2; ++it) {
            if (it >= 4 && !wait(&ms.s_free[it & 3], ((it >> 2) - 1) & 1)) break;
            if (lane == 0) {
              tc::mbar_arrive(&ms.s_full[it & 3]);
              tc::mbar_arrive(&ms.s_full[it & 3]);
            }
            __syncwarp();
          }
          break;
        }
        const int qslot = flags >> kQShift & 3;
        if ((flags & kFirst) && !wait(&ms.q_full[qslot], flags & kQPar ? 1 : 0)) break;
        bool ok = true;
        const uint64_t q0 = tc::sdesc_b8<D>(tc::smem_u32(sQ + qslot * L::Q_BUF));
        const uint64_t k0 = tc::sdesc_b8<D>(tc::smem_u32(sKV + s * L::STAGE));
        for (int w = 0; w < (PAIR ? 2 : 1) && ok; ++w) {
          const int it = it0 + w, b = it & 3;
          if (it >= 4) ok = wait(&ms.s_free[b], ((it >> 2) - 1) & 1);
          if (!ok) break;
          tc::tc_fence_after();
          if (elect_one()) {
            const uint32_t d = tmem + L::S_COL(b);
            const uint64_t q = q0 + (uint32_t)(w * NR * D / 16);
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk) {
              tc::mma_e4m3(d, k0 + 2 * kk, q + 2 * kk, idesc, kk > 0);
              tc::mma_e4m3(d, k0 + 2 * kk, q + (uint32_t)(L::ROWS * D / 16) + 2 * kk, idesc, 1u);
            }
            if (flags & kBlock) {  // the low parts of K follow its high parts
              const uint64_t kl = k0 + (lo_part >> 4);
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk) {
                tc::mma_e4m3(d, kl + 2 * kk, q + 2 * kk, idesc, 1u);
                tc::mma_e4m3(d, kl + 2 * kk, q + (uint32_t)(L::ROWS * D / 16) + 2 * kk, idesc, 1u);
              }
            }
            tc::mma_commit(&ms.s_full[b]);
            tc::mbar_arrive(&ms.s_full[b]);
          }
          __syncwarp();
        }
        if (!ok) break;
      }
      // no MMA or commit arrival may land after the CTA has finished
      if (elect_one()) tc::mma_commit(&ms.drain[0]);
      __syncwarp();
      tc::mbar_wait(&ms.drain[0], 0, err);
    } else if (warp == PV_WARP) {
      // ---------------------------------------------------------- O^T issuer
      // O^T_w += V_i^T . P^T in steps of 32 keys (V rows past the last key are zero) once the
      // item's P is in shared memory; the commit of a tile's last item frees the K/V stage
      // (its S^T finished before its softmax began).
      constexpr uint32_t idesc = tc::idesc_e4m3_f32(D, PN, true, true);
      const uint32_t lo_part = (uint32_t)(blk_rows(a.K) * D);
      for (int i = 0;; ++i) {
        const int s = i % NS;
        if (!wait(&ms.kv_full[s], (i / NS) & 1)) break;
        const TileMeta m = load_meta(&ms.meta[s]);
        if (m.flags & kEnd) break;
        const uint64_t v0 = tc::sdesc_b8<D>(tc::smem_u32(sKV + s * L::STAGE + L::KV));
        const int steps = (m.valid + 31) / 32;
        bool ok = true;
        for (int j = 0; j < (PAIR ? 2 : 1) && ok; ++j) {
          const int w = PAIR ? j : i & 1, n = PAIR ? i : i >> 1;
          ok = wait(&ms.p_full[w], n & 1);
          if (!ok) break;
          tc::tc_fence_after();
          if (elect_one()) {
            const uint32_t d = tmem + L::O_COL(w);
            const uint64_t p = tc::sdesc_b8<PN>(tc::smem_u32(sP + w * L::P_BUF));
            const uint32_t acc0 = m.flags & kGroupFirst ? 0u : 1u;
#pragma unroll
            for (int kk = 0; kk < TT / 32; ++kk)
              if (kk < steps) tc::mma_e4m3(d, v0 + kk * (32 * D / 16), p + kk * (32 * PN / 16), idesc, kk > 0 ? 1u : acc0);
            if (m.flags & kBlock) {  // the low parts of V follow its high parts
              const uint64_t vl = v0 + (lo_part >> 4);
#pragma unroll
              for (int kk = 0; kk < 2; ++kk)
                if (kk < steps) tc::mma_e4m3(d, vl + kk * (32 * D / 16), p + kk * (32 * PN / 16), idesc, 1u);
            }
            if (!PAIR || j == 1) {
              if (m.flags & kLast) tc::mbar_arrive(&ms.q_empty[m.flags >> kQShift & 3]);
              tc::mma_commit(&ms.kv_empty[s]);
            }
            tc::mma_commit(&ms.pv_done[w]);
          }
          __syncwarp();
        }
        if (!ok) break;
      }
      if (elect_one()) tc::mma_commit(&ms.drain[1]);
      __syncwarp();
      tc::mbar_wait(&ms.drain[1], 0, err);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
    // ------------------------------------------------------------ softmax groups
    // Groups CG w .. take the columns of the items of side w, NC each.  The thread's key is its
    // TMEM lane.  A wait that gave up (ok = false) is acted on only at the group's barriers, so
    // that all four warps leave together.
    const int gq = (warp - SM_WARP0) >> 2, w = gq / CG, quarter = warp & 3;
    const int c0 = gq % CG * NC;  // first column
    const int key = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t t_hi = tmem + lane_off + L::O_COL(w) + c0, t_lo = t_hi + PN / 2;
    float *cqs = ms.cq[gq], *nms = ms.nm[gq];
    float* alpha = ms.alpha[gq];
    auto group_or = [&](bool p) -> bool { return tc::bar_or(2 + gq, 128, p); };
    // rows of row block rb in the group's columns (none: <= 0)
    auto rows_of = [&](int rb) -> int { return min(NC, min(L::ROWS, R - rb * L::ROWS) - (PAIR ? w * NR : 0) - c0); };
    constexpr int CH = NR > 16 && NC % 16 == 0 ? 16 : 8;  // columns at a time
    // Chunks of columns without rows are passed over where they can be a third or more of the
    // columns (8 of 16 columns: 367 us against 379; 68 of 96: 194 and 198).  Where they are less,
    // the test in the unrolled loop costs more than it saves (128 of 128: 372 and 354).
    constexpr bool SKIP = NR == 16 || (PAIR && NR == 48);
    tc::F2 l2[NC / 2];  // this key lane's share of the columns' sums
    float Mv = 0.f, inv_mv = 0.f;  // largest V scale of the piece, 1 / it
    bool ok = true;
    // the previous piece's partial, still in O^T
    bool pend = false;
    // O^T (every product issued into it has finished) to the workspace
    auto write_partial = [&]() {
      tc::tc_fence_after();
      const int d = D == 128 ? key : quarter * 16 + lane;
      const bool on = D == 128 || lane < 16;
      const int pend_base = ms.pend_base[gq], pend_rows = ms.pend_rows[gq];
      const float pend_mul = ms.pend_mul[gq];
#pragma unroll 1
      for (int j0 = 0; j0 < pend_rows; j0 += 8) {
        float hi[8], lo[8];
        tc::tmem_ld(t_hi + j0, hi);
        tc::tmem_ld(t_lo + j0, lo);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (on && j0 + j < pend_rows)
            a.ws_acc[(size_t)(pend_base + j0 + j) * D + d] = fmaf(lo[j], 1.f / kLoScale, hi[j]) * pend_mul;
      }
      pend = false;
    };

    // Exponents e = s - m of CH columns from j0 on: s = S (key scale) (query scale).
    auto exponents = [&](uint32_t t_s, int j0, tc::F2 ck2, int cmin, float (&e)[CH]) {
      tc::tmem_ld(t_s + j0, e);
#pragma unroll
      for (int j = 0; j < CH; j += 4) {
        const ulonglong2 q = *(const ulonglong2*)&cqs[j0 + j], nm = *(const ulonglong2*)&nms[j0 + j];
        tc::f2_get(tc::f2_fma(tc::f2_mul(tc::f2(e[j], e[j + 1]), ck2), q.x, nm.x), e[j], e[j + 1]);
        tc::f2_get(tc::f2_fma(tc::f2_mul(tc::f2(e[j + 2], e[j + 3]), ck2), q.y, nm.y), e[j + 2], e[j + 3]);
      }
      if (cmin > j0) {
#pragma unroll
        for (int j = 0; j < CH; ++j)
          if (j0 + j < cmin) e[j] = -INFINITY;
      }
    };
    // The key's weights 2^e, times `add` added to the sums, and stored in two parts, times rv,
    // as its row of P.  `over` becomes the largest of them.
    float over = 0.f;
    auto weigh = [&](uint32_t t_s, float ck, float rv, int cmin, int cols, float add) {
      const tc::F2 ck2 = tc::f2(ck, ck), rv2 = tc::f2(rv, rv), add2 = tc::f2(add, add);
      uint8_t* prow = sP + w * L::P_BUF;
      float top[2] = {0.f, 0.f};
#pragma unroll
      for (int j0 = 0; j0 < NC; j0 += CH) {
        if (j0 >= cols) break;
        float e[CH];
        exponents(t_s, j0, ck2, cmin, e);
        uint32_t hi[CH / 4], lo[CH / 4];
#pragma unroll
        for (int q = 0; q < CH / 4; ++q) {
          __half2 ph[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int j = 4 * q + 2 * k;
            const float x = tc::ex2_ftz(e[j]), y = tc::ex2_ftz(e[j + 1]);
            top[k] = fmaxf(fmaxf(top[k], x), y);
            const tc::F2 p = tc::f2(x, y);
            l2[(j0 + j) / 2] = tc::f2_fma(p, add2, l2[(j0 + j) / 2]);
            float u, v;
            tc::f2_get(tc::f2_mul(p, rv2), u, v);
            ph[k] = __floats2half2_rn(u, v);
          }
          split_weights(ph[0], ph[1], hi[q], lo[q]);
        }
        // byte c0 + j0 of the row's high half, and of its low half PN / 2 bytes on
        const int ch = (c0 + j0) / 16;
        if constexpr (CH == 16) {
          *(uint4*)(prow + swz<PN>(key, ch)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *(uint4*)(prow + swz<PN>(key, PN / 32 + ch)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        } else {
          const int in = (c0 + j0) & 8;
          *(uint2*)(prow + swz<PN>(key, ch) + in) = make_uint2(hi[0], hi[1]);
          *(uint2*)(prow + swz<PN>(key, PN / 32 + ch) + in) = make_uint2(lo[0], lo[1]);
        }
      }
      over = fmaxf(top[0], top[1]);
    };
    int n = 0;      // items of the side so far
    int s = PAIR ? 0 : w;  // the item's stage
    for (;; ++n) {
      const int it = 2 * n + w, b = it & 3;
      if (ok) ok = wait(&ms.s_full[b], (it >> 2) & 1);
      const bool run = ok && it < *(volatile int*)&ms.end_item;
      TileMeta m = {};
      int cmin = 0, cols = NC;  // cols: the group's columns that are worked on, whole chunks
      bool first = false;
      float ck = 0.f, sv = 0.f;
      const uint32_t t_s = tmem + lane_off + L::S_COL(b) + c0;
      if (run) {
        tc::tc_fence_after();
        m = load_meta(&ms.meta[s]);
        first = (m.flags & kGroupFirst) != 0;
        if (key < m.valid) {
          if (m.flags & kBlock) {
            const float* bs = a.blk_scale + (size_t)m.cg * 2 * kBlkRows;
            ck = bs[key], sv = bs[kBlkRows + key];
          } else {
            ck = ms.scale[s][key >> 4], sv = ms.scale[s][8 + (key >> 4)];
          }
        }
        ck *= scale_log2;
        // columns below cmin do not see this key (row = rb ROWS + column, position row / G)
        cmin = key >= m.valid ? NC : max(m.joff + key, 0) * G - m.rb * L::ROWS - (PAIR ? w * NR : 0) - c0;
        cols = SKIP ? min(NC, (rows_of(m.rb) + CH - 1) & -CH) : NC;
      }
      // The weights are 2^(s - reference), under the references so far; only if one exceeds
      // kOver (or a V scale the largest so far) do the references rise to the maxima and the
      // tile's weights get computed again.  A piece's first tile has no references yet.  Where
      // the references are looked at, one far over the tile's own maximum comes down: weights far
      // below it have few bits in P.  The side's last product must be done: its P buffer is free
      // then, and O^T complete.
      if (ok && n > 0) ok = wait(&ms.pv_done[w], (n - 1) & 1);
      if (ok && pend) write_partial();  // (before this item's product may overwrite it)
      const bool forced = first || n == ms.look[gq];
      bool weighed = false, moved = false, leave = false;
      while (true) {
        if (run && ok && (moved || !forced)) {
          // (after a rise the sums hold the tile's weights already: under the old references,
          // and alpha has brought them to the new ones)
          weigh(t_s, ck, sv * inv_mv * kPScale, cmin, cols, weighed ? 0.f : 1.f);
          weighed = true;
        }
        if (!group_or(!run || !ok || (!moved && (forced || over > kOver || sv > Mv)))) break;
        // The references move (or the group leaves).
        const float* cq = (const float*)(sQ + (m.flags >> kQShift & 3) * L::Q_BUF + 2 * L::ROWS * D) +
                          (PAIR ? w * NR : 0) + c0;  // the queries' scales (in place during a first tile)
        if (run && ok) {
#pragma unroll 1
          for (int j0 = 0; j0 < cols; j0 += 8) {
            float v[8];
            tc::tmem_ld(t_s + j0, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float x = j0 + j < cmin ? -INFINITY : v[j] * ck * (first ? cq[j0 + j] : cqs[j0 + j]);
              const int top = __reduce_max_sync(0xffffffffu, float_key(x));
              if (lane == j) ms.cmax[gq][quarter][j0 + j] = key_float(top);
            }
          }
          const float t = warp_max(sv);
          if (lane == 0) ms.svmax[gq][quarter] = t;
        }
        if (group_or(!run || !ok)) {
          leave = true;
          break;
        }
        if (quarter == 0) {
          bool far = first;
          for (int j = lane; j < cols; j += 32) {
            const float cm =
                fmaxf(fmaxf(ms.cmax[gq][0][j], ms.cmax[gq][1][j]), fmaxf(ms.cmax[gq][2][j], ms.cmax[gq][3][j]));
            const float m_old = first ? -INFINITY : ms.m[gq][j], top = first ? cm : fmaxf(ms.top[gq][j], cm);
            float m_new = fmaxf(m_old, cm);
            if (forced && cm > -INFINITY) m_new = fmaxf(fmaxf(cm, fminf(m_old, cm + kSlack)), top - kBelow);
            const bool up = first || m_new - ms.base[gq][j] > kFar;
            if (up || forced) ms.base[gq][j] = m_new;
            far = far || up;
            ms.m[gq][j] = m_new;
            ms.top[gq][j] = top;
            if (first) cqs[j] = cq[j];
            nms[j] = m_new == -INFINITY ? 0.f : -m_new;
            alpha[j] = m_old == -INFINITY ? 1.f : exp2f(m_old - m_new);
          }
          far = __any_sync(0xffffffffu, far);
          if (lane == 0 && (far || forced)) {
            ms.gap[gq] = first ? kSettle / 4 : far ? 1 : min(ms.gap[gq] * 4, kSettle);
            ms.look[gq] = n + (far ? 1 : ms.gap[gq]);
          }
        }
        const float sv_top = fmaxf(fmaxf(ms.svmax[gq][0], ms.svmax[gq][1]), fmaxf(ms.svmax[gq][2], ms.svmax[gq][3]));
        // (at least the smallest normal number: its inverse is finite)
        const float mv_new = fmaxf(first ? sv_top : fmaxf(Mv, sv_top), 1.17549435e-38f);
        const float mv_ratio = Mv / mv_new;
        Mv = mv_new;
        inv_mv = 1.f / Mv;
        group_or(false);  // cq, nm, m, alpha and look are written
        if (first) {
#pragma unroll
          for (int j = 0; j < NC / 2; ++j) l2[j] = 0;
        } else {
#pragma unroll
          for (int j = 0; j < NC / 2; ++j) {
            float x, y;
            tc::f2_get(l2[j], x, y);
            l2[j] = tc::f2(x == INFINITY ? x : x * alpha[2 * j], y == INFINITY ? y : y * alpha[2 * j + 1]);
          }
          // O^T holds the side's earlier tiles of the piece
          tc::tc_fence_after();
#pragma unroll 1
          for (int j0 = 0; j0 < cols; j0 += 8) {
            float o[8], p[8];
            tc::tmem_ld(t_hi + j0, o);
            tc::tmem_ld(t_lo + j0, p);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float f = alpha[j0 + j] * mv_ratio;
              o[j] *= f, p[j] *= f;
            }
            tc::tmem_st8(t_hi + j0, o);
            tc::tmem_st8(t_lo + j0, p);
          }
        }
        moved = true;
      }
      if (leave) break;
      if (moved && !forced) {
        // a weight that overflowed under the old reference is what its sum comes to now
        bool lost = false;
#pragma unroll
        for (int j = 0; j < NC / 2; ++j) {
          float x, y;
          tc::f2_get(l2[j], x, y);
          lost = lost || x == INFINITY || y == INFINITY;
        }
        if (__any_sync(0xffffffffu, lost)) {
          const tc::F2 ck2 = tc::f2(ck, ck);
#pragma unroll
          for (int j0 = 0; j0 < NC; j0 += CH) {
            float e[CH];
            exponents(t_s, j0, ck2, cmin, e);
#pragma unroll
            for (int j = 0; j < CH; j += 2) {
              float x, y;
              tc::f2_get(l2[(j0 + j) / 2], x, y);
              if (x == INFINITY) x = tc::ex2_ftz(e[j]);
              if (y == INFINITY) y = tc::ex2_ftz(e[j + 1]);
              l2[(j0 + j) / 2] = tc::f2(x, y);
            }
          }
        }
      }
      // From here on nothing waits: the item is complete.
      // S is read
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&ms.s_free[b]);
      // A thread walks its V row from chunk `lane` on: the lanes' rows share their banks (32 requests
      // verifying 17 positions: 172 us, 193 with all from chunk 0 on).
      uint8_t* v_row = sKV + s * L::STAGE + L::KV + key * D;
      auto chunk = [&](int q) -> uint4* { return (uint4*)(v_row + ((q + lane) & (D / 16 - 1)) * 16); };
      if (m.flags & kMixed) {
        // a NaN in a V row that some column does not see: the product would carry it into
        // that column, too, so the row is cleared and the columns that see it get a NaN sum.
        // Another group may have cleared the row already, and has then marked it before.
        bool bad = false;
        if (key < m.valid)
          for (int h = 0; h < (m.flags & kBlock ? 2 : 1); ++h)
#pragma unroll 1
            for (int q = 0; q < D / 16; ++q) {
              const uint4 x = chunk(q)[h * blk_rows(a.K) * (D / 16)];
              const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int z = 0; z < 4; ++z) bad = bad || __vcmpeq4(xs[z] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
            }
        volatile uint32_t* mark = &ms.v_nan[s].x + quarter;
        if (bad) atomicOr((uint32_t*)mark, 1u << lane);
        __threadfence_block();
        bad = bad || (*mark >> lane & 1) != 0;
        if (bad) {
          for (int h = 0; h < (m.flags & kBlock ? 2 : 1); ++h)
#pragma unroll 1
            for (int q = 0; q < D / 16; ++q)
              chunk(q)[h * blk_rows(a.K) * (D / 16)] = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int j = 0; j < NC; j += 2) {
            float x, y;
            tc::f2_get(l2[j / 2], x, y);
            if (j >= cmin) x = __int_as_float(0x7fffffff);
            if (j + 1 >= cmin) y = __int_as_float(0x7fffffff);
            l2[j / 2] = tc::f2(x, y);
          }
        }
      }
      // V rows past the last key may hold anything (their weights are 0): clear them
      if (!(m.flags & kBlock) && key >= m.valid && key < ((m.valid + 31) & ~31)) {
#pragma unroll 1
        for (int q = 0; q < D / 16; ++q) *chunk(q) = make_uint4(0, 0, 0, 0);
      }
      tc::fence_proxy_async();
      tc::tc_fence_before();
      __syncwarp();
      if (ok && lane == 0) tc::mbar_arrive(&ms.p_full[w]);

      if (m.flags & kGroupLast) {
        // the side's part of the piece is complete: its sums now, its O^T during the next
        // item
        const int rows = rows_of(m.rb);
        const int base = (PAIR ? m.slot * RB + w * NR : (m.slot * 2 + (m.flags & kHalf ? 1 : 0)) * RB) + c0;
        // l summed over the lanes: while the count is even, a lane keeps one half of the
        // columns and hands the other half to its partner
        float l[NC];
#pragma unroll
        for (int j = 0; j < NC; j += 2) tc::f2_get(l2[j / 2], l[j], l[j + 1]);
        int cnt = NC, cc = 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const bool up = (lane & o) != 0;
          if (cnt % 2 == 0) {
            cnt /= 2;
#pragma unroll
            for (int j = 0; j < NC / 2; ++j)
              if (j < cnt) {
                const float give = up ? l[j] : l[j + cnt], keep = up ? l[j + cnt] : l[j];
                l[j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
              }
            cc += up ? cnt : 0;
          } else {
#pragma unroll
            for (int j = 0; j < NC / 2; ++j)
              if (j < cnt) l[j] += __shfl_xor_sync(0xffffffffu, l[j], o);
          }
        }
#pragma unroll
        for (int j = 0; j < NC / 2; ++j)
          if (j < cnt) ms.cmax[gq][quarter][cc + j] = l[j];
        group_or(false);
        if (quarter == 0)
          for (int j = lane; j < rows; j += 32) {
            float* ml = a.ws_ml + (size_t)(base + j) * 2;
            ml[0] = ms.m[gq][j];
            ml[1] = (ms.cmax[gq][0][j] + ms.cmax[gq][1][j]) + (ms.cmax[gq][2][j] + ms.cmax[gq][3][j]);
          }
        if (quarter == 0 && lane == 0)
          ms.pend_base[gq] = base, ms.pend_rows[gq] = rows, ms.pend_mul[gq] = Mv * (1.f / kPScale);
        group_or(false);  // cmax and m may be written again, the partial's place is there
        pend = true;
      }
      s += PAIR ? 1 : 2;
      if (s >= NS) s -= NS;
    }
    tc::tc_fence_before();
  }
  __syncthreads();
  if (warp == QK_WARP) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, L::TMEM_COLS);
  }
}

// Merges a sequence's partials: W warps share a row, or (W = 1) a warp takes U = 4 rows, of one
// sequence (request c, row block rb, kv head g).  The sequence holds t_seq tiles from unit s0 of
// the line, which is cut into chunks of Z units; its piece in chunk k0 + p has slot c * spr + rb *
// Hkv + g + k0 + p with one partial (pair) or two, q = 2 p + half: half h holds the piece's tiles
// of parity h and exists iff the piece has more than h tiles.  o = sum 2^(m_q - M) acc_q / sum
// 2^(m_q - M) l_q in a fixed order; a lane holds four dims, and the loads of several partials
// are in flight together.  Four rows a warp find their sequence once: 16384 rows of two partials
// 12.7 us, 14.2 with a warp a row.
template <int W>
struct MergeRows {
  static constexpr int U = W == 1 ? 4 : 1;    // rows a warp
  static constexpr int CTA = 8 / W * U;       // rows a CTA
};
template <int D, int W>
__global__ void __launch_bounds__(256) attn_kv8_merge_tc_kernel(const AttnKv8Args a, int blocks) {
  pdl_wait();  // the previous kernel on the stream is complete from here on
  pdl_trigger();
  constexpr int U = MergeRows<W>::U, P = W == 1 ? 2 : 4;  // P partials of a row in flight
  __shared__ float s_acc[W > 1 ? 8 : 1][D];
  __shared__ float2 s_ml[8];
  const int Hkv = a.kv.Hkv, G = a.Hq / Hkv, R = a.K * G, spr = Hkv * a.n_rb;
  const int wib = threadIdx.x >> 5, lane = threadIdx.x & 31, wq = wib % W;
  const int seq = blockIdx.x / blocks, c = seq / spr, r = seq - c * spr, rb = r / Hkv, g = r - rb * Hkv;
  const int rr = (blockIdx.x - seq * blocks) * MergeRows<W>::CTA + wib / W * U;  // first row, of the block
  const int RB = min(R, a.row_block), row0 = rb * a.row_block + rr;
  const int live = min(U, min(a.row_block - rr, R - row0));  // rows there are (none: <= 0)
  const int halves = a.pair ? 1 : 2;
  const int* off = a.sched + 64;
  const int Z = a.sched[2], o0 = off[c], tw = (off[c + 1] - o0) / spr;  // tw = 0: no tiles (or a bad length)
  const int t_seq = tw - kAttn8SeqUnits, s0 = o0 + r * tw + kAttn8SeqUnits, k0 = s0 / Z;
  const int ns = live > 0 && t_seq > 0 ? halves * ((s0 + t_seq - 1) / Z - k0 + 1) : 0;
  const size_t base = (size_t)(seq + k0) * halves * RB + rr;
  const bool on = lane * 4 < D;
  float M[U], L[U];
  float4 o[U];
#pragma unroll
  for (int i = 0; i < U; ++i) M[i] = -INFINITY, L[i] = 0.f, o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto fold = [&](int i, float2 ml, float4 x) {
    if (ml.y == 0.f) return;  // no key seen
    const float mn = fmaxf(M[i], ml.x);
    const float sc = L[i] == 0.f ? 0.f : exp2f(M[i] - mn), w = exp2f(ml.x - mn);
    L[i] = L[i] * sc + ml.y * w;
    o[i].x = o[i].x * sc + x.x * w, o[i].y = o[i].y * sc + x.y * w;
    o[i].z = o[i].z * sc + x.z * w, o[i].w = o[i].w * sc + x.w * w;
    M[i] = mn;
  };
  for (int q0 = wq; q0 < ns; q0 += P * W) {
    float2 ml[P][U];
    float4 x[P][U];
#pragma unroll
    for (int u = 0; u < P; ++u) {
      const int q = q0 + u * W;
      bool has = q < ns;
      if (halves == 2 && has) {
        const int lo = max(s0, (k0 + (q >> 1)) * Z), hi = min(s0 + t_seq, (k0 + (q >> 1) + 1) * Z);
        has = hi - lo > (q & 1);
      }
      const size_t b = base + (size_t)q * RB;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const bool there = has && i < live;
        ml[u][i] = there ? *(const float2*)(a.ws_ml + (b + i) * 2) : make_float2(-INFINITY, 0.f);
        x[u][i] = there && on ? *(const float4*)(a.ws_acc + (b + i) * D + lane * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
#pragma unroll
    for (int u = 0; u < P; ++u)
#pragma unroll
      for (int i = 0; i < U; ++i) fold(i, ml[u][i], x[u][i]);
  }
  if constexpr (W > 1) {
    if (on) *(float4*)&s_acc[wib][lane * 4] = o[0];
    if (lane == 0) s_ml[wib] = make_float2(M[0], L[0]);
    __syncthreads();
    if (wq != 0) return;
    for (int w = 1; w < W; ++w) fold(0, s_ml[wib + w], on ? *(const float4*)&s_acc[wib + w][lane * 4] : o[0]);
  }
  if (!on) return;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if (i >= live) return;
    const int row = row0 + i, j = row / G;
    bf16* out = (bf16*)a.out + (size_t)(c * a.K + j) * a.o_rs + (size_t)(g * G + row - j * G) * D + lane * 4;
    const float inv = L[i] == 0.f ? 0.f : 1.f / L[i];
    const __nv_bfloat162 y = __floats2bfloat162_rn(o[i].x * inv, o[i].y * inv),
                         z = __floats2bfloat162_rn(o[i].z * inv, o[i].w * inv);
    *(uint2*)out = make_uint2(*reinterpret_cast<const uint32_t*>(&y), *reinterpret_cast<const uint32_t*>(&z));
  }
}

// ------------------------------------------------------------------ host side

template <int D, int W>
void launch_merge_w(const AttnKv8Args& a, cudaStream_t s) {
  const int R = a.K * (a.Hq / a.kv.Hkv), rows = R < a.row_block ? R : a.row_block;
  const int blocks = cdiv(rows, MergeRows<W>::CTA);
  launch_pdl_on(attn_kv8_merge_tc_kernel<D, W>, (unsigned)(a.C * a.kv.Hkv * a.n_rb * blocks), 256, 0, s, a, blocks);
  note_launch();
}

template <int D>
void launch_merge(const AttnKv8Args& a, cudaStream_t s) {
  // warps per output row: enough warps in all for about 32 per SM
  const long rows = (long)a.C * a.K * a.Hq;
  if (rows >= 148L * 32) launch_merge_w<D, 1>(a, s);
  else if (rows * 2 >= 148L * 32) launch_merge_w<D, 2>(a, s);
  else if (rows * 4 >= 148L * 32) launch_merge_w<D, 4>(a, s);
  else launch_merge_w<D, 8>(a, s);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return (EncodeTiledFn)p;
  }();
  return fn;
}

// Codes [num_pages * Hkv][page_size][D] bytes, box of box_rows rows of one page and head,
// swizzled over D bytes.
bool make_map(CUtensorMap* m, const Kv8& kv, const uint8_t* base, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)kv.D, (cuuint64_t)kv.page_size, (cuuint64_t)kv.num_pages * kv.Hkv};
  cuuint64_t strides[2] = {(cuuint64_t)kv.D, (cuuint64_t)kv.D * kv.page_size};
  cuuint32_t box[3] = {(cuuint32_t)kv.D, (cuuint32_t)box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, kv.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NR, bool PAIR>
bool launch(const AttnKv8Args& a, int grid, cudaStream_t s) {
  using L = Lay<D, NR, PAIR>;
  auto kernel = attn_kv8_tc_kernel<D, NR, PAIR>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM) != cudaSuccess) {
    set_error("cudaFuncSetAttribute(attn_kv8_tc_kernel) failed");
    return false;
  }
  int box_shift = 4;  // boxes of the largest power of two of rows that divides the page, up to a tile
  while ((1 << box_shift) < TT && a.kv.page_size % (2 << box_shift) == 0) ++box_shift;
  Maps maps;
  if (!make_map(&maps.k, a.kv, a.kv.k, 1 << box_shift) || !make_map(&maps.v, a.kv, a.kv.v, 1 << box_shift)) {
    set_error("cuTensorMapEncodeTiled failed for the 8-bit cache");
    return false;
  }
  const float scale_log2 = 1.4426950408889634f / sqrtf((float)D);
  launch_pdl_on(kernel, grid, Warps<NR>::THREADS, L::SMEM, s, maps, a, scale_log2, box_shift);
  note_launch();
  return true;
}

template <int D>
bool launch_d(const AttnKv8Args& a, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int grid = min(sms > 0 ? sms : 148, kMaxChunksAuto);
  const long rows = (long)a.C * a.kv.Hkv * a.n_rb * a.row_block + (a.kb ? (long)a.C * a.kv.Hkv * 2 * blk_rows(a.K) : 0);
  // rows a CTA in one pass; four passes once that still fills the GPU
  const long per = 8 * (32 / (D / 8));
  const int passes = rows >= per * 4 * 4 * sms ? 4 : 1;
  launch_pdl(attn_kv8_prep_kernel<D>, 1 + (unsigned)((rows + per * passes - 1) / (per * passes)), 256, 0, s, a, grid,
             passes);
  note_launch();
  bool ok;
  if (a.pair) ok = a.row_block == 96 ? launch<D, 48, true>(a, grid, s) : launch<D, 64, true>(a, grid, s);
  else if (a.row_block == 16) ok = launch<D, 16, false>(a, grid, s);
  else if (a.row_block == 32) ok = launch<D, 32, false>(a, grid, s);
  else if (a.row_block == 48) ok = launch<D, 48, false>(a, grid, s);
  else ok = launch<D, 64, false>(a, grid, s);
  if (ok) launch_merge<D>(a, s);
  return ok;
}

}  // namespace

// The pages must hold whole 16-key groups (one TMA box and one scale each); the rows are
// one swizzle width.
bool attn_kv8_tc_shape(int dtype, int D, int page_size) {
  return dtype == HSPEC_DTYPE_BF16 && (D == 64 || D == 128) && page_size % 16 == 0;
}

size_t attn_kv8_tc_plan(AttnKv8Args& a, int split_req, void* ws) {
  const int D = a.kv.D, Hkv = a.kv.Hkv, R = a.K * (a.Hq / Hkv);
  // The columns of a side in 16s: the tensor time, the exponentials and the registers all go
  // by them.  Up to 64 rows the sides take the tiles in turn; more rows are two halves of up to
  // 64 that the sides take from every tile, in blocks of 128 (64 rows as two halves of 32: 922
  // us against 828 at 128 requests of 16 positions).
  a.pair = R > 64;
  a.n_rb = cdiv(R, 128);
  a.row_block = a.pair ? 32 * cdiv(cdiv(R, a.n_rb), 32) : 16 * cdiv(R, 16);
  a.chunk_units = split_req > 0 ? cdiv(split_req, TT) : 0;
  a.max_chunks = a.chunk_units > 0 ? kMaxChunksExplicit : kMaxChunksAuto;
  const size_t seqs = (size_t)a.C * Hkv * a.n_rb;
  const size_t rows = (seqs + a.max_chunks) * (a.pair ? 1 : 2) * (R < a.row_block ? R : a.row_block);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    uint8_t* p = (uint8_t*)ws + off;
    off += (bytes + 255) & ~(size_t)255;
    return p;
  };
  uint8_t* acc = take(rows * D * 4);
  uint8_t* ml = take(rows * 8);
  uint8_t* sched = take((64 + (size_t)a.C + 1) * 4);
  uint8_t* qi = take(seqs * q_img_bytes(a.row_block, D));
  uint8_t* bi = take((size_t)a.C * Hkv * 4 * blk_rows(a.K) * D);
  uint8_t* bs = take((size_t)a.C * Hkv * 2 * kBlkRows * 4);
  if (ws) {
    a.ws_acc = (float*)acc, a.ws_ml = (float*)ml, a.sched = (int*)sched;
    a.q_img = qi, a.blk_img = bi, a.blk_scale = (float*)bs;
  }
  return off;
}

bool attn_kv8_tc_fits(int C, int K, int Hq, const Kv8& kv, int split_req, const char** why) {
  AttnKv8Args a = {};
  a.kv = kv, a.C = C, a.K = K, a.Hq = Hq;
  attn_kv8_tc_plan(a, split_req, nullptr);
  const double most = 2147483647.0, seqs = (double)C * kv.Hkv * a.n_rb;
  // the line is indexed in 32 bits, with room for a chunk more
  const long tiles = ((long)kv.max_pages * kv.page_size + TT - 1) / TT + 1;
  if (seqs * (tiles + kAttn8SeqUnits) >= (double)(1 << 30))
    return *why = "C * Hkv * blocks of 128 query rows * (table tokens / 128 + 5) must be below 2^30", false;
  if ((double)kv.num_pages * kv.Hkv > most) return *why = "num_pages * Hkv must be below 2^31", false;
  if ((double)C * kv.Hkv * (a.n_rb * a.row_block + 2.0 * blk_rows(K)) > most || (double)C * K * Hq > most ||
      (seqs + a.max_chunks) * 2 * a.row_block > most)
    return *why = "the query rows of the call must be below 2^30", false;
  return true;
}

bool attn_kv8_tc_launch(AttnKv8Args& a, cudaStream_t s) {
  if (a.wait_ns == 0) a.wait_ns = tc::kWaitLimitNs;
  return a.kv.D == 128 ? launch_d<128>(a, s) : launch_d<64>(a, s);
}

}  // namespace hspec
