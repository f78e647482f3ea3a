// sfa_paged_attend_tc.cu — attention of new tokens over the paged cache on the
// 5th-generation tensor cores (bf16).
//
// A CTA walks its run of key tiles (sfa_paged.cuh) with eleven warps:
//   warps 8, 10  loads: q by one tensor copy per 64 columns, keys (8) and values
//                (10) page by page into a ring of 128-key buffers;
//   warp 9       issues the products: S = Q K^T (both operands in shared memory,
//                K-major), O += P V (P in tensor memory, V MN-major);
//   warps 0-3    the softmax of stream 0, a thread per row;
//   warps 4-7    the softmax of stream 1.
// With more rows than one 128-row tile (PAIR) the streams are two row tiles that
// share every key and value tile; with fewer they take the key tiles of one row
// tile in turn (or the halves of an only one), each with its own maximum, sum and
// output, which are joined in tensor memory at the end.  Rows are (node, query head of the group), so that
// one KV head's tile serves all of its query heads.
//
// Scores, P and their products go by steps: a whole tile with PAIR, where the
// other stream's products fill the time of a softmax, and half a tile without,
// so that a stream's products of one half run under the softmax of its other.
// P overwrites the scores that it came from.  A product with q in shared memory
// costs about as much for 64 keys as for 128 (it reads all of q), so PAIR, bound
// by the tensor cores and the softmax together, loses by half steps what it gains
// in overlap: 221 against 201 us (37 sequences of 8,192 tokens, 36 new ones
// each); 64 keys of a row per thread with two threads a row took 260 us where the
// present form, then with P in one part, took 160.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "sfa_paged.cuh"
#include "sfa_umma.cuh"

namespace sfa {
namespace {

constexpr int kTcThreads = 384;  // warp 11 only fills the last group of four
// Registers of a thread after the split: 256 x 208 + 128 x 80 = 63,488, within
// the 384 x 168 = 64,512 of the launch.
constexpr int kTcSoftmaxRegs = 208;
constexpr int kTcOtherRegs = 80;
constexpr int kTcSoftmaxThreads = 256;
constexpr int kTcKeyWarp = 8;
constexpr int kTcMmaWarp = 9;
constexpr int kTcValueWarp = 10;
constexpr int kTcKeys = 128;     // keys of a tile
constexpr int kTcRows = 128;     // rows of a row tile (tensor-memory lanes)
constexpr uint32_t kTmemCols = 512;
constexpr unsigned kTcPollLimit = kAttendPollLimit;
constexpr float kRescaleLog2 = 8.0f;  // the maximum moves only when it grows by more than this (log2)

// Shared memory: q (one row tile, or two), then the ring; all blocks
// [64 columns][128 rows][128 bytes], 128-byte swizzled.
template <int D, bool PAIR>
struct TcPlan {
  static constexpr int tile = kTcKeys * D * 2;          // a key, value or q tile
  static constexpr int q = 0;
  static constexpr int ring = (PAIR ? 2 : 1) * tile;
  static constexpr int stages = D == 128 ? (PAIR ? 5 : 6) : (PAIR ? 11 : 12);
  static constexpr int shared = ring + stages * tile;   // TcShared
  // Keys of a step: scores, P and their products go by steps, each with its
  // own columns of tensor memory.
  static constexpr int step = PAIR ? 128 : 64;
  static constexpr int steps = kTcKeys / step;
};

struct TcMaps {
  CUtensorMap q, k, v;
};

struct TcBars {
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[12], kv_empty[12];
  uint64_t s_full[2][2], p_full[2][2];  // [stream][step]
  uint64_t o_step[2];                   // a step is added to the stream's output
  uint64_t o_done[2], drain;            // the piece's last one (PAIR: of each stream, else of both)
};

struct TcShared {
  TcBars bars;
  float2 ml[2][kTcRows];  // maximum and sum of both streams' rows
  int bad[2][2];          // [piece & 1][stream]: clean_values found elements that are not finite
  unsigned kv_fills[12], q_fills[2];  // copies issued into every buffer, for an exit after a wait that ran out
  uint32_t tmem;
};

// Shared-memory matrix descriptor with 128-byte swizzle.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr, unsigned lbo, unsigned sbo) {
  uint64_t d = static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// D[tmem] (+)= A[tmem] * B[smem]; issued by one thread.
__device__ __forceinline__ void umma_bf16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t b, uint32_t idesc,
                                             bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(tmem_d), "r"(tmem_a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}

// 32 columns of this thread's lane, without waiting: tmem_ld_wait() before use.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]),
        "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]),
        "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}

template <int N>
__device__ __forceinline__ void tmem_ld_wait(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));  // no use before the wait
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};"
      ::"r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
      "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]),
      "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31]),
      "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// True in one lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// Two fp32 operations in one instruction, and a maximum of three (NaN if
// one of them is).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// P of N scores into tensor memory; returns its sum in 32 bits.  The tensor cores
// take bf16.  One bf16 number would put each weight off by up to 2^-8 of itself and
// add as much to a result as its own rounding does, so P is two, for two products:
// its upper half word H and the rest P - H (1 - 2^-22) (N / 2 columns each).  The
// rest is at most 2^-7 of a weight and rounded, so that both together are within
// 2^-15 of it.  Neither is negative, and the rest is above zero wherever P is: an
// infinite value that a row sees stays one in the sum of its products.
// Measured for a second with two parts and with one: 256 sequences of 1,024 to 4,096
// tokens 231 and 209 us, a tree of 64 over 65,500 tokens 109 and 88, chunks of
// 2,048 tokens 236 and 186; errors against 64 bits (2-norm) 1.7e-3, which is the
// result's rounding, and 2.1 to 2.3e-3.
template <int N>
__device__ __forceinline__ float store_probs(float* x, float scale, float base, uint32_t taddr) {
  const float2 sc = make_float2(scale, scale), nb = make_float2(-base, -base);
  const float2 less = make_float2(-(1.0f - 0x1p-22f), -(1.0f - 0x1p-22f));
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int c = 0; c < N; c += 64) {
    uint32_t w[32], rest[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const float2 e = fma2(make_float2(x[c + 2 * j], x[c + 2 * j + 1]), sc, nb);
      const float2 y = make_float2(exp2_approx(e.x), exp2_approx(e.y));
      sum[j & 1] = add2(sum[j & 1], y);
      w[j] = __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x7632);
      const float2 lo = fma2(make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u)), less, y);
      const __nv_bfloat162 r = __floats2bfloat162_rn(lo.x, lo.y);
      rest[j] = *reinterpret_cast<const uint32_t*>(&r);
    }
    tmem_st32(taddr + c / 2, w);
    tmem_st32(taddr + N / 2 + c / 2, rest);
  }
  return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

// Visibility of N keys from slot `slot` on to one row: those below `end`, and
// of the new tokens those of the row's mask words (tree).  The words are loaded
// before the scores are waited for.
template <int N>
struct RowMask {
  uint32_t w[N / 32 + 1];
  int end, shift;
};

template <int N>
__device__ __forceinline__ RowMask<N> row_mask(const AttendParams& p, const AttendItem& it, int node, int slot) {
  RowMask<N> r;
  r.end = (p.mask ? it.ctx + it.len : it.ctx + min(node + 1, it.len)) - slot;
  const int rel = slot - it.ctx;
  const int w0 = rel >> 5;
  r.shift = rel & 31;
  const uint32_t* m = p.mask + (static_cast<long long>(it.b) * p.c.n_max + node) * p.words;
#pragma unroll
  for (int i = 0; i < N / 32 + 1; ++i) {
    r.w[i] = 0xffffffffu;  // the context
    if (p.mask && w0 + i >= 0) r.w[i] = w0 + i < p.words ? m[w0 + i] : 0u;
  }
  return r;
}

// Bit i: key 32 * c + i of them is visible.
template <int N>
__device__ __forceinline__ uint32_t visible_bits(const RowMask<N>& r, int c) {
  const int n = r.end - 32 * c;
  const uint32_t below = n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
  return below & __funnelshift_r(r.w[c], r.w[c + 1], r.shift);
}

// The masked tiles' values, by the 128 threads of a stream (tid 0..127): rows
// from `rows` on (past the item's keys) become zero, and of the rows from `lo`
// on, which some row does not see, elements that are not finite too (their
// product with a zero weight would be NaN); *bad is set if there were any.
template <int D>
__device__ __forceinline__ void clean_values(unsigned char* v, int lo, int rows, int tid, int* bad) {
  constexpr int CH = D / 8;  // 16-byte chunks of a row
  lo = max(lo, 0);
  bool any = false;
  for (int i = tid; i < (kTcKeys - lo) * CH; i += 128) {
    const int r = lo + i / CH, c = i % CH;
    uint4* at = reinterpret_cast<uint4*>(v + (c >> 3) * (kTcKeys * 128) + r * 128 + (c & 7) * 16);
    if (r >= rows) {
      *at = make_uint4(0u, 0u, 0u, 0u);
      continue;
    }
    uint4 x = *at;
    uint32_t* w = &x.x;
    bool hit = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if ((w[j] & 0x7f80u) == 0x7f80u) { w[j] &= 0xffff0000u; hit = true; }
      if ((w[j] & 0x7f800000u) == 0x7f800000u) { w[j] &= 0x0000ffffu; hit = true; }
    }
    if (hit) {
      *at = x;
      any = true;
    }
  }
  if (any) *bad = 1;
  fence_proxy_async_smem();
}

// Elements that clean_values took out of slots slot0 .. slot1 - 1, for the rows
// that do see them: an infinity or NaN times a positive weight.
template <int N>
__device__ __forceinline__ void add_nonfinite(const AttendParams& p, const AttendItem& it, int node, int slot0, int slot1,
                                           int head_dim, int col, float* o) {
#pragma unroll 1
  for (int slot = slot0; slot < slot1; ++slot) {
    if (slot >= it.ctx && !sees_new(p, it.b, node, it.len, slot - it.ctx)) continue;
    const int pg = page_of(p.c, it.b, slot);
    if (pg < 0) continue;
    const long long base = ((static_cast<long long>(p.c.l0 + it.l) * p.c.n_pages + pg) * p.c.nkv + it.kh) * p.c.ps;
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.c.v_pages) + (base + (slot & (p.c.ps - 1))) * head_dim + col;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float x = __bfloat162float(v[e]);
      o[e] += isfinite(x) ? 0.f : x;
    }
  }
}

// Kernels by the rows of a call: up to 64 (products of 64 rows), one row tile, or
// pairs of row tiles.  Each has its code alone: a switch at run time between the
// ways out of the first two cost a call of one token 0.6 us.
enum TcMode { kFew = 0, kOne = 1, kPair = 2 };

template <int D, int MODE>
__global__ void __launch_bounds__(kTcThreads, 1)
attend_tc_kernel(const __grid_constant__ AttendParams p, const __grid_constant__ TcMaps maps) {
  constexpr bool PAIR = MODE == kPair, m64 = MODE == kFew;
  using P = TcPlan<D, PAIR>;
  constexpr int NS = P::stages, HK = P::step, NH = P::steps;
  // the kernel has no other shared memory: the dynamic block starts on the 1024
  // bytes that the swizzled tiles need
  extern __shared__ __align__(1024) unsigned char smem[];
  TcShared& sh = *reinterpret_cast<TcShared*>(smem + P::shared);
  TcBars& bars = sh.bars;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.q_full[i], 1);
      mbar_init(&bars.q_empty[i], 1);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(&bars.kv_full[i], 1);
      mbar_init(&bars.kv_empty[i], 1);
    }
    for (int s = 0; s < 2; ++s) {
      for (int h = 0; h < 2; ++h) {
        mbar_init(&bars.s_full[s][h], 1);
        mbar_init(&bars.p_full[s][h], 4);
      }
      mbar_init(&bars.o_step[s], 1);
      mbar_init(&bars.o_done[s], 1);
      sh.bad[0][s] = sh.bad[1][s] = 0;
    }
    for (int i = 0; i < NS; ++i) sh.kv_fills[i] = 0u;
    sh.q_fills[0] = sh.q_fills[1] = 0u;
    mbar_init(&bars.drain, 1);
    mbar_fence_init();
  }
  if (warp == kTcMmaWarp) tmem_alloc(&sh.tmem, kTmemCols);
  // Rows of q that no copy writes stay zero: their products cost the tensor
  // cores less power, which sets the clock of a card that streams a cache
  // (256 sequences of one token for a second: 231 us, 240 with whatever lay there,
  // and 254 with products of 128 rows).
  for (int i = tid; i < (PAIR ? 2 : 1) * P::tile / 16; i += kTcThreads)
    reinterpret_cast<uint4*>(smem + P::q)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();  // barriers and tensor memory are set up
  tc_fence_after();
  pdl_trigger();
  pdl_wait();
  const AttendRun run = find_run(p, blockIdx.x == 0 && warp == 0);
  const uint32_t tmem = sh.tmem;
  // Up to 64 rows leave room for the next item's q behind this one's, and take
  // products of 64 rows, whose rows lie in the first 16 lanes of every quarter
  // of tensor memory.
  constexpr int q_bufs = m64 ? 2 : 1;
  const int q_next = m64 ? (p.rows_step + 7) / 8 * 1024 : 0;
  const int tile_rows = PAIR ? p.rows_step / 2 : p.rows_step;  // rows of one row tile
  bool ok = true;
  // Every wait has a limit.  A role whose wait runs out stops, and those that wait
  // for it run out in turn; the exit below ends what is then in flight.
  const unsigned limit = p.wait_limit;
  if (p.withhold >= 0 && p.withhold == (warp >= kTcKeyWarp ? warp : warp >> 2 << 2))  // a test's role
    ok = mbar_wait_bounded(&bars.drain, 0, limit, p.c.err);

  if (warp >= kTcKeyWarp) {
  if constexpr (PAIR) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTcOtherRegs));
  if (warp == kTcKeyWarp || warp == kTcValueWarp) {
    // ---- loads: keys and q by one warp, values by another, each into its
    // buffers of the ring in the order of use: PAIR K0 V0 K1 V1 .., else K0 K1
    // V0 K2 V1 ..  A lane copies one page's share of one 64-column block; its
    // page ids are read kIdsAhead tiles ahead and looked at when they are used.
    constexpr int kIdsAhead = 3;
    const bool keys = warp == kTcKeyWarp;
    const CUtensorMap* map = keys ? &maps.k : &maps.v;
    const int prow = min(p.c.ps, kTcKeys);                  // rows of a box
    const int ppt = kTcKeys / prow;                          // pages of a tile
    const int boxes = ppt * (D / 64);
    const int my_page = lane % ppt, my_half = lane / ppt;
    const unsigned box_off = static_cast<unsigned>(my_half * (kTcKeys * 128) + my_page * prow * 128);
    const int z_none = static_cast<int>(static_cast<long long>(p.c.nkv) * p.c.n_pages * (p.c.l0 + p.c.Lc));
    unsigned base = 0;  // ring position of the piece
    int n_q = 0;
    for (PieceWalk w(run); w.more() && ok; w.next(p)) {
      const int n = w.t1 - w.t0;
      const int* table = p.c.table + static_cast<long long>(w.it.b) * p.c.max_pages;
      // the slot of this lane's box in tile t, and its page id (raw; -1: no key there, zeros)
      auto page_id = [&](int t) -> int {
        const int slot = t * kTcKeys + my_page * prow;
        return lane < boxes && t < w.t1 && slot < w.it.kv_end ? table[slot >> p.c.ps_log2] : -1;
      };
      const int z_head = (p.c.l0 + w.it.l) * static_cast<int>(p.c.n_pages);
      auto fill = [&](int i, int pg) {
        const unsigned at = base + static_cast<unsigned>(PAIR ? 2 * i + (keys ? 0 : 1) : keys ? (i < 2 ? i : 2 * i - 1)
                                                                                        : (n == 1 ? 1 : min(2 * i + 2, n + i)));
        const unsigned st = at % NS, turn = at / NS;
        if (turn > 0) ok = ok && mbar_wait_bounded(&bars.kv_empty[st], (turn - 1) & 1u, limit, p.c.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        const int t = w.t0 + i;
        int z = z_none;
        if (pg >= 0 && pg < p.c.n_pages)
          z = (z_head + pg) * p.c.nkv + w.it.kh;
        else if (lane < boxes && t * kTcKeys + my_page * prow < w.it.kv_end)
          latch_error(p.c.err, SFA_ERR_INVALID_ARG);  // a page that is needed: read as zeros
        if (lane == 0) {
          sh.kv_fills[st] = turn + 1;
          mbar_arrive_expect_tx(&bars.kv_full[st], P::tile);
        }
        __syncwarp();
        if (lane < boxes)
          tma_load_3d(smem + P::ring + st * P::tile + box_off, map, my_half * 64, (t * kTcKeys) & (p.c.ps - 1) & ~(prow - 1), z,
                      &bars.kv_full[st]);
      };
      // q goes behind the item's first keys: its buffer may still be in use
      auto load_q = [&]() {
        const int qb = n_q % q_bufs, turn = n_q / q_bufs;
        if (turn > 0)
          ok = ok && mbar_wait_bounded(&bars.q_empty[qb], static_cast<unsigned>((turn - 1) & 1), limit, p.c.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        const int node0 = p.by_group(w.it.row0);
        const int nb = p.by_group(tile_rows);
        if (lane == 0) {
          sh.q_fills[qb] = static_cast<unsigned>(turn + 1);
          mbar_arrive_expect_tx(&bars.q_full[qb], static_cast<unsigned>(tile_rows * 128 * (D / 64) * (PAIR ? 2 : 1)));
          for (int s = 0; s < (PAIR ? 2 : 1); ++s)
            for (int h = 0; h < D / 64; ++h)
              tma_load_4d(smem + P::q + s * P::tile + qb * q_next + h * (kTcRows * 128), &maps.q, h * 64,
                          w.it.kh * p.c.G, node0 + s * nb, w.it.l * p.c.B + w.it.b, &bars.q_full[qb]);
        }
        __syncwarp();
        ++n_q;
      };
      int id[kIdsAhead];
#pragma unroll
      for (int j = 0; j < kIdsAhead; ++j) id[j] = page_id(w.t0 + j);
      const int q_after = PAIR ? 0 : min(n, 2) - 1;  // q follows this tile's keys
      for (int i = 0; i < n && ok; ++i) {
        const int next = page_id(w.t0 + i + kIdsAhead);
        fill(i, id[0]);
        if (keys && i == q_after && ok) load_q();
#pragma unroll
        for (int j = 0; j + 1 < kIdsAhead; ++j) id[j] = id[j + 1];
        id[kIdsAhead - 1] = next;
      }
      base += 2u * static_cast<unsigned>(n);
    }
  } else if (warp == kTcMmaWarp) {
    // ---- products.  The whole warp walks and waits, so that addresses stay
    // uniform; one elected lane issues.
    {
      const bool leader = elect_one();
      const uint32_t idesc_qk = umma_idesc_bf16(m64 ? 64 : kTcRows, HK, false);
      const uint32_t idesc_pv = umma_idesc_bf16(m64 ? 64 : kTcRows, D, true);
      const uint64_t d_q = desc_sw128(smem_u32(smem + P::q), 16, 1024);
      const uint64_t d_k = desc_sw128(smem_u32(smem + P::ring), 16, 1024);
      const uint64_t d_v = desc_sw128(smem_u32(smem + P::ring), kTcKeys * 128, 1024);
      int ring_st = 0;
      unsigned ring_turn = 0;
      int n_q = 0;
      unsigned n_p[2][2] = {{0u, 0u}, {0u, 0u}};  // [stream][step]: how often its P was waited for
      auto wait = [&](uint64_t* bar, unsigned parity) {
        ok = ok && mbar_wait_bounded(bar, parity & 1u, limit, p.c.err);
        ok = __all_sync(0xffffffffu, ok);  // no lane may fall two phases behind
        tc_fence_after();
        return ok;
      };
      // takes the ring's next buffer
      auto next_kv = [&](int* st) {
        *st = ring_st;
        const bool r = wait(&bars.kv_full[ring_st], ring_turn);
        if (++ring_st == NS) {
          ring_st = 0;
          ++ring_turn;
        }
        return r;
      };
      auto commit = [&](uint64_t* bar) {
        if (leader) umma_commit(bar);
      };
      // scores of half h of the keys in buffer st
      auto qk = [&](int s, int h, int st, uint64_t q_desc) {
        const uint64_t a = q_desc + (PAIR ? s * (P::tile >> 4) : 0);
        const uint64_t b = d_k + ((st * P::tile + h * (HK * 128)) >> 4);
        const uint32_t d = tmem + static_cast<uint32_t>(s * kTcKeys + h * HK);
        if (leader) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = ((k >> 2) * (kTcKeys * 128) + (k & 3) * 32) >> 4;
            umma_bf16(d, a + off, b + off, idesc_qk, k > 0);
          }
          umma_commit(&bars.s_full[s][h]);
        }
      };
      // their P times the values in buffer st
      auto pv = [&](int s, int h, int st, bool first) {
        const uint64_t b = d_v + ((st * P::tile + h * (HK * 128)) >> 4);
        const uint32_t d = tmem + 256u + static_cast<uint32_t>(s) * D;
        const uint32_t a = tmem + static_cast<uint32_t>(s * kTcKeys + h * HK);
        if (leader) {
#pragma unroll
          for (int k = 0; k < HK / 16; ++k)
            umma_bf16_ts(d, a + k * 8, b + ((k * 2048) >> 4), idesc_pv, k > 0 || !first);
#pragma unroll
          for (int k = 0; k < HK / 16; ++k)  // and what rounding P left
            umma_bf16_ts(d, a + HK / 2 + k * 8, b + ((k * 2048) >> 4), idesc_pv, true);
          if (NH > 1) umma_commit(&bars.o_step[s]);
        }
      };
      for (PieceWalk w(run); w.more() && ok; w.next(p)) {
        const int n = w.t1 - w.t0;
        const int qb = n_q % q_bufs;
        if (!wait(&bars.q_full[qb], static_cast<unsigned>(n_q / q_bufs))) break;
        ++n_q;
        const uint64_t d_qb = d_q + (qb * q_next >> 4);
        int st_k = 0, st_v = 0;
        if (PAIR) {
          if (!next_kv(&st_k)) break;
#pragma unroll
          for (int hs = 0; hs < 2 * NH; ++hs) qk(hs & 1, hs >> 1, st_k, d_qb);
          commit(&bars.kv_empty[st_k]);
          if (n == 1) commit(&bars.q_empty[qb]);
          for (int i = 0; i < n && ok; ++i) {
            const bool more = i + 1 < n;
            if (!next_kv(&st_v)) break;
#pragma unroll
            for (int hs = 0; hs < 2 * NH; ++hs) {  // a step of both streams, then the next
              const int h = hs >> 1, s = hs & 1;
              if (!wait(&bars.p_full[s][h], n_p[s][h]++)) continue;
              pv(s, h, st_v, i == 0 && h == 0);
              if (more && hs == 0 && !next_kv(&st_k)) continue;
              if (more) qk(s, h, st_k, d_qb);
            }
            if (!ok) break;
            if (more) {  // (the piece's last values' buffer is the softmax's, for its result)
              commit(&bars.kv_empty[st_v]);
              commit(&bars.kv_empty[st_k]);
            }
            if (i + 2 == n) commit(&bars.q_empty[qb]);
            if (!more)
              for (int s = 0; s < 2; ++s) commit(&bars.o_done[s]);
          }
        } else if (n == 1) {
          // one tile: a half for each stream
          if (!next_kv(&st_k)) break;
          qk(0, 0, st_k, d_qb);
          qk(1, 1, st_k, d_qb);
          commit(&bars.kv_empty[st_k]);
          commit(&bars.q_empty[qb]);
          if (!next_kv(&st_v)) break;
          if (!wait(&bars.p_full[0][0], n_p[0][0]++)) break;
          pv(0, 0, st_v, true);
          if (!wait(&bars.p_full[1][1], n_p[1][1]++)) break;
          pv(1, 1, st_v, true);
          if (m64) commit(&bars.kv_empty[st_v]);
          commit(&bars.o_done[0]);
        } else {
          for (int i = 0; i < 2 && ok; ++i) {
            if (!next_kv(&st_k)) break;
            for (int h = 0; h < NH; ++h) qk(i, h, st_k, d_qb);
            commit(&bars.kv_empty[st_k]);
          }
          if (!ok) break;
          if (n == 2) commit(&bars.q_empty[qb]);
          for (int i = 0; i < n && ok; ++i) {
            const int s = i & 1;
            const bool more = i + 2 < n;
            if (!next_kv(&st_v)) break;
            for (int h = 0; h < NH && ok; ++h) {
              if (!wait(&bars.p_full[s][h], n_p[s][h]++)) break;
              pv(s, h, st_v, i < 2 && h == 0);
              if (more && h == 0 && !next_kv(&st_k)) break;
              if (more) qk(s, h, st_k, d_qb);
            }
            if (!ok) break;
            if (i + 1 < n || m64) commit(&bars.kv_empty[st_v]);  // (the last one is the softmax's, for its result)
            if (more) commit(&bars.kv_empty[st_k]);
            if (i + 3 == n) commit(&bars.q_empty[qb]);
          }
          if (!ok) break;
          commit(&bars.o_done[0]);
        }
        if (!ok) break;
      }
    }
    __syncwarp();
  }
  } else {
    if constexpr (PAIR) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTcSoftmaxRegs));
    // ---- softmax of stream s, a thread per row
    const int s = warp >> 2, sub = warp & 3;
    const int tl = sub * 32 + lane;  // tensor-memory lane
    const int r = !m64 ? tl : lane < 16 ? sub * 16 + lane : kTcRows;  // its row of the tile
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(sub * 32) << 16);
    const uint32_t t_o = lane_base + 256u + static_cast<uint32_t>(s) * D;
    unsigned n_s[2] = {0u, 0u};      // scores of each step's columns so far
    unsigned n_o = 0, n_piece = 0;   // steps of this stream, and pieces, so far
    unsigned n_kv = 0;  // ring position of the piece's first buffer
    bool wrote = false;
    // after a wait that ran out a warp only keeps the CTA's barriers company
    for (PieceWalk w(run); w.more(); w.next(p)) {
      const AttendItem& it = w.it;
      const int n = w.t1 - w.t0;
      const int row0 = it.row0 + (PAIR ? s * tile_rows : 0);
      const int rows = min(tile_rows, it.rows - (PAIR ? s * tile_rows : 0));  // <= 0: an empty second tile
      const bool warp_live = sub * (m64 ? 16 : 32) < rows;
      const int nd = p.by_group(row0 + r), node = min(nd, max(it.len - 1, 0));
      // keys below this are visible to every row of the piece
      const int full_end = p.mask ? it.ctx : it.ctx + p.by_group(it.row0) + 1;
      float m = -INFINITY, l = 0.f;
      const bool halves = !PAIR && n == 1;  // one tile: stream s takes its half s
      for (int i = PAIR || halves ? 0 : s; i < n && ok; i += PAIR ? 1 : 2) {
        const int t = w.t0 + i;
        const bool masked = (t + 1) * kTcKeys > full_end;
#pragma unroll 1
        for (int h = 0; h < NH; ++h) {
          if (halves && h != s) continue;
          const bool first = halves || (h == 0 && (PAIR ? i == 0 : i < 2));
          RowMask<HK> vis;
          if (masked) vis = row_mask<HK>(p, it, node, t * kTcKeys + h * HK);
          ok = mbar_wait_bounded(&bars.s_full[s][h], (h == 0 ? n_s[0] : n_s[1]) & 1u, limit, p.c.err);
          h == 0 ? ++n_s[0] : ++n_s[1];
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (masked && h == 0 && (!PAIR || s == 0)) {  // (a tile in halves: by stream 0, whose product comes first)
            // This tile's values: their buffer's place in the loaders' order.  The
            // scores came after the values before the last were used, so the
            // buffer's phase can be told from its last but one.
            const unsigned at = n_kv + static_cast<unsigned>(PAIR ? 2 * i + 1 : (n == 1 ? 1 : min(2 * i + 2, n + i)));
            const unsigned st = at % NS;
            ok = mbar_wait_bounded(&bars.kv_full[st], (at / NS) & 1u, limit, p.c.err);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            clean_values<D>(smem + P::ring + st * P::tile, full_end - t * kTcKeys, it.kv_end - t * kTcKeys, tl,
                            &sh.bad[n_piece & 1u][s]);
          }
          tc_fence_after();
          if (warp_live) {
            const uint32_t t_s = lane_base + static_cast<uint32_t>(s * kTcKeys + h * HK);
            float x[HK];
#pragma unroll
            for (int c = 0; c < HK; c += 32) tmem_ld32_async(t_s + c, x + c);
            tmem_ld_wait<HK>(x);
            if (masked) {
#pragma unroll
              for (int c = 0; c < HK / 32; ++c) {
                const uint32_t bits = visible_bits(vis, c);
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (!((bits >> j) & 1u)) x[c * 32 + j] = -INFINITY;
              }
            }
            float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int j = 4; j + 1 < HK; j += 2) mx[(j >> 1) & 3] = max3(mx[(j >> 1) & 3], x[j], x[j + 1]);
            const float top = max3(mx[0], mx[1], max3(mx[2], mx[3], mx[3])) * p.scale_log2;
            // the maximum in use may lag behind by 2^8 (and 1), which fp32 sums and outputs hold easily
            const bool move = !(top <= m + kRescaleLog2);  // a NaN score moves it to NaN, and the row with it
            float fix = 1.f;
            if (move) {  // to a whole power of two: P's digits, and so its rounding, hardly depend on m
              const float to = floorf(top);
              fix = exp2_approx(m - to);
              m = to;
              l *= fix;
            }
            if (!first && __any_sync(0xffffffffu, move && r < rows)) {
              // O holds the step before the last of this stream (these scores came
              // after it); with two steps a tile the last one is waited for
              if (NH > 1) {
                ok = mbar_wait_bounded(&bars.o_step[s], (n_o - 1u) & 1u, limit, p.c.err);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
              }
              tc_fence_after();
              float o[32];
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                tmem_ld32_async(t_o + c, o);
                tmem_ld_wait<32>(o);
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] *= fix;
                tmem_st32(t_o + c, reinterpret_cast<const uint32_t*>(o));
              }
            }
            // (rows that are not there get P = 0, as those of warps without rows have)
            l += store_probs<HK>(x, p.scale_log2, r >= rows ? INFINITY : m == -INFINITY ? 0.f : m, t_s);
            tmem_st_wait();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.p_full[s][h]);
          ++n_o;
        }
        if (!ok) break;
      }
      n_kv += 2u * static_cast<unsigned>(n);
      // ---- result of the piece
      const bool starts = w.t0 == 0, whole = starts && w.t1 == it.nt;
      ok = ok && mbar_wait_bounded(&bars.o_done[PAIR ? s : 0], n_piece & 1u, limit, p.c.err);
      ok = __all_sync(0xffffffffu, ok);
      if (!PAIR) {
        sh.ml[s][tl] = make_float2(m, l);
        named_bar_sync(1, kTcSoftmaxThreads);
      }
      const unsigned st_last = (n_kv - 1u) % NS;  // the last values: used up, and not given back yet
      if (ok) {
        tc_fence_after();
        float w0 = 1.f, w1 = 0.f;
        if (!PAIR) {
          const float2 a = sh.ml[0][tl], b = sh.ml[1][tl];
          m = fmaxf(a.x, b.x);
          const float base = m == -INFINITY ? 0.f : m;
          w0 = exp2_approx(a.x - base);
          w1 = exp2_approx(b.x - base);
          l = a.y * w0 + b.y * w1;
        }
        const int* bad = sh.bad[n_piece & 1u];
        const bool fix = PAIR ? bad[0] != 0 : (bad[0] | bad[1]) != 0;
        const float inv = l == 0.f ? 0.f : 1.0f / l;
        constexpr int NC = PAIR ? D : D / 2;       // columns of this warp group
        constexpr int RB = P::tile / 8 / 32;       // bytes of a row in a warp's share of the buffer
        constexpr int CH = RB / 16, W = RB / 2;    // 16-byte chunks of it; columns at a time
        const int c0 = PAIR ? 0 : s * NC;
        const int row_w = sub * (m64 ? 16 : 32);   // the warp's first row, and its rows
        const int rows_w = min(m64 ? 16 : 32, rows - row_w);
        const long long slot_row =
            static_cast<long long>(piece_slot(static_cast<int>(blockIdx.x), starts)) * p.rows_step + (PAIR ? s * tile_rows : 0);
        const long long out_row = static_cast<long long>(it.l) * p.c.B + it.b;
        if (!whole && r < rows && c0 == 0)
          *reinterpret_cast<float2*>(p.part_ml + (slot_row + r) * 2) = make_float2(m, l);
        // More than 64 rows go out through shared memory, so that a store covers
        // whole lines (a row per lane touches 32 lines with every 16 bytes: a call
        // of 64 new tokens took 29 us and takes 27); fewer go out from registers,
        // which is 0.5 us sooner for a handful.
        unsigned char* stage = smem + P::ring + st_last * P::tile + warp * (P::tile / 8);
        auto chunk = [&](int row, int c) {  // conflict-free both ways
          return reinterpret_cast<uint4*>(stage + row * RB + ((c ^ (CH == 8 ? row & 7 : (row >> 1) & 3)) << 4));
        };
        auto flush = [&](unsigned char* base, bool token_rows, long long pitch) {
          __syncwarp();
#pragma unroll 4
          for (int k = 0; k < rows_w; k += 32 / CH) {
            const int row = k + lane / CH;
            if (row >= rows_w) break;
            long long at = row_w + row;
            if (token_rows) {
              const int gr = row0 + row_w + row, node_r = p.by_group(gr);
              at = (out_row * p.c.n_max + node_r) * p.c.nq + it.kh * p.c.G + (gr - node_r * p.c.G);
            }
            *reinterpret_cast<uint4*>(base + at * pitch + (lane % CH) * 16) = *chunk(row, lane % CH);
          }
          __syncwarp();
        };
        if (warp_live) {
#pragma unroll 1
          for (int c = 0; c < NC; c += W) {
            float o[W];
            const uint32_t t_c = lane_base + 256u + (PAIR ? s * D : c0) + c;
#pragma unroll
            for (int j = 0; j < W; j += 32) tmem_ld32_async(t_c + j, o + j);
            if constexpr (!PAIR) {
              float o1[W];
#pragma unroll
              for (int j = 0; j < W; j += 32) tmem_ld32_async(t_c + D + j, o1 + j);
              tmem_ld_wait<W>(o);
              tmem_ld_wait<W>(o1);
#pragma unroll
              for (int j = 0; j < W; ++j) o[j] = fmaf(o1[j], w1, o[j] * w0);
            } else {
              tmem_ld_wait<W>(o);
            }
            if (fix && r < rows)
              add_nonfinite<W>(p, it, node, max(w.t0 * kTcKeys, full_end), min(w.t1 * kTcKeys, it.kv_end), D, c0 + c, o);
            if (m64) {
              if (r < rows) {
                if (whole) {
                  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) +
                                       ((out_row * p.c.n_max + nd) * p.c.nq + it.kh * p.c.G + (row0 + r - nd * p.c.G)) * D + c0 + c;
#pragma unroll
                  for (int j = 0; j < W; j += 8) {
                    uint32_t u[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                      const __nv_bfloat162 b = __floats2bfloat162_rn(o[j + 2 * e] * inv, o[j + 2 * e + 1] * inv);
                      u[e] = *reinterpret_cast<const uint32_t*>(&b);
                    }
                    *reinterpret_cast<uint4*>(dst + j) = make_uint4(u[0], u[1], u[2], u[3]);
                  }
                } else {
#pragma unroll
                  for (int j = 0; j < W; j += 4)
                    *reinterpret_cast<float4*>(p.part_o + (slot_row + r) * D + c0 + c + j) =
                        make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                }
              }
            } else if (whole) {
              if (r < rows) {
#pragma unroll
                for (int j = 0; j < W; j += 8) {
                  uint32_t u[4];
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    // (a row that sees nothing has zeros in O and inv)
                    const __nv_bfloat162 b = __floats2bfloat162_rn(o[j + 2 * e] * inv, o[j + 2 * e + 1] * inv);
                    u[e] = *reinterpret_cast<const uint32_t*>(&b);
                  }
                  *chunk(r - row_w, j / 8) = make_uint4(u[0], u[1], u[2], u[3]);
                }
              }
              flush(reinterpret_cast<unsigned char*>(p.out) + (c0 + c) * 2, true, D * 2);
            } else {
#pragma unroll
              for (int q = 0; q < W; q += W / 2) {
                if (r < rows)
#pragma unroll
                  for (int j = 0; j < W / 2; j += 4)
                    *chunk(r - row_w, j / 4) = make_uint4(__float_as_uint(o[q + j]), __float_as_uint(o[q + j + 1]),
                                                          __float_as_uint(o[q + j + 2]), __float_as_uint(o[q + j + 3]));
                flush(reinterpret_cast<unsigned char*>(p.part_o) + slot_row * D * 4 + (c0 + c + q) * 4, false, D * 4);
              }
            }
          }
        }
        if (starts && !whole) {
          if (tid == 0) write_meta(p, run, true, it, w.item_first(run));
          wrote = true;
        }
        tc_fence_before();
      }
      // outputs, flags and the buffer are read: the next piece may overwrite them
      if (!m64) fence_proxy_async_smem();
      named_bar_sync(1, kTcSoftmaxThreads);
      if (tid == 0) {
        sh.bad[n_piece & 1u][0] = sh.bad[n_piece & 1u][1] = 0;
        if (!m64 && ok) mbar_arrive(&bars.kv_empty[st_last]);
      }
      ++n_piece;
    }
    if (!wrote && tid == 0) write_meta(p, run, false, run.it, 0);
  }
  tc_fence_before();
  const bool all_ok = __syncthreads_and(ok);
  if (warp == kTcMmaWarp) {
    tc_fence_after();
    // After a wait that ran out: products end before tensor memory is freed, and
    // copies land before the CTA leaves its shared memory to another.
    if (!all_ok) {
      if (elect_one()) umma_commit(&bars.drain);
      mbar_wait_bounded(&bars.drain, 0, kTcPollLimit, p.c.err);
      for (int i = 0; i < NS; ++i)
        if (sh.kv_fills[i] > 0) mbar_wait_bounded(&bars.kv_full[i], (sh.kv_fills[i] - 1) & 1u, kTcPollLimit, p.c.err);
      for (int i = 0; i < q_bufs; ++i)
        if (sh.q_fills[i] > 0) mbar_wait_bounded(&bars.q_full[i], (sh.q_fills[i] - 1) & 1u, kTcPollLimit, p.c.err);
      __syncwarp();
    }
    tmem_dealloc(tmem, kTmemCols);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 tc_map_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
  }();
  return fn;
}

// q as (D, n_q, node, layer x sequence) with boxes of 64 x G x nodes x 1, keys
// and values as (D, slot of the page, layer x page x head) with boxes of 64 x
// page rows x 1; what lies outside reads as zeros.
cudaError_t encode_maps(const AttendParams& p, int D, int nodes, TcMaps* m) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = tc_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const PagedParams& c = p.c;
  const cuuint64_t row = static_cast<cuuint64_t>(D) * 2;
  const cuuint64_t qd[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(c.nq), static_cast<cuuint64_t>(c.n_max),
                            static_cast<cuuint64_t>(c.Lc) * static_cast<cuuint64_t>(c.B)};
  const cuuint64_t qs[3] = {row, row * c.nq, row * c.nq * c.n_max};
  const cuuint32_t qb[4] = {64, static_cast<cuuint32_t>(c.G), static_cast<cuuint32_t>(nodes), 1};
  if (enc(&m->q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(p.q), qd, qs, qb, estr,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  const cuuint64_t kd[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(c.ps),
                            static_cast<cuuint64_t>(c.l0 + c.Lc) * static_cast<cuuint64_t>(c.n_pages) *
                                static_cast<cuuint64_t>(c.nkv)};
  const cuuint64_t ks[2] = {row, row * c.ps};
  const cuuint32_t kb[3] = {64, static_cast<cuuint32_t>(std::min(c.ps, kTcKeys)), 1};
  auto kv = [&](CUtensorMap* map, void* base) {
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, kd, ks, kb, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  return kv(&m->k, c.k_pages) && kv(&m->v, c.v_pages) ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, int MODE>
constexpr int tc_smem() { return TcPlan<D, MODE == kPair>::shared + static_cast<int>(sizeof(TcShared)); }

template <int D, int MODE>
cudaError_t launch_tc(const AttendParams& p, cudaStream_t s) {
  TcMaps maps;
  const cudaError_t e = encode_maps(p, D, p.rows_step / (MODE == kPair ? 2 : 1) / p.c.G, &maps);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.n_cta), 1, 1);
  cfg.blockDim = dim3(kTcThreads, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(tc_smem<D, MODE>());
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attend_tc_kernel<D, MODE>, p, maps);
}

template <int D, int MODE>
cudaError_t allow_tc() {
  return cudaFuncSetAttribute(attend_tc_kernel<D, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              tc_smem<D, MODE>());
}

}  // namespace

// Nodes of a row tile; the call takes two row tiles at a time when its nodes
// do not fit one.
void attend_tc_rows(int G, int n_max, AttendPlan* a) {
  const int nodes = kTcRows / G;
  const bool pairs = n_max > nodes;
  a->rows_step = pairs ? 2 * nodes * G : n_max * G;
  a->kt = kTcKeys;
  a->item_cost = pairs ? kAttendItemCostPairs : kAttendItemCost;
}

cudaError_t attend_tc_prepare() {
  cudaError_t e = allow_tc<64, kFew>();
  if (e == cudaSuccess) e = allow_tc<64, kOne>();
  if (e == cudaSuccess) e = allow_tc<64, kPair>();
  if (e == cudaSuccess) e = allow_tc<128, kFew>();
  if (e == cudaSuccess) e = allow_tc<128, kOne>();
  if (e == cudaSuccess) e = allow_tc<128, kPair>();
  return e;
}

cudaError_t launch_attend_tc(const AttendParams& p, int head_dim, cudaStream_t s) {
  const int mode = p.c.n_max > kTcRows / p.c.G ? kPair : p.rows_step > kTcRows / 2 ? kOne : kFew;
  const bool small = head_dim == 64;
  switch (mode) {
    case kPair: return small ? launch_tc<64, kPair>(p, s) : launch_tc<128, kPair>(p, s);
    case kOne: return small ? launch_tc<64, kOne>(p, s) : launch_tc<128, kOne>(p, s);
    default: return small ? launch_tc<64, kFew>(p, s) : launch_tc<128, kFew>(p, s);
  }
}

}  // namespace sfa
