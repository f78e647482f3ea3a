// sfa_paged.cuh — device helpers of the paged key/value cache calls: the
// lengths of a sequence and the page of a slot.
#pragma once

#include "sfa_common.cuh"

namespace sfa {

struct SeqLens {
  int ctx, len;  // tokens cached before the call, new tokens; len 0 for a skipped sequence
};

// Lengths of sequence b, with a sequence that does not fit its pages (or a
// count out of range) turned into one without new tokens and latched.
__device__ __forceinline__ SeqLens seq_lens(const PagedParams& c, int b, bool latch) {
  SeqLens r;
  r.ctx = c.ctx[b];
  r.len = c.lens ? c.lens[b] : c.n_max;
  const bool ok = r.ctx >= 0 && r.len >= 0 && r.len <= c.n_max &&
                  static_cast<long long>(r.ctx) + r.len <= static_cast<long long>(c.max_pages) * c.ps;
  if (!ok) {
    if (latch) latch_error(c.err, SFA_ERR_INVALID_ARG);
    r.ctx = 0;
    r.len = 0;
  }
  return r;
}

// Page id of slot `slot` of sequence b, or -1 (latched) if the table's entry
// is out of range.
__device__ __forceinline__ int page_of(const PagedParams& c, int b, int slot, bool latch = true) {
  const int pg = c.table[static_cast<long long>(b) * c.max_pages + (slot >> c.ps_log2)];
  if (pg >= 0 && pg < c.n_pages) return pg;
  if (latch) latch_error(c.err, SFA_ERR_INVALID_ARG);
  return -1;
}

// Element offset of row 0 of KV head kh in page pg of layer l (a state layer).
template <int D>
__device__ __forceinline__ long long page_base(const PagedParams& c, int l, int pg, int kh) {
  return ((static_cast<long long>(l) * c.n_pages + pg) * c.nkv + kh) * c.ps * D;
}

// ---- the work of an attend call ---------------------------------------------
// A work item is (layer, sequence, KV head, row tile): rows_step consecutive
// rows (node * G + head of the group) against the keys that any of them sees,
// in tiles of kt.  The tiles of all items, in the order layer, sequence, row
// tile, KV head, are dealt out in equal runs, one to a CTA: a run may end inside
// an item, whose pieces are then joined by the combine kernel.  Lengths live on
// the device, so every CTA works out its own run.

struct AttendItem {
  int l, b, kh, rt;   // rt: row tile
  int ctx, len;
  int nt;             // key tiles
  int kv_end;         // keys that any of its rows sees
  int row0, rows;
};

struct AttendRun {
  AttendItem it;      // item of the first tile
  int tile;           // its first tile
  long long first;    // global index of the first tile
  long long tiles;    // tiles of this CTA
  long long chunk;    // tiles of every CTA but the last ones
};

__device__ __forceinline__ int row_tiles(const AttendParams& p, int len) {
  return (len * p.c.G + p.rows_step - 1) / p.rows_step;
}

// Keys that any row of row tile rt sees.
__device__ __forceinline__ int kv_end_of(const AttendParams& p, int ctx, int len, int rt) {
  if (p.mask) return ctx + len;
  const int row_end = min((rt + 1) * p.rows_step, len * p.c.G);
  return ctx + (row_end - 1) / p.c.G + 1;
}

__device__ __forceinline__ void set_item(const AttendParams& p, AttendItem& it) {
  it.row0 = it.rt * p.rows_step;
  it.rows = min(p.rows_step, it.len * p.c.G - it.row0);
  it.kv_end = kv_end_of(p, it.ctx, it.len, it.rt);
  it.nt = (it.kv_end + p.kt - 1) / p.kt;
}

// The item after `it`; only called where one follows.
__device__ __forceinline__ void next_item(const AttendParams& p, AttendItem& it) {
  if (++it.kh < p.c.nkv) return;
  it.kh = 0;
  if (++it.rt >= row_tiles(p, it.len)) {
    it.rt = 0;
    do {
      if (++it.b >= p.c.B) {
        it.b = 0;
        ++it.l;
      }
      const SeqLens s = seq_lens(p.c, it.b, false);
      it.ctx = s.ctx;
      it.len = s.len;
    } while (it.len == 0);
  }
  set_item(p, it);
}

// This CTA's run, by all NT threads.  s_pre: shared scratch of B + 1 long longs.
template <int NT>
__device__ __forceinline__ void find_run(const AttendParams& p, long long* s_pre, AttendRun* s_run) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = p.c.B;
  const int most = row_tiles(p, p.c.n_max);
  if (p.mask || most <= 8) {
    for (int b = tid; b < B; b += NT) {
      const SeqLens s = seq_lens(p.c, b, blockIdx.x == 0);
      long long n = 0;
      const int nrt = row_tiles(p, s.len);
      if (p.mask)
        n = static_cast<long long>(nrt) * ((s.ctx + s.len + p.kt - 1) / p.kt);
      else
        for (int rt = 0; rt < nrt; ++rt) n += (kv_end_of(p, s.ctx, s.len, rt) + p.kt - 1) / p.kt;
      s_pre[b] = n * p.c.nkv;
    }
  } else {
    for (int b = warp; b < B; b += NT / 32) {
      const SeqLens s = seq_lens(p.c, b, blockIdx.x == 0);
      const int nrt = row_tiles(p, s.len);
      long long n = 0;
      for (int rt = lane; rt < nrt; rt += 32) n += (kv_end_of(p, s.ctx, s.len, rt) + p.kt - 1) / p.kt;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
      if (lane == 0) s_pre[b] = n * p.c.nkv;
    }
  }
  __syncthreads();
  if (warp == 0) {
    // exclusive prefix sums: a run of sequences per lane, then a warp scan
    const int per = (B + 31) / 32;
    const int b0 = min(B, lane * per), b1 = min(B, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += s_pre[b];
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    const long long layer = __shfl_sync(0xffffffffu, inc, 31);
    long long at = inc - mine;
    for (int b = b0; b < b1; ++b) {
      const long long n = s_pre[b];
      s_pre[b] = at;
      at += n;
    }
    if (lane == 31) s_pre[B] = layer;
    __syncwarp();
    const long long total = layer * p.c.Lc;
    const long long chunk = max(static_cast<long long>(p.min_tiles), (total + p.n_cta - 1) / p.n_cta);
    const long long first = static_cast<long long>(blockIdx.x) * chunk;
    const long long tiles = max(0LL, min(chunk, total - first));
    AttendRun r;
    r.first = first;
    r.tiles = tiles;
    r.chunk = chunk;
    if (tiles > 0) {
      const int l = static_cast<int>(first / layer);
      long long rem = first - l * layer;
      int lo = 0, hi = B - 1;  // last sequence whose prefix is <= rem (one with tiles: empty ones share the next's prefix)
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_pre[mid] <= rem) lo = mid;
        else hi = mid - 1;
      }
      rem -= s_pre[lo];
      r.it.l = l;
      r.it.b = lo;
      const SeqLens s = seq_lens(p.c, lo, false);
      r.it.ctx = s.ctx;
      r.it.len = s.len;
      const int nrt = row_tiles(p, s.len);
      int rt = 0, nt = 0;
      if (p.mask) {
        nt = (s.ctx + s.len + p.kt - 1) / p.kt;
        const long long per_rt = static_cast<long long>(nt) * p.c.nkv;
        rt = static_cast<int>(rem / per_rt);
        rem -= rt * per_rt;
      } else {
        for (int base = 0; base < nrt; base += 32) {  // the row tile that holds the remainder, 32 at a time
          const int mine_rt = base + lane;
          const int t = mine_rt < nrt ? (kv_end_of(p, s.ctx, s.len, mine_rt) + p.kt - 1) / p.kt : 0;
          const long long n = static_cast<long long>(t) * p.c.nkv;
          long long inc2 = n;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const long long up = __shfl_up_sync(0xffffffffu, inc2, o);
            if (lane >= o) inc2 += up;
          }
          const unsigned hit = __ballot_sync(0xffffffffu, inc2 > rem);
          if (hit) {
            const int src = __ffs(hit) - 1;
            rt = base + src;
            nt = __shfl_sync(0xffffffffu, t, src);
            rem -= __shfl_sync(0xffffffffu, inc2 - n, src);
            break;
          }
          rem -= __shfl_sync(0xffffffffu, inc2, 31);
        }
      }
      r.it.rt = rt;
      r.it.kh = static_cast<int>(rem / nt);
      r.tile = static_cast<int>(rem - static_cast<long long>(r.it.kh) * nt);
      set_item(p, r.it);
    }
    if (lane == 0) *s_run = r;
  }
  __syncthreads();
}

// Partial result slot of a piece: a CTA has at most one piece that continues an
// item and one that starts an item without finishing it.
__device__ __forceinline__ int piece_slot(int cta, bool starts) { return cta * 2 + (starts ? 1 : 0); }

// Written once per run by one thread: the split item that this run starts, if any.
__device__ __forceinline__ void write_meta(const AttendParams& p, const AttendRun& r, bool starts_split,
                                           const AttendItem& it, long long item_first) {
  SplitMeta m = {};
  m.last_cta = -1;
  if (starts_split) {
    m.last_cta = static_cast<int>((item_first + it.nt - 1) / r.chunk);
    m.l = it.l;
    m.b = it.b;
    m.kh = it.kh;
    m.row0 = it.row0;
    m.rows = it.rows;
  }
  p.meta[blockIdx.x] = m;
}

// Whether new token rel (slot less ctx) is visible to node `node`.
__device__ __forceinline__ bool sees_new(const AttendParams& p, int b, int node, int len, int rel) {
  if (rel >= len) return false;
  if (!p.mask) return rel <= node;
  return (p.mask[(static_cast<long long>(b) * p.c.n_max + node) * p.words + (rel >> 5)] >> (rel & 31)) & 1u;
}

// 2^x, of a log2-scaled score less the running maximum.
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

}  // namespace sfa
