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
// in tiles of kt.  An item counts item_cost units for its start and result and
// one for every tile; the units of all items, in the order layer, sequence, row
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
  AttendItem it;      // item of the first unit
  int unit;           // which of its units that is
  int first;          // global index of the first unit
  int units;          // units of this CTA
  int chunk;          // units of every CTA but the last ones
  int cost;           // units that an item counts besides its tiles
};

__device__ __forceinline__ int row_tiles(const AttendParams& p, int len) {
  return p.by_rows(len * p.c.G + p.rows_step - 1);
}

// Key tiles that cover keys 0 .. n - 1.
__device__ __forceinline__ int tiles_up_to(const AttendParams& p, int n) {
  return static_cast<int>((static_cast<unsigned>(n) + static_cast<unsigned>(p.kt) - 1u) >> p.kt_log2);
}

// Keys that any row of row tile rt sees.
__device__ __forceinline__ int kv_end_of(const AttendParams& p, int ctx, int len, int rt) {
  if (p.mask) return ctx + len;
  const int row_end = min((rt + 1) * p.rows_step, len * p.c.G);
  return ctx + p.by_group(row_end - 1) + 1;
}

__device__ __forceinline__ void set_item(const AttendParams& p, AttendItem& it) {
  it.row0 = it.rt * p.rows_step;
  it.rows = min(p.rows_step, it.len * p.c.G - it.row0);
  it.kv_end = kv_end_of(p, it.ctx, it.len, it.rt);
  it.nt = tiles_up_to(p, it.kv_end);
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

__device__ __forceinline__ int tiles_of(const AttendParams& p, int ctx, int len, int rt) {
  return tiles_up_to(p, kv_end_of(p, ctx, len, rt));
}

__device__ __forceinline__ int warp_scan(int v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += up;
  }
  return v;
}

// Tiles of one KV head of sequence s, by one thread (few row tiles).
__device__ __forceinline__ int seq_tiles(const AttendParams& p, const SeqLens& s) {
  const int nrt = row_tiles(p, s.len);
  if (p.mask || nrt <= 1) return nrt * tiles_up_to(p, s.ctx + s.len);
  int n = 0;
  for (int rt = 0; rt < nrt; ++rt) n += tiles_of(p, s.ctx, s.len, rt);
  return n;
}

// The same by a whole warp, for causal calls of many row tiles.
__device__ __forceinline__ int seq_tiles_warp(const AttendParams& p, const SeqLens& s, int lane) {
  const int nrt = row_tiles(p, s.len);
  int n = 0;
  for (int rt = lane; rt < nrt; rt += 32) n += tiles_of(p, s.ctx, s.len, rt);
  return __reduce_add_sync(0xffffffffu, n);
}

// This CTA's run, worked out by every calling warp for itself: prefix sums over
// the sequences by shuffles, so that no warp waits for another.  The host
// bounds the call's units by 2^31.
__device__ __forceinline__ AttendRun find_run(const AttendParams& p, bool latch) {
  const int lane = threadIdx.x & 31;
  const int B = p.c.B, nkv = p.c.nkv;
  const bool wide = !p.mask && row_tiles(p, p.c.n_max) > 8;
  const int per = (B + 31) >> 5, b0 = min(B, lane * per), b1 = min(B, b0 + per);
  SeqLens s = {0, 0};  // of this lane's last sequence
  int mine = 0, rows = 0, layer, items;  // tiles and row tiles of one KV head: of this lane's sequences, of all
  if (wide) {
    layer = items = 0;
    for (int b = 0; b < B; ++b) {
      s = seq_lens(p.c, b, latch && lane == 0);
      layer += seq_tiles_warp(p, s, lane);
      items += row_tiles(p, s.len);
    }
  } else {
    for (int b = b0; b < b1; ++b) {
      s = seq_lens(p.c, b, latch);
      mine += seq_tiles(p, s);
      rows += row_tiles(p, s.len);
    }
    layer = __reduce_add_sync(0xffffffffu, mine);
    items = __reduce_add_sync(0xffffffffu, rows);
  }
  AttendRun r;
  // few tiles: every CTA gets one or two, whatever their items; else an item's
  // start and result weigh as much as item_cost tiles
  const int c = layer * nkv * p.c.Lc <= p.spread * p.n_cta ? 0 : p.item_cost;
  r.cost = c;
  layer += c * items;
  mine += c * rows;
  const int total = layer * nkv * p.c.Lc;
  r.chunk = max(1, p.by_ctas(total + p.n_cta - 1));
  const long long first = static_cast<long long>(blockIdx.x) * r.chunk;
  r.first = static_cast<int>(min(first, static_cast<long long>(total)));
  r.units = min(r.chunk, total - r.first);
  r.unit = 0;
  if (r.units <= 0) return r;
  const int l = p.c.Lc > 1 ? r.first / (layer * nkv) : 0;
  int rem = r.first - l * layer * nkv;  // unit within the layer
  // the sequence: prefix sums count one KV head, the order within a sequence is row tile, KV head
  int b = 0;
  if (wide) {
    for (;; ++b) {
      s = seq_lens(p.c, b, false);
      const int n = (seq_tiles_warp(p, s, lane) + c * row_tiles(p, s.len)) * nkv;
      if (rem < n) break;
      rem -= n;
    }
  } else {
    const int inc = warp_scan(mine, lane) * nkv;
    const int src = __ffs(__ballot_sync(0xffffffffu, inc > rem)) - 1;  // the lane whose sequences hold it
    rem -= __shfl_sync(0xffffffffu, inc - mine * nkv, src);
    b = src * per;
    if (per > 1) {
      for (;; ++b) {
        s = seq_lens(p.c, b, false);
        const int n = (seq_tiles(p, s) + c * row_tiles(p, s.len)) * nkv;
        if (rem < n) break;
        rem -= n;
      }
    } else {  // a sequence per lane: the lane has its lengths
      s.ctx = __shfl_sync(0xffffffffu, s.ctx, src);
      s.len = __shfl_sync(0xffffffffu, s.len, src);
    }
  }
  r.it.l = l;
  r.it.b = b;
  r.it.ctx = s.ctx;
  r.it.len = s.len;
  const int nrt = row_tiles(p, s.len);
  int rt = 0, nt = 0;  // nt: units of the row tile
  if (p.mask || nrt == 1) {
    nt = tiles_up_to(p, s.ctx + s.len) + c;
    if (nrt > 1) {
      rt = rem / (nt * nkv);
      rem -= rt * nt * nkv;
    }
  } else {
    for (int base = 0; base < nrt; base += 32) {  // the row tile that holds the remainder, 32 at a time
      const int t = base + lane < nrt ? tiles_of(p, s.ctx, s.len, base + lane) + c : 0;
      const int inc = warp_scan(t, lane) * nkv;
      const unsigned hit = __ballot_sync(0xffffffffu, inc > rem);
      if (hit) {
        const int src = __ffs(hit) - 1;
        rt = base + src;
        nt = __shfl_sync(0xffffffffu, t, src);
        rem -= __shfl_sync(0xffffffffu, inc, src) - nt * nkv;
        break;
      }
      rem -= __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  r.it.rt = rt;
  r.it.kh = nkv > 1 ? rem / nt : 0;
  r.unit = rem - r.it.kh * nt;
  set_item(p, r.it);
  return r;
}

// Pieces of a run, the same walk in every role: tiles t0 .. t1 - 1 of item `it`.
struct PieceWalk {
  AttendItem it;
  int t0, t1, unit, left, cost;  // unit: which of the item's units comes first; left: units of the run from there on
  __device__ __forceinline__ explicit PieceWalk(const AttendRun& r) : it(r.it), unit(r.unit), left(r.units), cost(r.cost) {
    if (left > 0) cut();
  }
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ void next(const AttendParams& p) {
    left -= cost + it.nt - unit;
    if (left <= 0) return;
    next_item(p, it);
    unit = 0;
    cut();
  }
  // global index of the item's first unit
  __device__ __forceinline__ int item_first(const AttendRun& r) const { return r.first + r.units - left - unit; }

 private:
  __device__ __forceinline__ void cut() {
    t0 = max(0, unit - cost);
    t1 = min(it.nt, unit + left - cost);
    if (t1 <= t0) left = 0;  // the run ends before the item's first tile, which the next CTA's takes
  }
};

// Partial result slot of a piece: a CTA has at most one piece that continues an
// item and one that starts an item without finishing it.
__device__ __forceinline__ int piece_slot(int cta, bool starts) { return cta * 2 + (starts ? 1 : 0); }

// Written once per run by one thread: the split item that this run starts, if any.
__device__ __forceinline__ void write_meta(const AttendParams& p, const AttendRun& r, bool starts_split,
                                           const AttendItem& it, int item_first) {
  SplitMeta m = {};
  m.last_cta = -1;
  if (starts_split) {
    m.last_cta = (item_first + r.cost + it.nt - 1) / r.chunk;
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
