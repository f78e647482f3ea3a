// sfa_paged_attend.cu — attention of new tokens over the paged cache on the
// CUDA cores, and the kernel that joins the pieces of split items.
#include <cuda_runtime.h>

#include <algorithm>

#include "sfa_paged.cuh"

namespace sfa {
namespace {

constexpr int kSimtThreads = 256;
constexpr int kSimtWarps = kSimtThreads / 32;
constexpr int kSimtKeys = 64;  // keys of a tile

// Shared memory: two stages of keys (rows padded by 16 bytes, so that the 32
// lanes' keys fall into different banks) and values, then q and P.
template <typename T, int D, int RPW>
struct SimtPlan {
  static constexpr int R = kSimtWarps * RPW;
  static constexpr int krow = D * static_cast<int>(sizeof(T)) + 16;
  static constexpr int kbytes = kSimtKeys * krow;
  static constexpr int vbytes = kSimtKeys * D * static_cast<int>(sizeof(T));
  static constexpr int stage = kbytes + vbytes;
  static constexpr int q = 2 * stage;
  static constexpr int pr = q + R * D * 4;
  static constexpr int total = pr + kSimtWarps * kSimtKeys * RPW * 4;
};

__device__ __forceinline__ void cp_async16_zfill(void* dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 16 : 0)
               : "memory");
}

// Keys and values of one tile into a stage; rows past the item's keys, and
// rows of a page out of range, are zero.
template <typename T, int D, int RPW>
__device__ __forceinline__ void simt_load(const AttendParams& p, const AttendItem& it, int tile, unsigned char* st) {
  using P = SimtPlan<T, D, RPW>;
  constexpr int CH = D * static_cast<int>(sizeof(T)) / 16;
  constexpr int EPC = 16 / static_cast<int>(sizeof(T));
  const T* kp = static_cast<const T*>(p.c.k_pages);
  const T* vp = static_cast<const T*>(p.c.v_pages);
  constexpr int N = kSimtKeys * CH / kSimtThreads;  // chunks of a thread
  long long off[N];  // -1: zeros; all page ids are asked for before the first copy
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int a = static_cast<int>(threadIdx.x) + i * kSimtThreads, row = a / CH, ch = a % CH;
    const int slot = tile * kSimtKeys + row;
    const int pg = slot < it.kv_end ? page_of(p.c, it.b, slot) : -1;
    off[i] = pg < 0 ? -1
                    : page_base<D>(p.c, p.c.l0 + it.l, pg, it.kh) + static_cast<long long>(slot & (p.c.ps - 1)) * D + ch * EPC;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int a = static_cast<int>(threadIdx.x) + i * kSimtThreads, row = a / CH, ch = a % CH;
    const bool in = off[i] >= 0;
    const long long o = in ? off[i] : 0;
    cp_async16_zfill(st + row * P::krow + ch * 16, kp + o, in);
    cp_async16_zfill(st + P::kbytes + row * D * static_cast<int>(sizeof(T)) + ch * 16, vp + o, in);
  }
}

// One CTA per run of tiles (sfa_paged.cuh).  A warp owns RPW rows and all 64
// keys of a tile: a lane scores keys lane and lane + 32, the row's maximum and
// sum are shuffles, P passes through the warp's own shared memory, and a lane
// then owns D / 32 output elements of its rows.  The running maximum, sum and
// output stay in fp32 registers.  Per tile a warp reads all keys and values
// once from shared memory for RPW rows, so RPW = 8 costs about as many
// shared-memory cycles as FMA cycles; few rows take a small RPW and are bound by
// the reads of keys and values from shared memory, once a warp.  Measured with
// 28/4 heads of 128: 37 sequences of one token over 2,048, 140 us (2.2 TB/s); two
// chunks of 256 tokens over 2,048, 457 us (31 TFLOP/s).
template <typename T, int D, int RPW>
__global__ void __launch_bounds__(kSimtThreads, 1) attend_simt_kernel(const __grid_constant__ AttendParams p) {
  using P = SimtPlan<T, D, RPW>;
  constexpr int DPL = D / 32;  // output elements of a lane
  extern __shared__ __align__(16) unsigned char smem[];
  pdl_trigger();
  pdl_wait();
  const AttendRun run = find_run(p, blockIdx.x == 0 && threadIdx.x < 32);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float* s_q = reinterpret_cast<float*>(smem + P::q);
  float* s_p = reinterpret_cast<float*>(smem + P::pr) + warp * kSimtKeys * RPW;
  bool wrote = false;
  for (PieceWalk w(run); w.more(); w.next(p)) {
    const AttendItem& it = w.it;
    const int t0 = w.t0, t1 = w.t1;
    // q of the item's rows, scaled to log2 units
    for (int a = tid; a < P::R * (D / 4); a += kSimtThreads) {
      const int r = a / (D / 4), d4 = (a - r * (D / 4)) * 4;
      float f[4] = {0.f, 0.f, 0.f, 0.f};
      if (r < it.rows) {
        const int row = it.row0 + r, node = p.by_group(row), g = row - node * p.c.G;
        const long long off = (((static_cast<long long>(it.l) * p.c.B + it.b) * p.c.n_max + node) * p.c.nq +
                               it.kh * p.c.G + g) * D + d4;
        VecLoad<T, 4>::run(static_cast<const T*>(p.q) + off, f);
      }
      *reinterpret_cast<float4*>(s_q + r * D + d4) =
          make_float4(f[0] * p.scale_log2, f[1] * p.scale_log2, f[2] * p.scale_log2, f[3] * p.scale_log2);
    }
    float m[RPW], l[RPW], o[RPW][DPL];
#pragma unroll
    for (int r = 0; r < RPW; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int e = 0; e < DPL; ++e) o[r][e] = 0.f;
    }
    simt_load<T, D, RPW>(p, it, t0, smem);
    cp_async_commit();
    for (int t = t0; t < t1; ++t) {
      if (t + 1 < t1) simt_load<T, D, RPW>(p, it, t + 1, smem + ((t + 1 - t0) & 1) * P::stage);
      cp_async_commit();
      cp_async_wait<1>();
      __syncthreads();
      const unsigned char* ks = smem + ((t - t0) & 1) * P::stage;
      const T* vs = reinterpret_cast<const T*>(ks + P::kbytes);
      float s[RPW][2];
#pragma unroll
      for (int r = 0; r < RPW; ++r) s[r][0] = s[r][1] = 0.f;
      const T* k0 = reinterpret_cast<const T*>(ks + lane * P::krow);
      const T* k1 = reinterpret_cast<const T*>(ks + (lane + 32) * P::krow);
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float a[4], b[4];
        VecLoad<T, 4>::run(k0 + d, a);
        VecLoad<T, 4>::run(k1 + d, b);
#pragma unroll
        for (int r = 0; r < RPW; ++r) {
          const float4 q = *reinterpret_cast<const float4*>(s_q + (warp * RPW + r) * D + d);
          s[r][0] = fmaf(q.x, a[0], fmaf(q.y, a[1], fmaf(q.z, a[2], fmaf(q.w, a[3], s[r][0]))));
          s[r][1] = fmaf(q.x, b[0], fmaf(q.y, b[1], fmaf(q.z, b[2], fmaf(q.w, b[3], s[r][1]))));
        }
      }
      const bool edge = (t + 1) * kSimtKeys > it.ctx;  // some key of the tile is not visible to all rows
      if (edge) {
#pragma unroll
        for (int r = 0; r < RPW; ++r) {
          const int node = min(p.by_group(it.row0 + warp * RPW + r), max(it.len - 1, 0));
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int rel = t * kSimtKeys + lane + 32 * u - it.ctx;
            if (rel >= 0 && !sees_new(p, it.b, node, it.len, rel)) s[r][u] = -INFINITY;
          }
        }
      }
      float mn[RPW];
#pragma unroll
      for (int r = 0; r < RPW; ++r) mn[r] = fmaxf(m[r], warp_max_redux(fmaxf(s[r][0], s[r][1])));
#pragma unroll
      for (int r = 0; r < RPW; ++r) {
        const float base = mn[r] == -INFINITY ? 0.f : mn[r];
        const float fix = exp2_approx(m[r] - base);
        const float p0 = exp2_approx(s[r][0] - base), p1 = exp2_approx(s[r][1] - base);
        m[r] = mn[r];
        l[r] = fmaf(l[r], fix, p0 + p1);
#pragma unroll
        for (int e = 0; e < DPL; ++e) o[r][e] *= fix;
        s_p[lane * RPW + r] = p0;
        s_p[(lane + 32) * RPW + r] = p1;
      }
      __syncwarp();
#pragma unroll 8
      for (int j = 0; j < kSimtKeys; ++j) {
        float v[DPL], w[RPW];
        VecLoad<T, DPL>::run(vs + j * D + lane * DPL, v);
#pragma unroll
        for (int r = 0; r < RPW; ++r) w[r] = s_p[j * RPW + r];
#pragma unroll
        for (int r = 0; r < RPW; ++r)
#pragma unroll
          for (int e = 0; e < DPL; ++e)
            // a new token that the row does not see may hold NaN: no product with it
            o[r][e] = edge && w[r] == 0.f ? o[r][e] : fmaf(w[r], v[e], o[r][e]);
      }
      __syncthreads();
    }
    cp_async_wait<0>();
    const bool starts = t0 == 0, whole = starts && t1 == it.nt;
    const int slot = piece_slot(static_cast<int>(blockIdx.x), starts);
#pragma unroll
    for (int r = 0; r < RPW; ++r) {
      const float sum = warp_sum(l[r]);
      const int rr = warp * RPW + r;
      if (rr >= it.rows) continue;
      if (whole) {
        const int row = it.row0 + rr, node = p.by_group(row), g = row - node * p.c.G;
        T* dst = static_cast<T*>(p.out) + (((static_cast<long long>(it.l) * p.c.B + it.b) * p.c.n_max + node) * p.c.nq +
                                           it.kh * p.c.G + g) * D + lane * DPL;
        const float inv = sum == 0.f ? 0.f : 1.0f / sum;  // a row that sees nothing is zero
#pragma unroll
        for (int e = 0; e < DPL; ++e) dst[e] = static_cast<T>(o[r][e] * inv);
      } else {
        const long long at = static_cast<long long>(slot) * p.rows_step + rr;
        if (lane == 0) *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(m[r], sum);
#pragma unroll
        for (int e = 0; e < DPL; ++e) p.part_o[at * D + lane * DPL + e] = o[r][e];
      }
    }
    if (starts && !whole) {
      if (tid == 0) write_meta(p, run, true, it, w.item_first(run));
      wrote = true;
    }
    __syncthreads();  // q and the stages are reused
  }
  if (!wrote && tid == 0) write_meta(p, run, false, run.it, 0);
}

// Joins the pieces of split items: a warp per row, in the order of the pieces,
// so results do not depend on timing.  Block (c, y) serves rows 8 y .. of the
// split item that CTA c's run starts.  Bound by its own latency: released 1.3 us
// after the last CTA of the attention, done 1 to 2 us later.
template <typename T, int D>
__global__ void __launch_bounds__(256) attend_combine_kernel(const __grid_constant__ AttendParams p) {
  constexpr int DPL = D / 32;
  pdl_trigger();
  pdl_wait();
  const int c = static_cast<int>(blockIdx.x), lane = threadIdx.x & 31;
  const SplitMeta m = p.meta[c];
  const int r = static_cast<int>(blockIdx.y) * 8 + (threadIdx.x >> 5);
  if (m.last_cta < 0 || r >= m.rows) return;
  auto at = [&](int piece) {  // piece 0 is CTA c's, the rest continue it
    return static_cast<long long>(piece_slot(c + piece, piece == 0)) * p.rows_step + r;
  };
  const int np = m.last_cta - c + 1;
  float mx = -INFINITY;
  for (int i = lane; i < np; i += 32) mx = fmaxf(mx, p.part_ml[at(i) * 2]);
  mx = warp_max(mx);
  const float base = mx == -INFINITY ? 0.f : mx;
  float sum = 0.f, o[DPL];
#pragma unroll
  for (int e = 0; e < DPL; ++e) o[e] = 0.f;
#pragma unroll 4
  for (int i = 0; i < np; ++i) {
    const long long a = at(i);
    const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + a * 2);
    const float w = exp2_approx(ml.x - base);
    float v[DPL];
    VecLoad<float, DPL>::run(p.part_o + a * D + lane * DPL, v);
    const bool some = ml.y != 0.f;  // a piece without visible keys holds nothing
    sum = some ? fmaf(ml.y, w, sum) : sum;
#pragma unroll
    for (int e = 0; e < DPL; ++e) o[e] = some ? fmaf(v[e], w, o[e]) : o[e];
  }
  const float inv = sum == 0.f ? 0.f : 1.0f / sum;
  const int row = m.row0 + r, node = p.by_group(row), g = row - node * p.c.G;
  T* dst = static_cast<T*>(p.out) + (((static_cast<long long>(m.l) * p.c.B + m.b) * p.c.n_max + node) * p.c.nq +
                                     m.kh * p.c.G + g) * D + lane * DPL;
#pragma unroll
  for (int e = 0; e < DPL; ++e) dst[e] = static_cast<T>(o[e] * inv);
}

template <typename K>
cudaError_t launch_pdl(K kernel, dim3 grid, int threads, int smem, const AttendParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

int simt_rpw(int rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 32 ? 4 : 8; }

template <typename T, int D, int RPW>
cudaError_t launch_simt(const AttendParams& p, cudaStream_t s) {
  return launch_pdl(attend_simt_kernel<T, D, RPW>, dim3(static_cast<unsigned>(p.n_cta), 1, 1), kSimtThreads,
                    SimtPlan<T, D, RPW>::total, p, s);
}

template <int D>
cudaError_t launch_simt_rows(const AttendParams& p, cudaStream_t s) {
  switch (p.rows_step / kSimtWarps) {
    case 1: return launch_simt<float, D, 1>(p, s);
    case 2: return launch_simt<float, D, 2>(p, s);
    case 4: return launch_simt<float, D, 4>(p, s);
    default: return launch_simt<float, D, 8>(p, s);
  }
}

template <typename T, int D>
cudaError_t launch_combine(const AttendParams& p, cudaStream_t s) {
  const long long rows = std::min<long long>(p.rows_step, static_cast<long long>(p.c.n_max) * p.c.G);
  return launch_pdl(attend_combine_kernel<T, D>,
                    dim3(static_cast<unsigned>(p.n_cta), static_cast<unsigned>((rows + 7) / 8), 1), 256, 0, p, s);
}

template <int D, int RPW>
cudaError_t allow() {
  return cudaFuncSetAttribute(attend_simt_kernel<float, D, RPW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              SimtPlan<float, D, RPW>::total);
}
template <int D>
cudaError_t allow_all() {
  cudaError_t e = allow<D, 1>();
  if (e == cudaSuccess) e = allow<D, 2>();
  if (e == cudaSuccess) e = allow<D, 4>();
  if (e == cudaSuccess) e = allow<D, 8>();
  return e;
}

}  // namespace

AttendPlan attend_plan(int in_dtype, int head_dim, int G, int n_max, int n_sm) {
  AttendPlan a;
  if (in_dtype == SFA_F32) {
    a.kt = kSimtKeys;
    a.item_cost = kAttendItemCost;
    a.rows_step = kSimtWarps * simt_rpw(static_cast<int>(std::min<long long>(static_cast<long long>(n_max) * G, 64)));
  } else {
    attend_tc_rows(G, n_max, &a);
  }
  a.n_cta = n_sm;
  a.off_ml = static_cast<size_t>(align256(static_cast<long long>(sizeof(SplitMeta)) * a.n_cta));
  a.off_o = a.off_ml + static_cast<size_t>(align256(16LL * a.n_cta * a.rows_step));
  a.total = a.off_o + static_cast<size_t>(align256(8LL * a.n_cta * a.rows_step * head_dim));
  return a;
}

cudaError_t attend_prepare(int device) {
  (void)device;
  cudaError_t e = allow_all<64>();
  if (e == cudaSuccess) e = allow_all<128>();
  if (e == cudaSuccess) e = attend_tc_prepare();
  return e;
}

cudaError_t launch_kv_attend(const AttendParams& p, int in_dtype, int head_dim, cudaStream_t s) {
  cudaError_t e;
  if (in_dtype == SFA_F32)
    e = head_dim == 64 ? launch_simt_rows<64>(p, s) : launch_simt_rows<128>(p, s);
  else
    e = launch_attend_tc(p, head_dim, s);
  if (e != cudaSuccess) return e;
  if (in_dtype == SFA_F32) return head_dim == 64 ? launch_combine<float, 64>(p, s) : launch_combine<float, 128>(p, s);
  return head_dim == 64 ? launch_combine<__nv_bfloat16, 64>(p, s) : launch_combine<__nv_bfloat16, 128>(p, s);
}

}  // namespace sfa
