// sfa_paged.cu — the paged cache calls around the attention: masks and
// positions of drafted trees, append with rotation, and the accepted path.
#include <cuda_runtime.h>

#include "sfa_paged.cuh"

namespace sfa {
namespace {

constexpr int kPlanThreads = 128;
constexpr int kAppendThreads = 128;
constexpr int kAppendAhead = 3;  // rows of a lane in flight
constexpr int kAcceptThreads = 128;
constexpr int kAcceptBatch = 8;

// One CTA per sequence, nodes over threads.  A node's ancestors have smaller
// indices, so one walk up the parents meets them in falling order and writes
// each finished mask word once.  The walk is a chain of shared-memory reads:
// the depth of the tree bounds the kernel, besides its launch (256 trees of 64
// nodes: 3.5 us).
__global__ void __launch_bounds__(kPlanThreads) tree_plan_kernel(PlanParams p) {
  __shared__ int s_par[SFA_TREE_MAX];
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.x;
  const int ctx = p.ctx[b];
  const int len = p.lens ? p.lens[b] : p.n_max;
  bool ok = ctx >= 0 && len >= 0 && len <= p.n_max && ctx <= 0x7fffffff - len;  // positions fit 32 bits
  if (ok)
    for (int i = threadIdx.x; i < len; i += kPlanThreads) {
      const int q = p.parents[static_cast<long long>(b) * p.n_max + i];
      s_par[i] = q;
      if (q < -1 || q >= i) ok = false;
    }
  if (!__syncthreads_and(ok)) {
    if (threadIdx.x == 0) latch_error(p.err, SFA_ERR_INVALID_ARG);
    return;
  }
  for (int i = threadIdx.x; i < len; i += kPlanThreads) {
    const long long row = static_cast<long long>(b) * p.n_max + i;
    uint32_t* m = p.mask ? p.mask + row * p.words : nullptr;
    if (m)
      for (int w = p.words - 1; w > (i >> 5); --w) m[w] = 0u;
    int depth = -1, w = i >> 5;
    uint32_t bits = 0u;
    for (int j = i; j >= 0; j = s_par[j]) {
      ++depth;
      if ((j >> 5) != w) {
        if (m) {
          m[w] = bits;
          for (--w; w > (j >> 5); --w) m[w] = 0u;
        }
        w = j >> 5;
        bits = 0u;
      }
      bits |= 1u << (j & 31);
    }
    if (m) {
      m[w] = bits;
      for (--w; w >= 0; --w) m[w] = 0u;
    }
    if (p.positions) p.positions[row] = ctx + depth;
  }
}

// Rotation of one 16-byte chunk pair.  HALF: a[e] pairs with b[e]; PAIRS:
// neighbours within a chunk.  cs holds (cos, sin) of the token's pairs.
template <typename T>
__device__ __forceinline__ uint4 pack16(const float* f);
template <>
__device__ __forceinline__ uint4 pack16<float>(const float* f) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
template <>
__device__ __forceinline__ uint4 pack16<__nv_bfloat16>(const float* f) {
  uint4 r;
  unsigned* w = &r.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const unsigned*>(&v);
  }
  return r;
}
template <typename T>
__device__ __forceinline__ void unpack16(const uint4& r, float* f) {
  Load16<T>::run(reinterpret_cast<const T*>(&r), f);
}

// A warp per token.  A task is a pair of 16-byte chunks of one head row (q heads,
// then keys, then values): TPH neighbouring lanes share a row, so that accesses
// are whole 128-byte lines, and a lane keeps its chunks and steps over the rows,
// kAppendAhead of them loaded before the first is used.  The token's angles are
// computed once, D / 64 of them by a lane, and handed round by shuffles: turns
// p * f_j in 64 bits less their whole part, then sine and cosine of the rest in
// fp32.  Nothing is shared between warps, so that the other warps of the SM
// cover the chain from the lengths over the page table to the stores (65,536
// tokens of 28 + 4 + 4 heads of 128, half of them past their sequence's length:
// 72 us, 6.0 TB/s; tokens in groups of 8 that share their angles in shared
// memory took 121 us).
template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int V = 16 / static_cast<int>(sizeof(T));  // elements of a chunk
  constexpr int TPH = D / (2 * V);                     // lanes of a row
  constexpr int RPW = 32 / TPH;                        // rows of one pass
  constexpr int NA = D / 64;                           // angles of a lane
  const PagedParams& c = p.c;
  const int lane = threadIdx.x & 31;
  const long long t = static_cast<long long>(blockIdx.x) * (kAppendThreads / 32) + (threadIdx.x >> 5);
  pdl_trigger();
  pdl_wait();
  if (t >= static_cast<long long>(c.Lc) * c.B * c.n_max) return;
  const int lb = static_cast<int>(t / c.n_max), i = static_cast<int>(t - static_cast<long long>(lb) * c.n_max);
  const int l = lb / c.B, b = lb - l * c.B;
  const SeqLens sl = seq_lens(c, b, i == 0 && lane == 0);
  if (i >= sl.len) return;
  const int slot = sl.ctx + i;
  const int pg = page_of(c, b, slot, lane == 0);
  const long long dst = page_base<D>(c, c.l0 + l, max(pg, 0), 0) + static_cast<long long>(slot & (c.ps - 1)) * D;

  const int rc = p.dims / V;  // chunks of a row that are rotated
  // the two chunks of this lane: a rotated pair of halves, or neighbours
  const int ch = lane % TPH;
  const bool halves = p.style == SFA_ROPE_HALF && ch < rc / 2;
  const int c0 = halves ? ch : 2 * ch, c1 = halves ? ch + rc / 2 : 2 * ch + 1;
  const bool turns_here = c0 < rc;
  float co[V], si[V];  // of this lane's V pairs
  if (p.dims > 0) {
    const int pos = p.positions ? p.positions[static_cast<long long>(b) * c.n_max + i] : slot;
    float mc[NA], ms[NA];
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      const double turns = static_cast<double>(pos) * p.turns[lane * NA + a];  // zero past dims / 2
      sincospif(2.0f * static_cast<float>(turns - rint(turns)), &ms[a], &mc[a]);
    }
    const int first = p.style == SFA_ROPE_HALF ? c0 * V : c0 * V / 2;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int j = first + e;
      co[e] = __shfl_sync(0xffffffffu, mc[e % NA], j / NA);
      si[e] = __shfl_sync(0xffffffffu, ms[e % NA], j / NA);
    }
  }
  const int qh = p.q ? c.nq : 0, heads = qh + 2 * c.nkv;
  for (int h0 = lane / TPH; h0 < heads; h0 += RPW * kAppendAhead) {
    uint4 x0[kAppendAhead], x1[kAppendAhead];
#pragma unroll
    for (int u = 0; u < kAppendAhead; ++u) {
      const int hd = h0 + u * RPW;
      if (hd >= heads) break;
      const T* src = hd < qh ? static_cast<const T*>(p.q) + (t * c.nq + hd) * D
                   : hd < qh + c.nkv ? static_cast<const T*>(p.k) + (t * c.nkv + hd - qh) * D
                                     : static_cast<const T*>(p.v) + (t * c.nkv + hd - qh - c.nkv) * D;
      x0[u] = *reinterpret_cast<const uint4*>(src + c0 * V);
      x1[u] = *reinterpret_cast<const uint4*>(src + c1 * V);
    }
#pragma unroll
    for (int u = 0; u < kAppendAhead; ++u) {
      const int hd = h0 + u * RPW;
      if (hd >= heads) break;
      T* dst0 = nullptr;  // token-major output
      T* dst1 = nullptr;  // page
      if (hd < qh) {
        dst0 = static_cast<T*>(p.q_out) + (t * c.nq + hd) * D;
      } else if (hd < qh + c.nkv) {
        if (p.k_out) dst0 = static_cast<T*>(p.k_out) + (t * c.nkv + hd - qh) * D;
        if (pg >= 0) dst1 = static_cast<T*>(c.k_pages) + dst + static_cast<long long>(hd - qh) * c.ps * D;
      } else if (pg >= 0) {
        dst1 = static_cast<T*>(c.v_pages) + dst + static_cast<long long>(hd - qh - c.nkv) * c.ps * D;
      }
      if (hd < qh + c.nkv && turns_here) {
        float f0[V], f1[V];
        unpack16<T>(x0[u], f0);
        unpack16<T>(x1[u], f1);
        if (p.style == SFA_ROPE_HALF) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float a0 = f0[e], a1 = f1[e];
            f0[e] = a0 * co[e] - a1 * si[e];
            f1[e] = a1 * co[e] + a0 * si[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < V; e += 2) {
            const int j = e / 2, k = V / 2 + e / 2;
            const float a0 = f0[e], a1 = f0[e + 1], b0 = f1[e], b1 = f1[e + 1];
            f0[e] = a0 * co[j] - a1 * si[j];
            f0[e + 1] = a1 * co[j] + a0 * si[j];
            f1[e] = b0 * co[k] - b1 * si[k];
            f1[e + 1] = b1 * co[k] + b0 * si[k];
          }
        }
        x0[u] = pack16<T>(f0);
        x1[u] = pack16<T>(f1);
      }
      if (dst0) {
        *reinterpret_cast<uint4*>(dst0 + c0 * V) = x0[u];
        *reinterpret_cast<uint4*>(dst0 + c1 * V) = x1[u];
      }
      if (dst1) {
        *reinterpret_cast<uint4*>(dst1 + c0 * V) = x0[u];
        *reinterpret_cast<uint4*>(dst1 + c1 * V) = x1[u];
      }
    }
  }
}

// One CTA per (layer, sequence); a thread owns 16-byte columns of (K or V, KV
// head) and moves the path's rows of its column in order, kAcceptBatch loads
// ahead of their stores.  path[i] >= i and rising, so a row is never read
// after it has been overwritten: every later source lies behind every
// earlier destination.  Bound by its launch and the reads path -> page -> rows (32
// sequences, 28 layers of 4 heads of 128: 4.2 us).
template <typename T, int D>
__global__ void __launch_bounds__(kAcceptThreads) accept_kernel(const __grid_constant__ AcceptParams p) {
  constexpr int CH = D * static_cast<int>(sizeof(T)) / 16;
  constexpr int V = 16 / static_cast<int>(sizeof(T));
  __shared__ long long s_src[SFA_TREE_MAX], s_dst[SFA_TREE_MAX];
  const PagedParams& c = p.c;
  pdl_trigger();
  pdl_wait();
  const int b = static_cast<int>(blockIdx.x) % c.B, l = static_cast<int>(blockIdx.x) / c.B;
  const int n = p.n_accept[b], ctx = c.ctx[b];
  bool ok = n >= 0 && n <= c.n_max && ctx >= 0;
  if (ok) {
    const int* path = p.path + static_cast<long long>(b) * c.n_max;
    const long long room = static_cast<long long>(c.max_pages) * c.ps;
    for (int i = threadIdx.x; i < n; i += kAcceptThreads) {
      const int s = path[i];
      const bool in = s >= 0 && s < c.n_max && (i == 0 || path[i - 1] < s) && static_cast<long long>(ctx) + s < room;
      long long src = -1, dst = -1;
      if (in && s != i) {  // a rising path has path[i] >= i
        const int ps = page_of(c, b, ctx + s), pd = s > i ? page_of(c, b, ctx + i) : -1;
        if (ps >= 0 && pd >= 0) {
          src = page_base<D>(c, c.l0 + l, ps, 0) + static_cast<long long>((ctx + s) & (c.ps - 1)) * D;
          dst = page_base<D>(c, c.l0 + l, pd, 0) + static_cast<long long>((ctx + i) & (c.ps - 1)) * D;
        }
      }
      s_src[i] = src;
      s_dst[i] = dst;
      ok = ok && in;
    }
  }
  if (!__syncthreads_and(ok)) {
    if (threadIdx.x == 0) latch_error(c.err, SFA_ERR_INVALID_ARG);
    return;
  }
  const int cols = 2 * c.nkv * CH;
  for (int a = threadIdx.x; a < cols; a += kAcceptThreads) {
    const int kh = (a / CH) % c.nkv;
    T* base = static_cast<T*>(a >= c.nkv * CH ? c.v_pages : c.k_pages) + static_cast<long long>(kh) * c.ps * D + (a % CH) * V;
    for (int i0 = 0; i0 < n; i0 += kAcceptBatch) {
      uint4 r[kAcceptBatch];
#pragma unroll
      for (int u = 0; u < kAcceptBatch; ++u)
        if (i0 + u < n && s_src[i0 + u] >= 0) r[u] = *reinterpret_cast<const uint4*>(base + s_src[i0 + u]);
#pragma unroll
      for (int u = 0; u < kAcceptBatch; ++u)
        if (i0 + u < n && s_src[i0 + u] >= 0) *reinterpret_cast<uint4*>(base + s_dst[i0 + u]) = r[u];
    }
  }
}

template <typename K, typename P>
cudaError_t launch_pdl(K kernel, dim3 grid, int threads, const P& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename T, int D>
cudaError_t launch_append_t(const AppendParams& p, unsigned grid, cudaStream_t s) {
  return launch_pdl(append_kernel<T, D>, dim3(grid, 1, 1), kAppendThreads, p, s);
}

}  // namespace

cudaError_t launch_tree_plan(const PlanParams& p, cudaStream_t s) {
  return launch_pdl(tree_plan_kernel, dim3(static_cast<unsigned>(p.B), 1, 1), kPlanThreads, p, s);
}

cudaError_t launch_kv_append(const AppendParams& p, int in_dtype, int head_dim, cudaStream_t s) {
  const long long total = static_cast<long long>(p.c.Lc) * p.c.B * p.c.n_max;
  const long long grid = (total + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
  const unsigned g = static_cast<unsigned>(grid);
  if (in_dtype == SFA_F32)
    return head_dim == 64 ? launch_append_t<float, 64>(p, g, s) : launch_append_t<float, 128>(p, g, s);
  return head_dim == 64 ? launch_append_t<__nv_bfloat16, 64>(p, g, s) : launch_append_t<__nv_bfloat16, 128>(p, g, s);
}

cudaError_t launch_kv_accept(const AcceptParams& p, int in_dtype, int head_dim, cudaStream_t s) {
  const dim3 g(static_cast<unsigned>(p.c.Lc) * static_cast<unsigned>(p.c.B), 1, 1);
  if (in_dtype == SFA_F32)
    return head_dim == 64 ? launch_pdl(accept_kernel<float, 64>, g, kAcceptThreads, p, s)
                          : launch_pdl(accept_kernel<float, 128>, g, kAcceptThreads, p, s);
  return head_dim == 64 ? launch_pdl(accept_kernel<__nv_bfloat16, 64>, g, kAcceptThreads, p, s)
                        : launch_pdl(accept_kernel<__nv_bfloat16, 128>, g, kAcceptThreads, p, s);
}

}  // namespace sfa
