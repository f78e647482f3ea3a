// sfa_paged.cu — the paged cache calls around the attention: masks and
// positions of drafted trees, append with rotation, and the accepted path.
#include <cuda_runtime.h>

#include <algorithm>

#include "sfa_paged.cuh"

namespace sfa {
namespace {

constexpr int kPlanThreads = 128;
constexpr int kAppendThreads = 256;
constexpr int kAppendMaxTokens = 8;
constexpr int kAcceptThreads = 128;
constexpr int kAcceptBatch = 8;

// One CTA per sequence, nodes over threads.  A node's ancestors have smaller
// indices, so one walk up the parents meets them in falling order and writes
// each finished mask word once.  The walk is a chain of shared-memory reads:
// the depth of the tree bounds the kernel, besides its launch.
__global__ void __launch_bounds__(kPlanThreads) tree_plan_kernel(PlanParams p) {
  __shared__ int s_par[SFA_TREE_MAX];
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.x;
  const int ctx = p.ctx[b];
  const int len = p.lens ? p.lens[b] : p.n_max;
  bool ok = ctx >= 0 && len >= 0 && len <= p.n_max;
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

// Tokens of the call in runs of tokens_per_cta; a task is one pair of 16-byte
// chunks of one head of one token: q heads, then keys, then values.  The
// angles of a token are computed once for its n_q + n_kv heads: turns p * f_j
// in 64 bits less their whole part, then sine and cosine of the rest in fp32.
template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int V = 16 / static_cast<int>(sizeof(T));  // elements of a chunk
  constexpr int TPH = D / (2 * V);                     // tasks of a head
  __shared__ float2 s_cs[kAppendMaxTokens][D / 2];
  __shared__ long long s_dst[kAppendMaxTokens];        // row offset in kv head 0 of the page; -1: not written
  __shared__ int s_live[kAppendMaxTokens];
  const PagedParams& c = p.c;
  pdl_trigger();
  pdl_wait();
  const long long total = static_cast<long long>(c.Lc) * c.B * c.n_max;
  const long long t0 = static_cast<long long>(blockIdx.x) * p.tokens_per_cta;
  const int nt = static_cast<int>(min(static_cast<long long>(p.tokens_per_cta), total - t0));
  if (static_cast<int>(threadIdx.x) < nt) {
    const long long t = t0 + threadIdx.x;
    const int i = static_cast<int>(t % c.n_max);
    const long long lb = t / c.n_max;
    const int b = static_cast<int>(lb % c.B), l = static_cast<int>(lb / c.B);
    const SeqLens sl = seq_lens(c, b, i == 0);
    s_live[threadIdx.x] = i < sl.len;
    if (i < sl.len) {
      const int slot = sl.ctx + i;
      const int pg = page_of(c, b, slot);
      s_dst[threadIdx.x] = pg < 0 ? -1 : page_base<D>(c, c.l0 + l, pg, 0) + static_cast<long long>(slot & (c.ps - 1)) * D;
    }
  }
  const int half = p.dims / 2;
  for (int a = threadIdx.x; a < nt * half; a += kAppendThreads) {
    const int tt = a / half, j = a - tt * half;
    const long long t = t0 + tt;
    const long long lb = t / c.n_max;
    const int b = static_cast<int>(lb % c.B), i = static_cast<int>(t - lb * c.n_max);
    const int pos = p.positions ? p.positions[static_cast<long long>(b) * c.n_max + i] : c.ctx[b] + i;
    const double turns = static_cast<double>(pos) * p.turns[j];
    float s, co;
    sincospif(2.0f * static_cast<float>(turns - rint(turns)), &s, &co);
    s_cs[tt][j] = make_float2(co, s);
  }
  __syncthreads();
  const int heads = (p.q ? c.nq : 0) + 2 * c.nkv;
  const int qh = p.q ? c.nq : 0;
  const int tasks = nt * heads * TPH;
  const int rc = p.dims / V;  // chunks of a head that are rotated
  for (int a = threadIdx.x; a < tasks; a += kAppendThreads) {
    const int th = a / TPH, ch = a - th * TPH;
    const int tt = th / heads, head = th - tt * heads;
    if (!s_live[tt]) continue;
    const long long t = t0 + tt;
    const T* src;
    T* dst0 = nullptr;  // token-major output
    T* dst1 = nullptr;  // page
    const long long pg = s_dst[tt];
    bool rot = true;
    if (head < qh) {
      const long long off = (t * c.nq + head) * D;
      src = static_cast<const T*>(p.q) + off;
      dst0 = static_cast<T*>(p.q_out) + off;
    } else if (head < qh + c.nkv) {
      const int kh = head - qh;
      const long long off = (t * c.nkv + kh) * D;
      src = static_cast<const T*>(p.k) + off;
      if (p.k_out) dst0 = static_cast<T*>(p.k_out) + off;
      if (pg >= 0) dst1 = static_cast<T*>(c.k_pages) + pg + static_cast<long long>(kh) * c.ps * D;
    } else {
      const int kh = head - qh - c.nkv;
      src = static_cast<const T*>(p.v) + (t * c.nkv + kh) * D;
      if (pg >= 0) dst1 = static_cast<T*>(c.v_pages) + pg + static_cast<long long>(kh) * c.ps * D;
      rot = false;
    }
    // the two chunks of this task: a rotated pair of halves, or neighbours
    int c0, c1;
    if (p.style == SFA_ROPE_HALF && ch < rc / 2) {
      c0 = ch;
      c1 = ch + rc / 2;
    } else {
      c0 = 2 * ch;
      c1 = c0 + 1;
    }
    uint4 x0 = *reinterpret_cast<const uint4*>(src + c0 * V);
    uint4 x1 = *reinterpret_cast<const uint4*>(src + c1 * V);
    if (rot && c0 < rc) {
      float f0[V], f1[V];
      unpack16<T>(x0, f0);
      unpack16<T>(x1, f1);
      if (p.style == SFA_ROPE_HALF) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float2 cs = s_cs[tt][c0 * V + e];
          const float a0 = f0[e], a1 = f1[e];
          f0[e] = a0 * cs.x - a1 * cs.y;
          f1[e] = a1 * cs.x + a0 * cs.y;
        }
      } else {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          const float2 u = s_cs[tt][(c0 * V + e) / 2], w = s_cs[tt][(c1 * V + e) / 2];
          const float a0 = f0[e], a1 = f0[e + 1], b0 = f1[e], b1 = f1[e + 1];
          f0[e] = a0 * u.x - a1 * u.y;
          f0[e + 1] = a1 * u.x + a0 * u.y;
          f1[e] = b0 * w.x - b1 * w.y;
          f1[e + 1] = b1 * w.x + b0 * w.y;
        }
      }
      x0 = pack16<T>(f0);
      x1 = pack16<T>(f1);
    }
    if (dst0) {
      *reinterpret_cast<uint4*>(dst0 + c0 * V) = x0;
      *reinterpret_cast<uint4*>(dst0 + c1 * V) = x1;
    }
    if (dst1) {
      *reinterpret_cast<uint4*>(dst1 + c0 * V) = x0;
      *reinterpret_cast<uint4*>(dst1 + c1 * V) = x1;
    }
  }
}

// One CTA per (layer, sequence); a thread owns 16-byte columns of (K or V, KV
// head) and moves the path's rows of its column in order, kAcceptBatch loads
// ahead of their stores.  path[i] >= i and rising, so a row is never read
// after it has been overwritten: every later source lies behind every
// earlier destination.
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

cudaError_t launch_kv_append(const AppendParams& in, int in_dtype, int head_dim, int n_sm, cudaStream_t s) {
  AppendParams p = in;
  const long long total = static_cast<long long>(p.c.Lc) * p.c.B * p.c.n_max;
  // one token per CTA while the tokens do not fill the card twice, then more
  p.tokens_per_cta = static_cast<int>(std::min<long long>(kAppendMaxTokens, std::max<long long>(1, total / (8LL * n_sm))));
  const long long grid = (total + p.tokens_per_cta - 1) / p.tokens_per_cta;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
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
