// Gated feed-forward for few rows (tokens): y = act(x Wg^T) * (x Wu^T).
//
// Every weight is used a few times only, so the bytes of W bound the product.
//
// bfloat16 rows that 16-byte copies can read: a warp streams tiles of 8
// features -- their 8 gate rows and 8 up rows of W, 128 bytes (64 k) each --
// through its own ring of asynchronous copies and multiplies them on the tensor
// cores (m16n8k16: the 16 rows as M, the tokens as N).  Gate rows take the
// upper half of a tile and up rows the lower, so that both pre-activations of
// an output are in one thread.  The order of k inside a product is free: a
// lane's 16-byte piece is operand as it lies.  The eight warps of a block split
// K; where x does not fit shared memory the blocks of a cluster split it
// further.  Sums are joined in a fixed order in float32; one rounding.
//
// Other rows (float32, or a K that is no multiple of 8): fused multiply-adds,
// a warp taking two features and up to eight tokens at a time, the lanes
// splitting K.
#include <algorithm>

#include "common.cuh"
#include "glu.cuh"
#include "ops.h"

namespace lr {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kStages = 4;
constexpr int kStageBytes = 16 * 128;
constexpr int kXBytes = 64 * 1024;  // x of one block at most

struct RowsP {
  int M, K, F, nkb, tiles, tok, act;
  const bf16* x;
  const bf16* W;
  bf16* y;
  uint32_t x_bytes;
};

__device__ __forceinline__ uint32_t smem_at(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ unsigned cl_size() {
  unsigned n;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return n;
}
__device__ __forceinline__ unsigned cl_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cl_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
               "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_rank0(float2* local, float a, float b) {
  unsigned addr;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(addr) : "r"(smem_at(local)));
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(a), "f"(b) : "memory");
}

// NT: token tiles of 8
template <int NT>
__global__ void __launch_bounds__(kThreads) glu_rows_kernel(const RowsP p) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int kCols = 8 * NT;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const unsigned csize = cl_size(), rank = cl_rank();
  const int m0 = blockIdx.y * p.tok, toks = min(p.tok, p.M - m0);
  const int kb0 = (int)((int64_t)rank * p.nkb / csize), kb1 = (int)((int64_t)(rank + 1) * p.nkb / csize);
  const int clusters = gridDim.x / csize, first = blockIdx.x / csize;
  const int per = (kb1 - kb0 + kWarps - 1) / kWarps;
  const int items = (first < p.tiles ? (p.tiles - 1 - first) / clusters + 1 : 0) * per;
  unsigned char* ring = smem + p.x_bytes + warp * (kStages * kStageBytes);
  float* red = reinterpret_cast<float*>(smem + p.x_bytes + kWarps * kStages * kStageBytes);
  float2* gather = reinterpret_cast<float2*>(red + 2 * kWarps * 16 * kCols);
  const uint32_t ring_at = smem_at(ring), xs_at = smem_at(smem);

  int it_tile = first, it_kb = 0;
  // 16-byte piece c of row r at piece c ^ swz(r): eight lanes that read one
  // piece column of two rows touch all banks
  auto swz = [](int r) { return ((r & 1) << 2) | ((r >> 1) & 3); };
  auto issue = [&](int s) {
    const int kb = kb0 + it_kb * kWarps + warp;
    if (it_tile < p.tiles && kb < kb1) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = j * 4 + (lane >> 3), c = lane & 7;
        const int f = it_tile * 8 + (row & 7), k = kb * 64 + c * 8;
        const bool ok = f < p.F && k < p.K;
        copy16(ring_at + s * kStageBytes + row * 128 + ((c ^ swz(row)) << 4),
               p.W + (ok ? (int64_t)(row < 8 ? f : p.F + f) * p.K + k : 0), ok);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (++it_kb == per) { it_kb = 0; it_tile += clusters; }
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) issue(s);

  // x: 16-byte piece (block of 64 k, half h, token, t) holds k = 64 kb + 8 (t + 4 h)
  for (int i = threadIdx.x; i < (kb1 - kb0) * 8 * toks; i += kThreads) {
    const int c = i & 7, r = i >> 3, kb = r / toks, m = r - kb * toks;
    const int k = (kb0 + kb) * 64 + c * 8;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (k < p.K) v = __ldg(reinterpret_cast<const uint4*>(p.x + (int64_t)(m0 + m) * p.K + k));
    reinterpret_cast<uint4*>(smem)[((kb * 2 + (c >> 2)) * toks + m) * 4 + (c & 3)] = v;
  }
  __syncthreads();

  float acc[NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[nt][i] = 0.f;
  int tile = first, kbi = 0, par = 0;
  const uint32_t row_at = ring_at + g * 128;
  for (int it = 0, s = 0; it < items; ++it, s = s + 1 == kStages ? 0 : s + 1) {
    issue(s == 0 ? kStages - 1 : s - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();
    const int kb = kb0 + kbi * kWarps + warp;
    if (kb < kb1) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t at = row_at + s * kStageBytes + (((t + 4 * h) ^ swz(g)) << 4);
        const uint4 a = lds128(at), b = lds128(at + 1024);
        const uint32_t xa = xs_at + (uint32_t)((((kb - kb0) * 2 + h) * toks + g) * 4 + t) * 16;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (nt * 8 + g < toks) v = lds128(xa + nt * 512);
          mma(acc[nt], a.x, b.x, a.y, b.y, v.x, v.y);
          mma(acc[nt], a.z, b.z, a.w, b.w, v.z, v.w);
        }
      }
    }
    __syncwarp();
    if (++kbi < per) continue;
    kbi = 0;
    float* rw = red + par * (kWarps * 16 * kCols);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float* d = rw + (warp * 16 + g) * kCols + nt * 8 + 2 * t;
      *reinterpret_cast<float2*>(d) = make_float2(acc[nt][0], acc[nt][1]);
      *reinterpret_cast<float2*>(d + 8 * kCols) = make_float2(acc[nt][2], acc[nt][3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[nt][i] = 0.f;
    }
    __syncthreads();
    const int f0 = tile * 8;
    for (int i = threadIdx.x; i < 8 * toks; i += kThreads) {
      const int r = i & 7, m = i >> 3;
      float gv = 0.f, uv = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        gv += rw[(w * 16 + r) * kCols + m];
        uv += rw[(w * 16 + 8 + r) * kCols + m];
      }
      if (csize > 1)
        st_rank0(gather + (par * csize + rank) * (8 * kCols) + i, gv, uv);
      else if (f0 + r < p.F)
        p.y[(int64_t)(m0 + m) * p.F + f0 + r] = __float2bfloat16_rn(glu::value(gv, p.act) * uv);
    }
    if (csize > 1) {
      cl_sync();
      if (rank == 0)
        for (int i = threadIdx.x; i < 8 * toks; i += kThreads) {
          const int r = i & 7, m = i >> 3;
          float gv = 0.f, uv = 0.f;
          for (unsigned c = 0; c < csize; ++c) {
            const float2 v = gather[(par * csize + c) * (8 * kCols) + i];
            gv += v.x;
            uv += v.y;
          }
          if (f0 + r < p.F)
            p.y[(int64_t)(m0 + m) * p.F + f0 + r] = __float2bfloat16_rn(glu::value(gv, p.act) * uv);
        }
    }
    par ^= 1;
    tile += clusters;
  }
}

template <int NT>
cudaError_t launch_rows(RowsP p, int csize, int num_sms, cudaStream_t st) {
  auto kernel = glu_rows_kernel<NT>;
  p.x_bytes = (uint32_t)((p.nkb + csize - 1) / csize * 128 * p.tok);
  const size_t smem = p.x_bytes + kWarps * kStages * kStageBytes + 2 * kWarps * 16 * 8 * NT * 4 +
                      (csize > 1 ? 2 * csize * 8 * 8 * NT * 8 : 0);
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 226 * 1024);
  if (e != cudaSuccess) return e;
  const int per_sm = std::max(1, std::min(3, (int)(224 * 1024 / (smem + 1024))));
  const int clusters = std::min(p.tiles, std::max(1, num_sms * per_sm / csize));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * csize), (unsigned)((p.M + p.tok - 1) / p.tok));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)csize;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, p);
  g_kernel_launches.fetch_add(1, std::memory_order_relaxed);
  return e;
}

// ---------------------------------------------------------------------------
// fused multiply-adds: E elements, V of them a load, TK tokens at a time
// ---------------------------------------------------------------------------
constexpr int kChunk = 1024;  // k of x in shared memory

template <typename E, int V> struct Load;
template <> struct Load<float, 4> {
  static __device__ __forceinline__ void get(const float* p, float (&v)[4]) {
    const float4 q = __ldg(reinterpret_cast<const float4*>(p));
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
  }
};
template <typename E> struct Load<E, 1> {
  static __device__ __forceinline__ void get(const E* p, float (&v)[1]) { v[0] = to_f(*p); }
};

__device__ __forceinline__ void from_shared(const float* p, float (&v)[4]) {
  const float4 q = *reinterpret_cast<const float4*>(p);
  v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
}
__device__ __forceinline__ void from_shared(const float* p, float (&v)[1]) { v[0] = *p; }

template <typename E, int V, int TK>
__global__ void __launch_bounds__(kThreads) glu_fma_kernel(int M, int K, int F, int act,
                                                           const E* __restrict__ x,
                                                           const E* __restrict__ W,
                                                           E* __restrict__ y) {
  __shared__ __align__(16) float xs[TK][kChunk];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int f0 = (blockIdx.x * kWarps + warp) * 2, m0 = blockIdx.y * TK;
  const E* rows[4];  // gate f0, gate f0 + 1, up f0, up f0 + 1
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int f = min(f0 + (r & 1), F - 1);
    rows[r] = W + ((int64_t)(r >> 1) * F + f) * K;
  }
  float acc[4][TK];
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int m = 0; m < TK; ++m) acc[r][m] = 0.f;
  for (int k0 = 0; k0 < K; k0 += kChunk) {
    __syncthreads();
    for (int i = threadIdx.x; i < TK * kChunk; i += kThreads) {
      const int m = i / kChunk, k = i % kChunk;
      xs[m][k] = m0 + m < M && k0 + k < K ? to_f(x[(int64_t)(m0 + m) * K + k0 + k]) : 0.f;
    }
    __syncthreads();
    const int n = min(kChunk, K - k0);
#pragma unroll 4
    for (int k = lane * V; k < n; k += 32 * V) {
      float w[4][V];
#pragma unroll
      for (int r = 0; r < 4; ++r) Load<E, V>::get(rows[r] + k0 + k, w[r]);
#pragma unroll
      for (int m = 0; m < TK; ++m) {
        float xv[V];
        from_shared(&xs[m][k], xv);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int v = 0; v < V; ++v) acc[r][m] = fmaf(w[r][v], xv[v], acc[r][m]);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < TK; ++m) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[r][m] += __shfl_xor_sync(0xffffffffu, acc[r][m], o);
    if (lane < 2 && f0 + lane < F && m0 + m < M)
      y[(int64_t)(m0 + m) * F + f0 + lane] =
          from_f<E>(glu::value(lane ? acc[1][m] : acc[0][m], act) * (lane ? acc[3][m] : acc[2][m]));
  }
}

template <typename E, int V>
cudaError_t launch_fma(const GluArgs& a, cudaStream_t st) {
  const int tk = a.M <= 2 ? 2 : 8;
  const dim3 grid((unsigned)((a.F + 2 * kWarps - 1) / (2 * kWarps)), (unsigned)((a.M + tk - 1) / tk));
  auto kernel = tk == 2 ? glu_fma_kernel<E, V, 2> : glu_fma_kernel<E, V, 8>;
  kernel<<<grid, kThreads, 0, st>>>((int)a.M, (int)a.K, (int)a.F, a.act, static_cast<const E*>(a.x),
                                    static_cast<const E*>(a.W), static_cast<E*>(a.y));
  g_kernel_launches.fetch_add(1, std::memory_order_relaxed);
  return cudaGetLastError();
}

}  // namespace

cudaError_t glu_rows_forward(const GluArgs& a, cudaStream_t st) {
  if (!a.bf16) return a.K % 4 == 0 ? launch_fma<float, 4>(a, st) : launch_fma<float, 1>(a, st);
  // at K beyond 8 blocks' shared memory for one token a row is split no further
  if (a.K % 8 != 0 || a.K > 8 * kXBytes / 2) return launch_fma<bf16, 1>(a, st);
  RowsP p = {};
  p.M = (int)a.M; p.K = (int)a.K; p.F = (int)a.F;
  p.nkb = (int)((a.K + 63) / 64);
  p.tiles = (int)((a.F + 7) / 8);
  p.act = a.act;
  p.x = static_cast<const bf16*>(a.x);
  p.W = static_cast<const bf16*>(a.W);
  p.y = static_cast<bf16*>(a.y);
  auto x_bytes = [&](int c, int tok) { return (int64_t)((p.nkb + c - 1) / c) * 128 * tok; };
  p.tok = 32;
  while (p.tok > 1 && (p.tok >= 2 * a.M || x_bytes(8, p.tok) > kXBytes)) p.tok /= 2;
  p.tok = (int)std::min<int64_t>(p.tok, a.M);
  int c = 1;
  while (c < 8 && x_bytes(c, p.tok) > kXBytes) c *= 2;
  if (p.tok <= 8) return launch_rows<1>(p, c, a.num_sms, st);
  if (p.tok <= 16) return launch_rows<2>(p, c, a.num_sms, st);
  return launch_rows<4>(p, c, a.num_sms, st);
}

}  // namespace lr
