// Matrix-vector products with 4-bit weights and group scales.
//
//   y[m][r] = sum_k x[m][k] (q[r][k] - zero[r][k / g]) scale[r][k / g]
//
// For a few tokens every weight is used a few times only, so the bytes of q
// bound the product.  A warp streams blocks of 16 (or 32) rows by 256 weights,
// 128 bytes a row, through its own ring of asynchronous copies, and multiplies
// them on the tensor cores (m16n8k16, the rows as M, the tokens as N): with
// one fused multiply-add a weight and token, the CUDA cores' conversions
// alone would take as long as the bytes.  The order of k inside a product is
// free, so the eight nibbles of a 32-bit word become operand pairs (k0, k4),
// (k1, k5), ... by one shift, one mask and one subtraction each, and x is laid
// out in shared memory to match.
//
// Exactness: q - zero is a small whole number, exact in bf16 and fp16.  bf16
// tokens are operands as they are.  float32 tokens become two fp16 columns,
// x s = hi + lo 2^-11, s a power of two that maps the token's largest
// magnitude below 2^14: 22 bits of every value near the largest.  Each group
// is summed in float32 and only then multiplied by its scale.
//
// The eight warps of a block share the rows and split K; blocks of a cluster
// split it further where x would not fit shared memory or the rows alone do
// not fill the card.  Partial sums are joined in a fixed order.
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "ops.h"

namespace lr {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kBlockK = 256;                 // weights of a row in one ring stage
constexpr int kXBytes = 64 * 1024;           // x of one block at most

struct W4P {
  int M, R, K, nkb, groups, tiles, tok;      // tok: tokens a pass
  int64_t ldq;
  const void* x;
  const uint8_t* q;
  const void* scales;
  const uint8_t* zeros;
  void* y;
  uint32_t x_bytes;                          // shared memory of x
};

__device__ __forceinline__ uint32_t smem_at(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes, or zeros where !ok (nothing is read then)
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}

template <bool HALF>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  if (HALF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The eight nibbles of w less the zero point, as pairs (k0, k4), (k1, k5),
// (k2, k6), (k3, k7).  zz: the zero point z in both halves, as the biased
// value: bf16 128 + z (the nibble under the exponent of 128) or fp16 1024 + z.
__device__ __forceinline__ void decode_bf16(uint32_t w, uint32_t zz, uint32_t (&a)[4]) {
  const __nv_bfloat162 z = *reinterpret_cast<const __nv_bfloat162*>(&zz);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t v = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&v), z);
    a[i] = *reinterpret_cast<const uint32_t*>(&d);
  }
}
// fp16 has room for the second nibble of a byte in place: 1024 + 16 q, of
// which a sixteenth less (64 + z) is q - z
__device__ __forceinline__ void decode_f16(uint32_t w, uint32_t zz, uint32_t (&a)[4]) {
  const __half2 z = *reinterpret_cast<const __half2*>(&zz);
  const __half2 z64 = __hsub2(__float2half2_rn(960.f), z);  // -(64 + z)
  const __half2 s = __float2half2_rn(0.0625f);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t lo = (w & 0x000F000Fu) | 0x64006400u, hi = (w & 0x00F000F0u) | 0x64006400u;
    const __half2 d = __hsub2(*reinterpret_cast<__half2*>(&lo), z);
    const __half2 e = __hfma2(*reinterpret_cast<__half2*>(&hi), s, z64);
    a[2 * i] = *reinterpret_cast<const uint32_t*>(&d);
    a[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&e);
    w >>= 8;
  }
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
__device__ __forceinline__ void st_rank0(float* local, float v) {
  unsigned a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_at(local)));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}

// 2^e as a float, e within the normal range
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

// F32: element type float32 (two columns a token), else bf16.  NT: column
// tiles of 8; MT: row tiles of 16; GS: 32-weight chunks a group; ST: stages.
template <bool F32, int NT, int MT, int GS, bool ZERO, int ST>
__global__ void __launch_bounds__(kThreads) w4_kernel(const W4P p) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int kRows = 16 * MT, kCols = 8 * NT;
  constexpr int kStage = kRows * 128;               // bytes of a stage of one warp
  constexpr int kGroups = 8 / GS;                   // groups of a block of 256 weights
  constexpr int kHeld = kGroups > 4 ? 2 : 1;        // of them held by a lane
  constexpr int kBufs = NT == 4 ? 1 : 2;            // of the joined partial sums
  __shared__ float inv_scale[16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const unsigned csize = cl_size(), rank = cl_rank();
  const int m0 = blockIdx.y * p.tok, toks = min(p.tok, p.M - m0);
  const int cols = F32 ? 2 * toks : toks;
  const int kb0 = (int)((int64_t)rank * p.nkb / csize), kb1 = (int)((int64_t)(rank + 1) * p.nkb / csize);
  const int clusters = gridDim.x / csize, first = blockIdx.x / csize;
  const int per = (kb1 - kb0 + kWarps - 1) / kWarps;  // blocks of a warp and tile
  const int my_tiles = first < p.tiles ? (p.tiles - 1 - first) / clusters + 1 : 0;
  const int items = my_tiles * per;
  unsigned char* xs = smem;
  unsigned char* ring = smem + p.x_bytes + warp * (ST * kStage);
  float* red = reinterpret_cast<float*>(smem + p.x_bytes + kWarps * ST * kStage);
  float* gather = red + kBufs * kWarps * kRows * kCols;  // clusters only: [2][csize][kRows * 16]
  const uint32_t ring_at = smem_at(ring), xs_at = smem_at(xs);

  // scales (and zero points) of a stage: rows g and g + 8 of each row tile,
  // groups t and t + 4
  uint32_t sc[ST][MT][2][kHeld], zp[F32 && ZERO ? ST : 1][MT][2][kHeld];
  int it_tile = first, it_kb = 0;  // of the next stage to load
  auto issue = [&](int s) {
    const int kb = kb0 + it_kb * kWarps + warp;
    if (it_tile < p.tiles && kb < kb1) {
      const int row0 = it_tile * kRows;
#pragma unroll
      for (int j = 0; j < 4 * MT; ++j) {
        const int row = j * 4 + (lane >> 3), c = lane & 7;
        const int64_t byte = (int64_t)kb * 128 + c * 16;
        const bool ok = row0 + row < p.R && byte < p.ldq;
        copy16(ring_at + s * kStage + row * 128 + ((c ^ (row & 7)) << 4),
               p.q + (ok ? (int64_t)(row0 + row) * p.ldq + byte : 0), ok);
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int u = 0; u < kHeld; ++u) {
            const int row = row0 + mt * 16 + h * 8 + g, gi = kb * kGroups + u * 4 + t;
            const bool ok = row < p.R && u * 4 + t < kGroups && gi < p.groups;
            const int64_t at = (int64_t)row * p.groups + gi;
            uint32_t sv = 0, zv = 8;
            if (ok) {
              sv = F32 ? __ldcs(static_cast<const unsigned*>(p.scales) + at)
                       : (uint32_t)__ldcs(static_cast<const unsigned short*>(p.scales) + at);
              if (ZERO) zv = __ldcs(p.zeros + at);
            }
            if (!F32 && ZERO) sv |= (0x4300u | zv) << 16;
            sc[s][mt][h][u] = sv;
            if (F32 && ZERO) zp[s][mt][h][u] = zv;
          }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (++it_kb == per) { it_kb = 0; it_tile += clusters; }
  };
#pragma unroll
  for (int s = 0; s < ST - 1; ++s) issue(s);

  // x into shared memory: chunk of 32 k, column, lane t's eight values
  // k0 k4 k1 k5 k2 k6 k3 k7 (t * 8 onwards)
  const int k_from = kb0 * kBlockK, chunks = (kb1 - kb0) * (kBlockK / 32);
  if (F32) {
    const float* x = static_cast<const float*>(p.x) + (int64_t)m0 * p.K;
    for (int m = warp; m < toks; m += kWarps) {
      unsigned mx = 0;
      const int k_to = min(p.K, kb1 * kBlockK);
      for (int k = k_from + lane; k < k_to; k += 32)
        mx = max(mx, __float_as_uint(x[(int64_t)m * p.K + k]) & 0x7fffffffu);
      mx = __reduce_max_sync(0xffffffffu, mx);
      // infinities and NaN: no scale, the row's results are not finite
      int e = mx >= 0x7f800000u || mx == 0 ? 0 : 13 - ((int)(mx >> 23) - 127);
      e = min(max(e, -126), 126);
      if (lane == 0) inv_scale[m] = exp2i(-e);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < chunks * toks * 4; i += kThreads) {
      const int tt = i & 3, cm = i >> 2, m = cm % toks, c = cm / toks;
      const float s = 1.0f / inv_scale[m];
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int k = k_from + c * 32 + tt * 8 + j + 4 * u;
          v[u] = k < p.K ? x[(int64_t)m * p.K + k] * s : 0.f;
        }
        const __half2 h = __floats2half2_rn(v[0], v[1]);
        const float2 hf = __half22float2(h);
        const __half2 l = __floats2half2_rn(isinf(hf.x) ? 0.f : (v[0] - hf.x) * 2048.f,
                                            isinf(hf.y) ? 0.f : (v[1] - hf.y) * 2048.f);
        hi[j] = *reinterpret_cast<const uint32_t*>(&h);
        lo[j] = *reinterpret_cast<const uint32_t*>(&l);
      }
      uint4* d = reinterpret_cast<uint4*>(xs) + (size_t)(c * cols + 2 * m) * 4 + tt;
      d[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      d[4] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  } else {
    const unsigned short* x = static_cast<const unsigned short*>(p.x) + (int64_t)m0 * p.K;
    for (int i = threadIdx.x; i < chunks * toks * 4; i += kThreads) {
      const int tt = i & 3, cm = i >> 2, m = cm % toks, c = cm / toks;
      uint32_t v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = k_from + c * 32 + tt * 8 + j;
        const uint32_t a = k < p.K ? x[(int64_t)m * p.K + k] : 0u;
        const uint32_t b = k + 4 < p.K ? x[(int64_t)m * p.K + k + 4] : 0u;
        v[j] = a | (b << 16);
      }
      reinterpret_cast<uint4*>(xs)[(size_t)(c * cols + m) * 4 + tt] = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
  __syncthreads();

  float fin[MT][NT][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) fin[mt][nt][i] = 0.f;

  int tile = first, kbi = 0, par = 0;
  for (int base = 0; base < items; base += ST) {
#pragma unroll
    for (int s = 0; s < ST; ++s) {
      if (base + s >= items) break;
      issue((s + ST - 1) % ST);
      asm volatile("cp.async.wait_group %0;" ::"n"(ST - 1) : "memory");
      __syncwarp();
      const int kb = kb0 + kbi * kWarps + warp;
      if (kb < kb1) {
        const uint32_t st = ring_at + s * kStage + g * 128 + t * 4;
        const uint32_t xa = xs_at + (uint32_t)((kb - kb0) * 8 * cols + g) * 64 + t * 16;
        float acc[MT][NT][4];
        float s0[MT], s1[MT];
        uint32_t z0[MT], z1[MT];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          if (c % GS == 0) {
            const int gi = c / GS;
            const int src = (lane & 28) | (gi & 3);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              const uint32_t u0 = __shfl_sync(0xffffffffu, sc[s][mt][0][gi >> 2], src);
              const uint32_t u1 = __shfl_sync(0xffffffffu, sc[s][mt][1][gi >> 2], src);
              s0[mt] = __uint_as_float(F32 ? u0 : u0 << 16);
              s1[mt] = __uint_as_float(F32 ? u1 : u1 << 16);
              if (F32) {
                z0[mt] = z1[mt] = 0x64086408u;
                if (ZERO) {
                  z0[mt] = 0x64006400u |
                           __shfl_sync(0xffffffffu, zp[F32 && ZERO ? s : 0][mt][0][gi >> 2], src) * 0x10001u;
                  z1[mt] = 0x64006400u |
                           __shfl_sync(0xffffffffu, zp[F32 && ZERO ? s : 0][mt][1][gi >> 2], src) * 0x10001u;
                }
              } else {
                z0[mt] = ZERO ? __byte_perm(u0, 0, 0x3232) : 0x43084308u;
                z1[mt] = ZERO ? __byte_perm(u1, 0, 0x3232) : 0x43084308u;
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[mt][nt][i] = 0.f;
            }
          }
          uint4 b[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            b[nt] = make_uint4(0, 0, 0, 0);
            if (nt * 8 + g < cols) b[nt] = lds128(xa + (uint32_t)(c * cols + nt * 8) * 64);
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const uint32_t at = st + mt * 2048 + ((c ^ g) << 4);
            uint32_t a[4], d[4];
            if (F32) {
              decode_f16(lds32(at), z0[mt], a);
              decode_f16(lds32(at + 1024), z1[mt], d);
            } else {
              decode_bf16(lds32(at), z0[mt], a);
              decode_bf16(lds32(at + 1024), z1[mt], d);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma<F32>(acc[mt][nt], a[0], d[0], a[1], d[1], b[nt].x, b[nt].y);
              mma<F32>(acc[mt][nt], a[2], d[2], a[3], d[3], b[nt].z, b[nt].w);
            }
          }
          if (c % GS == GS - 1) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                fin[mt][nt][0] = fmaf(s0[mt], acc[mt][nt][0], fin[mt][nt][0]);
                fin[mt][nt][1] = fmaf(s0[mt], acc[mt][nt][1], fin[mt][nt][1]);
                fin[mt][nt][2] = fmaf(s1[mt], acc[mt][nt][2], fin[mt][nt][2]);
                fin[mt][nt][3] = fmaf(s1[mt], acc[mt][nt][3], fin[mt][nt][3]);
              }
          }
        }
      }
      __syncwarp();
      if (++kbi < per) continue;
      // the tile is done: join the warps, then the blocks of the cluster
      kbi = 0;
      float* rw = red + (kBufs == 2 ? par : 0) * (kWarps * kRows * kCols);
      if (kBufs == 1) __syncthreads();  // the last tile's sums have been read
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float* d = rw + (warp * kRows + mt * 16 + g) * kCols + nt * 8 + 2 * t;
          *reinterpret_cast<float2*>(d) = make_float2(fin[mt][nt][0], fin[mt][nt][1]);
          *reinterpret_cast<float2*>(d + 8 * kCols) = make_float2(fin[mt][nt][2], fin[mt][nt][3]);
#pragma unroll
          for (int i = 0; i < 4; ++i) fin[mt][nt][i] = 0.f;
        }
      __syncthreads();
      const int row0 = tile * kRows;
      for (int i = threadIdx.x; i < kRows * toks; i += kThreads) {
        const int row = i % kRows, m = i / kRows;
        const float* d = rw + row * kCols + (F32 ? 2 * m : m);
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
          v += F32 ? fmaf(d[w * kRows * kCols + 1], 0x1p-11f, d[w * kRows * kCols])
                   : d[w * kRows * kCols];
        if (F32) v *= inv_scale[m];
        if (csize > 1)
          st_rank0(gather + (par * csize + rank) * (kRows * 16) + i, v);
        else if (row0 + row < p.R) {
          const int64_t at = (int64_t)(m0 + m) * p.R + row0 + row;
          if (F32) static_cast<float*>(p.y)[at] = v;
          else static_cast<bf16*>(p.y)[at] = __float2bfloat16_rn(v);
        }
      }
      if (csize > 1) {
        cl_sync();
        if (rank == 0)
          for (int i = threadIdx.x; i < kRows * toks; i += kThreads) {
            const int row = i % kRows, m = i / kRows;
            float v = 0.f;
            for (unsigned r = 0; r < csize; ++r) v += gather[(par * csize + r) * (kRows * 16) + i];
            if (row0 + row < p.R) {
              const int64_t at = (int64_t)(m0 + m) * p.R + row0 + row;
              if (F32) static_cast<float*>(p.y)[at] = v;
              else static_cast<bf16*>(p.y)[at] = __float2bfloat16_rn(v);
            }
          }
      }
      par ^= 1;
      tile += clusters;
    }
  }
}

template <bool F32, int NT, int MT, int GS, bool ZERO>
cudaError_t launch(W4P p, int csize, int num_sms, cudaStream_t st) {
  constexpr int ST = MT == 1 ? 4 : 3;
  auto kernel = w4_kernel<F32, NT, MT, GS, ZERO, ST>;
  constexpr int kRows = 16 * MT;
  p.tiles = (p.R + kRows - 1) / kRows;
  const int cols = p.tok * (F32 ? 2 : 1);
  p.x_bytes = (uint32_t)((p.nkb + csize - 1) / csize * 8 * cols * 64);
  const size_t smem = p.x_bytes + kWarps * ST * kRows * 128 + (NT == 4 ? 1 : 2) * kWarps * kRows * 8 * NT * 4 +
                      (csize > 1 ? 2 * csize * kRows * 16 * 4 : 0);
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024 - 1024);
  if (e != cudaSuccess) return e;
  const int per_sm = std::max(1, (int)(220 * 1024 / (smem + 1024)));
  const int clusters = std::min(p.tiles, std::max(1, num_sms * std::min(per_sm, 3) / csize));
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

template <bool F32, int NT, int MT>
cudaError_t by_group(const W4P& p, int group, int csize, int num_sms, cudaStream_t st) {
  const bool z = p.zeros != nullptr;
  if (group == 32)
    return z ? launch<F32, NT, MT, 1, true>(p, csize, num_sms, st)
             : launch<F32, NT, MT, 1, false>(p, csize, num_sms, st);
  if (group == 64)
    return z ? launch<F32, NT, MT, 2, true>(p, csize, num_sms, st)
             : launch<F32, NT, MT, 2, false>(p, csize, num_sms, st);
  return z ? launch<F32, NT, MT, 4, true>(p, csize, num_sms, st)
           : launch<F32, NT, MT, 4, false>(p, csize, num_sms, st);
}

// ---------------------------------------------------------------------------
// quantisation: one warp a group, two weights a lane and step
// ---------------------------------------------------------------------------
template <typename E>
__global__ void __launch_bounds__(256) w4_quantize_kernel(const E* __restrict__ w, int R, int K,
                                                          int group, int groups, int64_t ldq,
                                                          uint8_t* q, E* scales, uint8_t* zeros) {
  const int lane = threadIdx.x & 31;
  for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < (int64_t)R * groups;
       i += (int64_t)gridDim.x * 8) {
    const int r = (int)(i / groups), gi = (int)(i - (int64_t)r * groups);
    const E* row = w + (int64_t)r * K;
    const int k0 = gi * group, k1 = min(K, k0 + group);
    float lo = 0.f, hi = 0.f;
    for (int k = k0 + lane; k < k1; k += 32) {
      const float v = to_f(row[k]);
      lo = fminf(lo, v);
      hi = fmaxf(hi, v);
    }
    for (int o = 16; o > 0; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    // the scale as it is stored, so that the weights are nearest in its grid
    const float s = to_f(from_f<E>(zeros ? (hi - lo) / 15.f : fmaxf(-lo, hi) / 7.f));
    const float z = zeros ? (s > 0.f ? fminf(15.f, rintf(-lo / s)) : 0.f) : 8.f;
    if (lane == 0) {
      scales[i] = from_f<E>(s);
      if (zeros) zeros[i] = (uint8_t)z;
    }
    // the last group also clears the rest of the row
    const int64_t b1 = gi == groups - 1 ? ldq : (k0 + group) / 2;
    for (int64_t b = k0 / 2 + lane; b < b1; b += 32) {
      unsigned v = 0;
      for (int u = 0; u < 2; ++u) {
        const int64_t k = 2 * b + u;
        if (k >= k1) continue;
        const float n = s > 0.f ? rintf(to_f(row[k]) / s) : 0.f;
        v |= (unsigned)fminf(15.f, fmaxf(0.f, n + z)) << (4 * u);
      }
      q[(int64_t)r * ldq + b] = (uint8_t)v;
    }
  }
}

}  // namespace

cudaError_t w4_matvec(const W4Args& a, cudaStream_t st) {
  W4P p = {};
  p.M = (int)a.M; p.R = (int)a.R; p.K = (int)a.K;
  p.nkb = (int)((a.K + kBlockK - 1) / kBlockK);
  p.groups = (int)((a.K + a.group - 1) / a.group);
  p.ldq = a.ldq;
  p.x = a.x; p.q = a.q; p.scales = a.scales; p.zeros = a.zeros; p.y = a.y;
  const int per_tok = a.bf16 ? 1 : 2;
  // tokens a pass: as many as fit shared memory with K split over 8 blocks
  p.tok = 16;
  while (p.tok > 1 && (p.tok >= 2 * a.M ||
                       (int64_t)((p.nkb + 7) / 8) * 8 * 64 * p.tok * per_tok > kXBytes))
    p.tok /= 2;
  p.tok = (int)std::min<int64_t>(p.tok, a.M);
  const int cols = p.tok * per_tok;
  int c = 1;
  while (c < 8 && (int64_t)((p.nkb + c - 1) / c) * 8 * 64 * cols > kXBytes) c *= 2;
  // few rows: split K as long as every warp keeps a block of 256 weights
  while (c < 8 && (p.R + 15) / 16 * c < a.num_sms && p.nkb >= 2 * c * kWarps) c *= 2;
  if (a.bf16) {
    if (cols <= 8) return by_group<false, 1, 1>(p, a.group, c, a.num_sms, st);
    return by_group<false, 2, 2>(p, a.group, c, a.num_sms, st);
  }
  if (cols <= 8) return by_group<true, 1, 1>(p, a.group, c, a.num_sms, st);
  if (cols <= 16) return by_group<true, 2, 2>(p, a.group, c, a.num_sms, st);
  return by_group<true, 4, 2>(p, a.group, c, a.num_sms, st);
}

cudaError_t w4_quantize(const W4Args& a, const void* w, cudaStream_t st) {
  const int groups = (int)((a.K + a.group - 1) / a.group);
  const int64_t warps = a.R * groups;
  const int blocks = (int)std::min<int64_t>((warps + 7) / 8, (int64_t)a.num_sms * 16);
  uint8_t* q = const_cast<uint8_t*>(a.q);
  uint8_t* z = const_cast<uint8_t*>(a.zeros);
  void* s = const_cast<void*>(a.scales);
  if (a.bf16)
    w4_quantize_kernel<bf16><<<blocks, 256, 0, st>>>(static_cast<const bf16*>(w), (int)a.R, (int)a.K,
                                                     a.group, groups, a.ldq, q, static_cast<bf16*>(s), z);
  else
    w4_quantize_kernel<float><<<blocks, 256, 0, st>>>(static_cast<const float*>(w), (int)a.R, (int)a.K,
                                                      a.group, groups, a.ldq, q, static_cast<float*>(s), z);
  g_kernel_launches.fetch_add(1, std::memory_order_relaxed);
  return cudaGetLastError();
}

}  // namespace lr
