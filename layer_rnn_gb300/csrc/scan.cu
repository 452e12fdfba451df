// Gated linear recurrence over time, forward and backward.
//
//   f = sigmoid(p),  h_t = f_t h_{t-1} + (1 - f_t) z_t,  y_t = h_t or
//   sigmoid(q_t) h_t
//
// A run of steps acts on the state as h -> A h + B (A the product of its f),
// and such maps compose: (A2, B2) after (A1, B1) is (A1 A2, A2 B1 + B2).  So
// time is cut into tiles; each thread composes its own few steps, shared
// memory joins the threads of a tile, and the blocks of a cluster, which hold
// consecutive tiles, exchange their tiles' maps through distributed shared
// memory.  One pass over the data: every input is read once, into registers.
//
// Backward, from c_T = dhy against the walk:
//   dh_t = o_t dy_t + c_t,  c_{t-1} = f_t dh_t
//   dz = dh (1 - f),  dp = dh (h_{t-1} - z) f (1 - f),  dq = dy h o (1 - o)
// It needs h_{t-1}, which is not kept: the forward saves the state every
// kScanState steps and the backward composes the rest of the tile again.
//
// Bound by memory: 10 to 20 flop for every 4 to 16 bytes.
#include <algorithm>

#include "common.cuh"
#include "ops.h"

namespace lr {
namespace {

constexpr int kThreads = 256;

// f = sigmoid(p) and i = 1 - f, both to a few ulp: e = e^-p, f = 1 / (1 + e),
// i = e f.  e is held below 2^120 so that e f stays 1 where p is very
// negative; NaN goes through.
__device__ __forceinline__ void gate_pair(float p, float& f, float& i) {
  float e = __expf(-p);
  asm("min.NaN.f32 %0, %0, 0f7B800000;" : "+f"(e));
  f = __fdividef(1.0f, 1.0f + e);
  i = e * f;
}

// V consecutive elements of storage type E, held raw
template <typename E, int V> struct Raw;
template <> struct Raw<float, 4> { uint4 w; };
template <> struct Raw<bf16, 4> { uint2 w; };
template <> struct Raw<float, 1> { float w; };
template <> struct Raw<bf16, 1> { unsigned short w; };

template <typename E, int V>
__device__ __forceinline__ Raw<E, V> load_raw(const E* p) {
  Raw<E, V> r;
  r.w = __ldcs(reinterpret_cast<const decltype(r.w)*>(p));
  return r;
}
__device__ __forceinline__ void unpack(const Raw<float, 4>& r, float (&v)[4]) {
  v[0] = __uint_as_float(r.w.x); v[1] = __uint_as_float(r.w.y);
  v[2] = __uint_as_float(r.w.z); v[3] = __uint_as_float(r.w.w);
}
__device__ __forceinline__ void unpack(const Raw<bf16, 4>& r, float (&v)[4]) {
  v[0] = __uint_as_float(r.w.x << 16); v[1] = __uint_as_float(r.w.x & 0xffff0000u);
  v[2] = __uint_as_float(r.w.y << 16); v[3] = __uint_as_float(r.w.y & 0xffff0000u);
}
__device__ __forceinline__ void unpack(const Raw<float, 1>& r, float (&v)[1]) { v[0] = r.w; }
__device__ __forceinline__ void unpack(const Raw<bf16, 1>& r, float (&v)[1]) {
  v[0] = __uint_as_float((unsigned)r.w << 16);
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store_v(float* p, const float (&v)[4]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
}
__device__ __forceinline__ void store_v(bf16* p, const float (&v)[4]) {
  __stcs(reinterpret_cast<uint2*>(p), make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3])));
}
__device__ __forceinline__ void store_v(float* p, const float (&v)[1]) { *p = v[0]; }
__device__ __forceinline__ void store_v(bf16* p, const float (&v)[1]) {
  *p = __float2bfloat16_rn(v[0]);
}

struct ScanP {
  int64_t T, N, ldg, ldy, vecs, states_row;  // vecs = N * D * H / V
  int H, D, hv;                              // hv = H / V
  const int* lengths;
  const void* gx;
  const float* h0;
  void* y;
  float* hy;
  float* states;
  const void* dy;
  const float* dhy;
  void* dgx;
  float* dh0;
};

__device__ __forceinline__ unsigned cluster_size() {
  unsigned n;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return n;
}
__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
               "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_peer2(float2* local, unsigned rank, float a, float b) {
  unsigned addr;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(addr)
               : "r"(static_cast<unsigned>(__cvta_generic_to_shared(local))), "r"(rank));
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(a), "f"(b) : "memory");
}

// Where a thread works: CV lanes along the channels (V each), kThreads / CV
// slots along time, L steps a slot.
template <int V, int CV, int L>
struct Shape {
  static constexpr int kSlots = kThreads / CV;
  static constexpr int kChannels = CV * V;
  static constexpr int kTile = kSlots * L;
  static constexpr int kParts = kThreads / kChannels;  // threads a channel when slots are joined
  static constexpr int kPer = kSlots / kParts;         // slots each of them joins
  static_assert(kParts >= 1 && kPer >= 1 && kParts * kPer == kSlots, "shape");
};

// The tile's maps, slot by slot, and what goes into each slot.  Walks of the
// two passes differ in direction only: slot order s is the order in which the
// state passes through them.
template <int V, int CV, int L>
struct Join {
  using S = Shape<V, CV, L>;
  float2 slot[S::kSlots][S::kChannels];   // (A, B) of each slot; then .x = value going in
  float2 part[S::kParts][S::kChannels];
  float2 tile[2][8][S::kChannels];        // the cluster's tiles (by parity of the round)

  // state into the slots, given each slot's map in `slot`: returns the value
  // that leaves the whole round (all tiles of the cluster); `carry` enters
  // it.  Channel and part of this thread: tid % kChannels, tid / kChannels;
  // only these threads' carry matters.  All threads of the cluster call it.
  __device__ __forceinline__ float run(float carry, int round, unsigned rank, unsigned csize) {
    const int c = threadIdx.x % S::kChannels, q = threadIdx.x / S::kChannels;
    __syncthreads();
    float A = 1.f, B = 0.f;
#pragma unroll
    for (int k = 0; k < S::kPer; ++k) {
      const float2 m = slot[q * S::kPer + k][c];
      B = fmaf(m.x, B, m.y);
      A *= m.x;
    }
    if (S::kParts > 1) {
      part[q][c] = make_float2(A, B);
      __syncthreads();
    }
    float tA = 1.f, tB = 0.f, pA = 1.f, pB = 0.f;  // whole tile; the parts before this one
    if (S::kParts > 1) {
#pragma unroll
      for (int k = 0; k < S::kParts; ++k) {
        if (k == q) { pA = tA; pB = tB; }
        const float2 m = part[k][c];
        tB = fmaf(m.x, tB, m.y);
        tA *= m.x;
      }
    } else {
      tA = A; tB = B;
    }
    float in = carry, out = 0.f;
    if (csize > 1) {
      for (unsigned r = q; r < csize; r += S::kParts)
        st_peer2(&tile[round & 1][rank][c], r, tA, tB);
      cluster_sync();
      float h = carry;
      for (unsigned r = 0; r < csize; ++r) {
        if (r == rank) in = h;
        const float2 m = tile[round & 1][r][c];
        h = fmaf(m.x, h, m.y);
      }
      out = h;
    } else {
      out = fmaf(tA, carry, tB);
    }
    float h = fmaf(pA, in, pB);
#pragma unroll
    for (int k = 0; k < S::kPer; ++k) {
      float2& m = slot[q * S::kPer + k][c];
      const float nh = fmaf(m.x, h, m.y);
      m.x = h;
      h = nh;
    }
    __syncthreads();
    return out;
  }
};

// channel vector of a lane
struct Lane {
  bool live;
  int d, len;
  int64_t n, state;  // sequence; channel 0's place in [D, N, H]
  int64_t g0, y0;    // offset inside a time step's rows
  int64_t gh;        // the same in [N, D, H]
};
__device__ __forceinline__ Lane lane_of(const ScanP& p, int64_t vec, int V, int G) {
  Lane l;
  l.live = vec < p.vecs;
  if (!l.live) vec = 0;
  const int64_t nd = vec / p.hv;
  const int j = (int)(vec - nd * p.hv) * V;
  l.n = nd / p.D;
  l.d = (int)(nd - l.n * p.D);
  l.state = (l.d * p.N + l.n) * p.H + j;
  l.g0 = l.n * p.ldg + (int64_t)l.d * G * p.H + j;
  l.y0 = l.n * p.ldy + (int64_t)l.d * p.H + j;
  l.gh = nd * p.H + j;
  l.len = (int)p.T;
  if (p.lengths) l.len = min(max(p.lengths[l.n], 0), (int)p.T);
  return l;
}

template <typename E, int V, int CV, int L, bool GATE>
__global__ void __launch_bounds__(kThreads) scan_forward_kernel(const ScanP p) {
  using S = Shape<V, CV, L>;
  constexpr int G = GATE ? 3 : 2;
  __shared__ Join<V, CV, L> join;
  const unsigned csize = cluster_size(), rank = cluster_rank();
  const int cv = threadIdx.x % CV, slot = threadIdx.x / CV;
  const int64_t group = blockIdx.x / csize;
  const Lane l = lane_of(p, group * CV + cv, V, G);
  const E* gx = static_cast<const E*>(p.gx) + l.g0;
  E* y = static_cast<E*>(p.y) + l.y0;
  const int64_t tg = p.N * p.ldg, ty = p.N * p.ldy;
  // the carried state of channel threadIdx.x % kChannels
  float carry = 0.f;
  {
    const int c = threadIdx.x % S::kChannels;
    const Lane k = lane_of(p, group * CV + c / V, V, G);
    if (k.live && p.h0) carry = p.h0[k.state + c % V];
  }
  const int64_t rounds = (p.T + S::kTile * csize - 1) / (S::kTile * csize);
  for (int64_t r = 0; r < rounds; ++r) {
    const int64_t w0 = (r * csize + rank) * S::kTile + slot * L;  // first step of the walk
    Raw<E, V> rp[L], rz[L];
    unsigned valid = 0;
#pragma unroll
    for (int k = 0; k < L; ++k) {
      const int64_t t = l.d ? p.T - 1 - (w0 + k) : w0 + k;
      if (l.live && w0 + k < p.T && t < l.len) {
        valid |= 1u << k;
        rp[k] = load_raw<E, V>(gx + t * tg);
        rz[k] = load_raw<E, V>(gx + t * tg + p.H);
      }
    }
    float a[L][V], b[L][V], A[V], B[V];
#pragma unroll
    for (int v = 0; v < V; ++v) { A[v] = 1.f; B[v] = 0.f; }
#pragma unroll
    for (int k = 0; k < L; ++k) {
      float pv[V], zv[V];
      unpack(rp[k], pv);
      unpack(rz[k], zv);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float f, i;
        gate_pair(pv[v], f, i);
        const bool ok = (valid >> k) & 1u;
        a[k][v] = ok ? f : 1.f;
        b[k][v] = ok ? i * zv[v] : 0.f;
        B[v] = fmaf(a[k][v], B[v], b[k][v]);
        A[v] *= a[k][v];
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) join.slot[slot][cv * V + v] = make_float2(A[v], B[v]);
    carry = join.run(carry, (int)(r & 1), rank, csize);
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = join.slot[slot][cv * V + v].x;
    if (p.states && l.live && w0 < p.T && w0 % kScanState == 0) {
#pragma unroll
      for (int v = 0; v < V; ++v) p.states[w0 / kScanState * p.states_row + l.gh + v] = h[v];
    }
#pragma unroll
    for (int k = 0; k < L; ++k) {
      const int64_t t = l.d ? p.T - 1 - (w0 + k) : w0 + k;
      const bool ok = (valid >> k) & 1u;
      float out[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        h[v] = fmaf(a[k][v], h[v], b[k][v]);
        out[v] = ok ? h[v] : 0.f;
      }
      if (GATE && ok) {
        float q[V];
        unpack(load_raw<E, V>(gx + t * tg + 2 * p.H), q);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float o, i;
          gate_pair(q[v], o, i);
          out[v] *= o;
        }
      }
      if (l.live && w0 + k < p.T) store_v(y + t * ty, out);
    }
  }
  if (p.hy && rank == 0) {
    const int c = threadIdx.x % S::kChannels;
    const Lane k = lane_of(p, group * CV + c / V, V, G);
    if (threadIdx.x < S::kChannels && k.live) p.hy[k.state + c % V] = carry;
  }
}

template <typename E, int V, int CV, int L, bool GATE>
__global__ void __launch_bounds__(kThreads) scan_backward_kernel(const ScanP p) {
  using S = Shape<V, CV, L>;
  constexpr int G = GATE ? 3 : 2;
  static_assert(S::kTile % kScanState == 0, "a tile starts at a saved state");
  __shared__ Join<V, CV, L> join;
  const unsigned csize = cluster_size(), rank = cluster_rank();
  const int cv = threadIdx.x % CV, slot = threadIdx.x / CV;
  const int64_t group = blockIdx.x / csize;
  const Lane l = lane_of(p, group * CV + cv, V, G);
  const E* gx = static_cast<const E*>(p.gx) + l.g0;
  E* dgx = static_cast<E*>(p.dgx) + l.g0;
  const E* dy = static_cast<const E*>(p.dy) + l.y0;
  const int64_t tg = p.N * p.ldg, ty = p.N * p.ldy;
  const int c = threadIdx.x % S::kChannels;
  const Lane kc = lane_of(p, group * CV + c / V, V, G);
  float carry = 0.f;
  if (kc.live && p.dhy) carry = p.dhy[kc.state + c % V];
  const int64_t tiles = (p.T + S::kTile - 1) / S::kTile;
  const int64_t rounds = (tiles + csize - 1) / csize;
  for (int64_t r = 0; r < rounds; ++r) {
    // tiles from the end of the walk; a tile before the start is empty
    const int64_t tile = tiles - 1 - (r * csize + rank);
    const int64_t w0 = tile * S::kTile + slot * L;
    Raw<E, V> rp[L], rz[L], rd[L], rq[GATE ? L : 1];
    unsigned valid = 0;
#pragma unroll
    for (int k = 0; k < L; ++k) {
      const int64_t t = l.d ? p.T - 1 - (w0 + k) : w0 + k;
      if (l.live && tile >= 0 && w0 + k < p.T && t < l.len) {
        valid |= 1u << k;
        rp[k] = load_raw<E, V>(gx + t * tg);
        rz[k] = load_raw<E, V>(gx + t * tg + p.H);
        if (GATE) rq[k] = load_raw<E, V>(gx + t * tg + 2 * p.H);
        rd[k] = load_raw<E, V>(dy + t * ty);
      }
    }
    float start = 0.f;  // the state at the tile's start, of channel c
    if (tile >= 0 && kc.live)
      start = p.states[tile * (S::kTile / kScanState) * p.states_row + kc.gh + c % V];
    // forward over the tile: the state into each slot
    float f[L][V], A[V], B[V];
#pragma unroll
    for (int v = 0; v < V; ++v) { A[v] = 1.f; B[v] = 0.f; }
#pragma unroll
    for (int k = 0; k < L; ++k) {
      float pv[V], zv[V];
      unpack(rp[k], pv);
      unpack(rz[k], zv);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float i;
        gate_pair(pv[v], f[k][v], i);
        const bool ok = (valid >> k) & 1u;
        f[k][v] = ok ? f[k][v] : 1.f;
        B[v] = ok ? fmaf(f[k][v], B[v], i * zv[v]) : B[v];
        A[v] *= f[k][v];
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) join.slot[slot][cv * V + v] = make_float2(A[v], B[v]);
    join.run(start, 0, 0, 1);
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = join.slot[slot][cv * V + v].x;
    // against the walk: slot s of this order is the tile's slot kSlots - 1 - s
#pragma unroll
    for (int v = 0; v < V; ++v) B[v] = 0.f;
#pragma unroll
    for (int k = L - 1; k >= 0; --k) {
      float dv[V], o[V];
      unpack(rd[k], dv);
      if (GATE) unpack(rq[GATE ? k : 0], o);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const bool ok = (valid >> k) & 1u;
        float i;
        if (GATE) gate_pair(o[v], o[v], i); else o[v] = 1.f;
        B[v] = ok ? f[k][v] * fmaf(dv[v], o[v], B[v]) : B[v];
      }
    }
    __syncthreads();  // the states going in have been read
#pragma unroll
    for (int v = 0; v < V; ++v)
      join.slot[S::kSlots - 1 - slot][cv * V + v] = make_float2(A[v], B[v]);
    carry = join.run(carry, (int)(r & 1), rank, csize);
    float e[V];
#pragma unroll
    for (int v = 0; v < V; ++v) e[v] = join.slot[S::kSlots - 1 - slot][cv * V + v].x;
    // h before each step, then the gradients against the walk
    float hb[L][V];
#pragma unroll
    for (int k = 0; k < L; ++k) {
      float zv[V];
      unpack(rz[k], zv);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        hb[k][v] = h[v];
        const bool ok = (valid >> k) & 1u;
        // (1 - f) z + f h as z + f (h - z) would lose small differences; the
        // form of the forward pass is kept
        float fv, i, pv[V];
        unpack(rp[k], pv);
        gate_pair(pv[v], fv, i);
        h[v] = ok ? fmaf(fv, h[v], i * zv[v]) : h[v];
      }
    }
#pragma unroll
    for (int k = L - 1; k >= 0; --k) {
      const int64_t t = l.d ? p.T - 1 - (w0 + k) : w0 + k;
      const bool ok = (valid >> k) & 1u;
      float pv[V], zv[V], dv[V], qv[V], gp[V], gz[V], gq[V];
      unpack(rp[k], pv);
      unpack(rz[k], zv);
      unpack(rd[k], dv);
      if (GATE) unpack(rq[GATE ? k : 0], qv);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float fv, i, o = 1.f, oi = 0.f;
        gate_pair(pv[v], fv, i);
        if (GATE) gate_pair(qv[v], o, oi);
        const float hn = fmaf(fv, hb[k][v], i * zv[v]);
        const float dh = fmaf(dv[v], o, e[v]);
        gz[v] = ok ? dh * i : 0.f;
        gp[v] = ok ? dh * (hb[k][v] - zv[v]) * (fv * i) : 0.f;
        gq[v] = ok ? dv[v] * hn * (o * oi) : 0.f;
        e[v] = ok ? fv * dh : e[v];
      }
      if (l.live && tile >= 0 && w0 + k < p.T) {
        store_v(dgx + t * tg, gp);
        store_v(dgx + t * tg + p.H, gz);
        if (GATE) store_v(dgx + t * tg + 2 * p.H, gq);
      }
    }
    __syncthreads();  // the slots have been read
  }
  if (p.dh0 && rank == 0 && threadIdx.x < S::kChannels && kc.live)
    p.dh0[kc.state + c % V] = carry;
}

template <typename K>
cudaError_t launch(K kernel, const ScanP& p, int64_t groups, int csize, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(groups * csize));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)csize;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  g_kernel_launches.fetch_add(1, std::memory_order_relaxed);
  return e;
}

// Blocks of a cluster share the tiles of a channel group: the smallest power
// of two (at most 8) that gives the card two blocks an SM, and no more than
// there are tiles.
int cluster_for(int64_t groups, int64_t tiles, int num_sms) {
  int c = 1;
  while (c < 8 && groups * c < 2 * num_sms && c < tiles) c *= 2;
  return c;
}

ScanP params(const ScanArgs& a, int V) {
  ScanP p;
  p.T = a.T; p.N = a.N; p.ldg = a.ldg; p.ldy = a.ldy;
  p.H = (int)a.H; p.D = (int)a.D; p.hv = (int)(a.H / V);
  p.vecs = a.N * a.D * p.hv;
  p.states_row = a.N * a.D * a.H;
  p.lengths = a.lengths; p.gx = a.gx; p.h0 = a.h0; p.y = a.y; p.hy = a.hy; p.states = a.states;
  p.dy = a.dy; p.dhy = a.dhy; p.dgx = a.dgx; p.dh0 = a.dh0;
  return p;
}

template <typename E, int V, int CV, int L, bool BWD>
cudaError_t run(const ScanArgs& a, cudaStream_t st) {
  using S = Shape<V, CV, L>;
  const ScanP p = params(a, V);
  const int64_t groups = (p.vecs + CV - 1) / CV, tiles = (a.T + S::kTile - 1) / S::kTile;
  const int c = cluster_for(groups, tiles, a.num_sms);
  if (BWD)
    return a.gate ? launch(scan_backward_kernel<E, V, CV, L, true>, p, groups, c, st)
                  : launch(scan_backward_kernel<E, V, CV, L, false>, p, groups, c, st);
  return a.gate ? launch(scan_forward_kernel<E, V, CV, L, true>, p, groups, c, st)
                : launch(scan_forward_kernel<E, V, CV, L, false>, p, groups, c, st);
}

// four channels a load where every row starts on such a boundary
bool by_four(const ScanArgs& a) {
  const uintptr_t m = a.bf16 ? 8 : 16;
  auto ok = [&](const void* q) { return reinterpret_cast<uintptr_t>(q) % m == 0; };
  return a.H % 4 == 0 && a.ldg % 4 == 0 && a.ldy % 4 == 0 && ok(a.gx) && ok(a.y) && ok(a.dy) &&
         ok(a.dgx);
}

}  // namespace

cudaError_t scan_forward(const ScanArgs& a, cudaStream_t st) {
  if (by_four(a))
    return a.bf16 ? run<bf16, 4, 16, 8, false>(a, st) : run<float, 4, 16, 8, false>(a, st);
  return a.bf16 ? run<bf16, 1, 32, 16, false>(a, st) : run<float, 1, 32, 16, false>(a, st);
}

cudaError_t scan_backward(const ScanArgs& a, cudaStream_t st) {
  if (by_four(a))
    return a.bf16 ? run<bf16, 4, 16, 8, true>(a, st) : run<float, 4, 16, 4, true>(a, st);
  return a.bf16 ? run<bf16, 1, 32, 8, true>(a, st) : run<float, 1, 32, 8, true>(a, st);
}

}  // namespace lr
