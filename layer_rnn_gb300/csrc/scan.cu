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
#include <cuda.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "ops.h"
#include "wait.cuh"

namespace lr {
namespace {

constexpr int kThreads = 256;

// f = sigmoid(p) and i = 1 - f, both to a few ulp: e = e^-p, f = 1 / (1 + e),
// i = e f.  e is held below 2^120 so that e f stays 1 where p is very
// negative; NaN goes through.  The instructions are the ones that flush
// denormals (an i below 2^-126 becomes 0): the others cost eight more a gate,
// a third of the forward pass's instructions.
__device__ __forceinline__ float exp_neg(float p) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(p * -1.4426950408889634f));
  return e;
}
__device__ __forceinline__ float recip(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void gate_pair(float p, float& f, float& i) {
  float e = exp_neg(p);
  asm("min.NaN.f32 %0, %0, 0f7B800000;" : "+f"(e));
  f = recip(1.0f + e);
  i = e * f;
}
__device__ __forceinline__ float gate_one(float p) { return recip(1.0f + exp_neg(p)); }

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

// ---------------------------------------------------------------------------
// Rows that TMA can read: a block takes 128 bytes of a row (64 bf16 or 32
// float32 channels of one sequence and direction), each of its four warps 16
// consecutive steps, a lane a 4-byte word.  Tiles of 64 steps arrive in a ring
// of shared memory, so that the loads of the next tiles run under the
// arithmetic of this one; every input is still read once from memory.
//
// The arithmetic comes close to the memory's time (25 instructions an element
// forward, 50 backward), hence four warps with 16 steps each rather than eight
// with 8: joining slots costs half as much an element.  Blocks of a cluster
// exchange their tiles' maps by asynchronous stores that count on a barrier of
// the receiver; a cluster-wide barrier instead cost 5 us a round.
// ---------------------------------------------------------------------------
constexpr int kWarps = 4, kSteps = 16, kTileSteps = kWarps * kSteps;
constexpr int kRow = 128, kPlane = kTileSteps * kRow;
static_assert(kTileSteps == kScanState, "a tile starts at a saved state");

struct TileP {
  CUtensorMap gx, dy;
  int T, N, H, D, groups_h;  // groups_h: channel groups of a direction
  int64_t ldg, ldy;
  const int* lengths;
  const float* h0;
  void* y;
  float* hy;
  float* states;
  const float* dhy;
  void* dgx;
  float* dh0;
  int* status;
};

__device__ __forceinline__ void tile_load(uint32_t dst, const CUtensorMap* map, int x, int n, int t,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(n), "r"(t), "r"(bar)
      : "memory");
}

// V channels of a lane from its word
template <typename E> struct Word;
template <> struct Word<bf16> {
  static constexpr int V = 2;
  static __device__ __forceinline__ void get(uint32_t w, float (&v)[2]) {
    v[0] = __uint_as_float(w << 16);
    v[1] = __uint_as_float(w & 0xffff0000u);
  }
  static __device__ __forceinline__ uint32_t put(const float (&v)[2]) { return pack2(v[0], v[1]); }
};
template <> struct Word<float> {
  static constexpr int V = 1;
  static __device__ __forceinline__ void get(uint32_t w, float (&v)[1]) { v[0] = __uint_as_float(w); }
  static __device__ __forceinline__ uint32_t put(const float (&v)[1]) { return __float_as_uint(v[0]); }
};

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// maps of V channels, one lane: (A, B) pairs
template <int V> struct alignas(8 * V) MapV { float2 m[V]; };

// this block's map to block `rank`, counting on the barrier at `bar` there
template <int V>
__device__ __forceinline__ void push(uint32_t local, uint32_t bar, unsigned rank,
                                     const float (&A)[V], const float (&B)[V]) {
  uint32_t at, rbar;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(local), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(rbar) : "r"(bar), "r"(rank));
  if (V == 2)
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
            at),
        "f"(A[0]), "f"(B[0]), "f"(A[V - 1]), "f"(B[V - 1]), "r"(rbar)
        : "memory");
  else
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(at),
        "f"(A[0]), "f"(B[0]), "r"(rbar)
        : "memory");
}

typedef std::integral_constant<bool, true> Yes;
typedef std::integral_constant<bool, false> No;

// Where a block works, and which steps of its sequence count, in walk order
// [va, vb).
template <typename E>
struct Place {
  static constexpr int V = Word<E>::V, kCh = 32 * V;
  int n, d, j0, j, va, vb;
  bool live;
  int64_t state, gh;
  __device__ __forceinline__ Place(const TileP& p, int group) {
    const int lane = threadIdx.x & 31;
    const int nd = group / p.groups_h;
    n = nd / p.D;
    d = nd - n * p.D;
    j0 = (group - nd * p.groups_h) * kCh;
    j = j0 + lane * V;
    live = j < p.H;
    state = ((int64_t)d * p.N + n) * p.H + j;
    gh = (int64_t)nd * p.H + j;
    const int len = p.lengths ? min(max(p.lengths[n], 0), p.T) : p.T;
    va = d ? p.T - len : 0;
    vb = d ? p.T : len;
  }
};

// One tile's words of a lane: 16-byte piece c of row r lies at piece
// c ^ (r & 7).  Step k of a warp is row 16 warp + k, or, walking backwards, row
// 63 - (16 warp + k); both have k's low bits, straight or inverted.
struct Words {
  uint32_t at[8];  // step k & 7, without the warp's rows
  int32_t eight;   // bytes from step k to step k + 8
  __device__ __forceinline__ Words(int warp, int d) {
    const int lane = threadIdx.x & 31, piece = (lane >> 2) ^ (d ? 7 : 0);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int row = d ? kTileSteps - 1 - (warp * kSteps + k) : warp * kSteps + k;
      at[k] = (uint32_t)(row * kRow + ((piece ^ k) << 4) + (lane & 3) * 4);
    }
    eight = d ? -8 * kRow : 8 * kRow;
  }
  __device__ __forceinline__ uint32_t get(uint32_t plane, int k) const {
    return lds32(plane + at[k & 7] + (k >= 8 ? eight : 0));
  }
};

// The maps of a tile's warps, joined; the state (or gradient) into each warp's
// steps and past the whole round.  ORDER: the warps in the walk's order (+1) or
// against it (-1).
template <int V, int ORDER>
struct Chain {
  float pA[V], pB[V], A[V], B[V];
  __device__ __forceinline__ void join(const MapV<V> (&map)[kWarps][32], int warp, int lane) {
#pragma unroll
    for (int v = 0; v < V; ++v) { A[v] = pA[v] = 1.f; B[v] = pB[v] = 0.f; }
#pragma unroll
    for (int w0 = 0; w0 < kWarps; ++w0) {
      const int w = ORDER > 0 ? w0 : kWarps - 1 - w0;
      const MapV<V> m = map[w][lane];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (w == warp) { pA[v] = A[v]; pB[v] = B[v]; }
        B[v] = fmaf(m.m[v].x, B[v], m.m[v].y);
        A[v] *= m.m[v].x;
      }
    }
  }
  // to every block of the cluster
  __device__ __forceinline__ void send(MapV<V>* tile_map, uint32_t bar, unsigned rank,
                                       unsigned csize, int warp, int lane) {
    const uint32_t at = tc::smem_addr(tile_map + rank * 32 + lane);
    if (threadIdx.x == 0) tc::mbar_arrive_expect_tx(bar, csize * 32 * sizeof(MapV<V>));
    for (unsigned c = warp; c < csize; c += kWarps) push<V>(at, bar, c, A, B);
  }
  // `in`: the value into this warp's steps; `carry` moves past the round
  __device__ __forceinline__ void receive(const MapV<V>* tile_map, uint32_t bar, uint32_t parity,
                                          unsigned rank, unsigned csize, int lane, int* status,
                                          float (&carry)[V], float (&in)[V]) {
    if (csize > 1) {
      wait_phase<true>(bar, parity, status);
      __syncwarp();
      for (unsigned c = 0; c < csize; ++c) {
        const MapV<V> m = tile_map[c * 32 + lane];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (c == rank) in[v] = carry[v];
          carry[v] = fmaf(m.m[v].x, carry[v], m.m[v].y);
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v) in[v] = fmaf(pA[v], in[v], pB[v]);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        in[v] = fmaf(pA[v], carry[v], pB[v]);
        carry[v] = fmaf(A[v], carry[v], B[v]);
      }
    }
  }
};

// The ring of tiles: `planes` planes of 64 rows of 128 bytes a stage
struct Ring {
  uint32_t base, bar0, phase = 0;
  __device__ __forceinline__ Ring(unsigned char* smem, uint64_t* bars, int n) {
    base = (tc::smem_addr(smem) + 1023u) & ~1023u;
    bar0 = tc::smem_addr(bars);
    if (threadIdx.x == 0) {
      for (int s = 0; s < n; ++s) tc::mbar_init(bar0 + 8 * s, 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    if (cluster_size() > 1) cluster_sync();  // every block runs before it is written to
  }
  __device__ __forceinline__ void wait(int s, int* status) {
    wait_phase<false>(bar0 + 8 * s, (phase >> s) & 1u, status);
    phase ^= 1u << s;
  }
};

template <typename E, bool GATE, int ST>
__global__ void __launch_bounds__(32 * kWarps, 3)
    scan_forward_tiles(const __grid_constant__ TileP p) {
  constexpr int G = GATE ? 3 : 2, V = Word<E>::V, L = kSteps;
  constexpr int kStage = G * kPlane;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bars[ST + 2];
  __shared__ __align__(16) MapV<V> map[2][kWarps][32];
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const unsigned csize = cluster_size(), rank = cluster_rank();
  const Place<E> at(p, (int)(blockIdx.x / csize));
  Ring ring(smem_raw, bars, ST + 2);
  // the cluster's tiles: [parity of the round][block][lane]
  MapV<V>* tile_map = reinterpret_cast<MapV<V>*>(smem_raw + (ring.base - tc::smem_addr(smem_raw)) + ST * kStage);
  const int rounds = (int)((p.T + (int64_t)kTileSteps * csize - 1) / ((int64_t)kTileSteps * csize));
  auto first_of = [&](int r) { return ((int64_t)r * csize + rank) * kTileSteps; };
  auto active = [&](int64_t w0) { return w0 < at.vb && w0 + kTileSteps > at.va; };
  auto load = [&](int r, int s) {
    const int64_t w0 = first_of(r);
    if (r >= rounds || !active(w0)) return;
    const int t0 = at.d ? (int)(p.T - w0 - kTileSteps) : (int)w0;
    const uint32_t bar = ring.bar0 + 8 * s;
    tc::mbar_arrive_expect_tx(bar, kStage);
#pragma unroll
    for (int b = 0; b < G; ++b)
      tile_load(ring.base + s * kStage + b * kPlane, &p.gx, (at.d * G + b) * p.H + at.j0, at.n, t0, bar);
  };
  if (threadIdx.x == 0)
    for (int r = 0; r < ST; ++r) load(r, r);
  const Words words(warp, at.d);
  float carry[V];
#pragma unroll
  for (int v = 0; v < V; ++v) carry[v] = at.live && p.h0 ? p.h0[at.state + v] : 0.f;
  const int64_t ty = (int64_t)p.N * p.ldy * (int64_t)sizeof(E);
  const int64_t step = at.d ? -ty : ty;
  char* y0 = static_cast<char*>(p.y) +
             ((int64_t)at.n * p.ldy + (int64_t)at.d * p.H + at.j0) * (int64_t)sizeof(E);
  int s = 0, before = ST - 1;  // this tile's stage and the last one's
  for (int r = 0; r < rounds; ++r) {
    __syncwarp();
    const int par = r & 1;
    const int64_t w0 = first_of(r), ws = w0 + warp * L;
    const bool on = ws < at.vb && ws + L > at.va;     // this warp has steps that count
    const bool all = ws >= at.va && ws + L <= at.vb;  // and no others
    if (active(w0)) ring.wait(s, p.status);
    const uint32_t stage = ring.base + s * kStage;
    float a[L][V], b[L][V], A[V], B[V];
#pragma unroll
    for (int v = 0; v < V; ++v) { A[v] = 1.f; B[v] = 0.f; }
    if (on) {
#pragma unroll
      for (int k = 0; k < L; ++k) {
        float pv[V], zv[V];
        Word<E>::get(words.get(stage, k), pv);
        Word<E>::get(words.get(stage + kPlane, k), zv);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float i;
          gate_pair(pv[v], a[k][v], i);
          b[k][v] = i * zv[v];
        }
      }
      if (!all) {
#pragma unroll
        for (int k = 0; k < L; ++k) {
          const bool ok = ws + k >= at.va && ws + k < at.vb;
#pragma unroll
          for (int v = 0; v < V; ++v) {
            a[k][v] = ok ? a[k][v] : 1.f;
            b[k][v] = ok ? b[k][v] : 0.f;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < L; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          B[v] = fmaf(a[k][v], B[v], b[k][v]);
          A[v] *= a[k][v];
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) map[par][warp][lane].m[v] = make_float2(A[v], B[v]);
    __syncthreads();
    // the tile before this one has been used by every warp
    if (threadIdx.x == 0 && r > 0) load(r - 1 + ST, before);
    Chain<V, 1> chain;
    chain.join(map[par], warp, lane);
    MapV<V>* tm = tile_map + par * csize * 32;
    const uint32_t xbar = ring.bar0 + 8 * (ST + par);
    if (csize > 1) chain.send(tm, xbar, rank, csize, warp, lane);
    float o[GATE ? L : 1][V];  // under the exchange
    if (GATE && on) {
#pragma unroll
      for (int k = 0; k < L; ++k) {
        float q[V];
        Word<E>::get(words.get(stage + 2 * kPlane, k), q);
#pragma unroll
        for (int v = 0; v < V; ++v) o[GATE ? k : 0][v] = gate_one(q[v]);
      }
    }
    float h[V];
    chain.receive(tm, xbar, (uint32_t)(r >> 1) & 1u, rank, csize, lane, p.status, carry, h);
    before = s;
    if (++s == ST) s = 0;
    if (ws >= p.T) continue;
    if (p.states && warp == 0 && at.live) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        p.states[ws / kScanState * ((int64_t)p.N * p.D * p.H) + at.gh + v] = h[v];
    }
    char* y = y0 + (at.d ? p.T - 1 - ws : ws) * ty;
    if (on && all) {
#pragma unroll
      for (int k = 0; k < L; ++k, y += step) {
        float out[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          h[v] = fmaf(a[k][v], h[v], b[k][v]);
          out[v] = GATE ? h[v] * o[GATE ? k : 0][v] : h[v];
        }
        if (at.live) __stcs(reinterpret_cast<uint32_t*>(y) + lane, Word<E>::put(out));
      }
    } else {
#pragma unroll
      for (int k = 0; k < L; ++k, y += step) {
        const bool ok = ws + k >= at.va && ws + k < at.vb;
        float out[V];
#pragma unroll
        for (int v = 0; v < V; ++v) out[v] = 0.f;
        if (on) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            h[v] = fmaf(a[k][v], h[v], b[k][v]);
            out[v] = GATE ? h[v] * o[GATE ? k : 0][v] : h[v];
          }
        }
        if (at.live && ws + k < p.T) __stcs(reinterpret_cast<uint32_t*>(y) + lane, ok ? Word<E>::put(out) : 0u);
      }
    }
  }
  if (p.hy && rank == 0 && warp == 0 && at.live) {
#pragma unroll
    for (int v = 0; v < V; ++v) p.hy[at.state + v] = carry[v];
  }
  if (csize > 1) cluster_sync();  // no block leaves before the others' stores to it
}

template <typename E, bool GATE, int ST>
__global__ void __launch_bounds__(32 * kWarps, 3)
    scan_backward_tiles(const __grid_constant__ TileP p) {
  constexpr int G = GATE ? 3 : 2, V = Word<E>::V, L = kSteps;
  constexpr int kStage = (G + 1) * kPlane;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bars[ST + 2];
  __shared__ __align__(16) MapV<V> map[2][kWarps][32];  // against the walk
  __shared__ float forth[2][kWarps][V][32];             // B of the walk's maps
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const unsigned csize = cluster_size(), rank = cluster_rank();
  const Place<E> at(p, (int)(blockIdx.x / csize));
  Ring ring(smem_raw, bars, ST + 2);
  MapV<V>* tile_map = reinterpret_cast<MapV<V>*>(smem_raw + (ring.base - tc::smem_addr(smem_raw)) + ST * kStage);
  const int tiles = (p.T + kTileSteps - 1) / kTileSteps;
  const int rounds = (int)((tiles + (int64_t)csize - 1) / csize);
  // tiles from the end of the walk; one before its start is empty
  auto tile_of = [&](int r) { return tiles - 1 - (int64_t)r * csize - rank; };
  auto active = [&](int64_t tile) {
    return tile >= 0 && tile * kTileSteps < at.vb && (tile + 1) * kTileSteps > at.va;
  };
  auto load = [&](int r, int s) {
    const int64_t tile = tile_of(r);
    if (r >= rounds || !active(tile)) return;
    const int t0 = at.d ? (int)(p.T - (tile + 1) * kTileSteps) : (int)(tile * kTileSteps);
    const uint32_t bar = ring.bar0 + 8 * s, dst = ring.base + s * kStage;
    tc::mbar_arrive_expect_tx(bar, kStage);
#pragma unroll
    for (int b = 0; b < G; ++b)
      tile_load(dst + b * kPlane, &p.gx, (at.d * G + b) * p.H + at.j0, at.n, t0, bar);
    tile_load(dst + G * kPlane, &p.dy, at.d * p.H + at.j0, at.n, t0, bar);
  };
  if (threadIdx.x == 0)
    for (int r = 0; r < ST; ++r) load(r, r);
  const Words words(warp, at.d);
  const int64_t states_row = (int64_t)p.N * p.D * p.H;
  auto state_of = [&](int r, float (&h)[V]) {
    const int64_t tile = tile_of(r);
#pragma unroll
    for (int v = 0; v < V; ++v)
      h[v] = r < rounds && active(tile) && at.live ? __ldg(p.states + tile * states_row + at.gh + v) : 0.f;
  };
  float carry[V], next[V];
#pragma unroll
  for (int v = 0; v < V; ++v) carry[v] = at.live && p.dhy ? p.dhy[at.state + v] : 0.f;
  state_of(0, next);
  const int64_t tg = (int64_t)p.N * p.ldg * (int64_t)sizeof(E);
  const int64_t step = at.d ? tg : -tg;  // from a step to the one before it
  const int64_t bytes_h = (int64_t)p.H * (int64_t)sizeof(E);
  char* d0 = static_cast<char*>(p.dgx) +
             ((int64_t)at.n * p.ldg + (int64_t)at.d * G * p.H + at.j0) * (int64_t)sizeof(E);
  int s = 0, before = ST - 1;
  for (int r = 0; r < rounds; ++r) {
    __syncwarp();
    const int par = r & 1;
    const int64_t tile = tile_of(r), ws = tile * kTileSteps + warp * L;
    const bool on = tile >= 0 && ws < at.vb && ws + L > at.va;
    const bool all = on && ws >= at.va && ws + L <= at.vb;
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = next[v];
    state_of(r + 1, next);
    if (active(tile)) ring.wait(s, p.status);
    const uint32_t stage = ring.base + s * kStage;
    float f[L][V], i[L][V], A[V], B[V], C[V];
#pragma unroll
    for (int v = 0; v < V; ++v) { A[v] = 1.f; B[v] = C[v] = 0.f; }
    auto first_pass = [&](auto full) {
#pragma unroll
      for (int k = 0; k < L; ++k) {
        float pv[V], zv[V];
        Word<E>::get(words.get(stage, k), pv);
        Word<E>::get(words.get(stage + kPlane, k), zv);
        const bool ok = full.value || (ws + k >= at.va && ws + k < at.vb);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          gate_pair(pv[v], f[k][v], i[k][v]);
          const float b = i[k][v] * zv[v];
          f[k][v] = ok ? f[k][v] : 1.f;
          A[v] *= f[k][v];
          B[v] = fmaf(f[k][v], B[v], ok ? b : 0.f);
        }
      }
#pragma unroll
      for (int k = L - 1; k >= 0; --k) {
        float dv[V], q[V];
        Word<E>::get(words.get(stage + G * kPlane, k), dv);
        if (GATE) Word<E>::get(words.get(stage + 2 * kPlane, k), q);
        const bool ok = full.value || (ws + k >= at.va && ws + k < at.vb);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float direct = GATE ? dv[v] * gate_one(q[v]) : dv[v];
          C[v] = f[k][v] * (C[v] + (ok ? direct : 0.f));
        }
      }
    };
    if (all) first_pass(Yes());
    else if (on) first_pass(No());
#pragma unroll
    for (int v = 0; v < V; ++v) {
      map[par][warp][lane].m[v] = make_float2(A[v], C[v]);
      forth[par][warp][v][lane] = B[v];
    }
    __syncthreads();
    if (threadIdx.x == 0 && r > 0) load(r - 1 + ST, before);
    Chain<V, -1> chain;
    chain.join(map[par], warp, lane);
    MapV<V>* tm = tile_map + par * csize * 32;
    const uint32_t xbar = ring.bar0 + 8 * (ST + par);
    if (csize > 1) chain.send(tm, xbar, rank, csize, warp, lane);
    // under the exchange: the state before each step
    float hb[L][V];
    if (on) {
#pragma unroll
      for (int w = 0; w < kWarps - 1; ++w)
        if (w < warp) {
#pragma unroll
          for (int v = 0; v < V; ++v) h[v] = fmaf(map[par][w][lane].m[v].x, h[v], forth[par][w][v][lane]);
        }
      auto states = [&](auto full) {
#pragma unroll
        for (int k = 0; k < L; ++k) {
          float zv[V];
          Word<E>::get(words.get(stage + kPlane, k), zv);
          const bool ok = full.value || (ws + k >= at.va && ws + k < at.vb);
#pragma unroll
          for (int v = 0; v < V; ++v) {
            hb[k][v] = h[v];
            const float b = i[k][v] * zv[v];
            h[v] = fmaf(f[k][v], h[v], ok ? b : 0.f);
          }
        }
      };
      if (all) states(Yes());
      else states(No());
    }
    float c[V];
    chain.receive(tm, xbar, (uint32_t)(r >> 1) & 1u, rank, csize, lane, p.status, carry, c);
    before = s;
    if (++s == ST) s = 0;
    if (tile < 0 || ws >= p.T) continue;
    // from the warp's last step back
    const int64_t tl = at.d ? p.T - ws - L : ws + L - 1;
    char* d = d0 + tl * tg;
    if (!on) {
      for (int k = L - 1; k >= 0; --k, d += step)
        if (at.live && ws + k < p.T)
          for (int b = 0; b < G; ++b) __stcs(reinterpret_cast<uint32_t*>(d + b * bytes_h) + lane, 0u);
      continue;
    }
    auto gradients = [&](auto full) {
#pragma unroll
      for (int k = L - 1; k >= 0; --k, d += step) {
        float zv[V], dv[V], qv[V], gp[V], gz[V], gq[V];
        Word<E>::get(words.get(stage + kPlane, k), zv);
        Word<E>::get(words.get(stage + G * kPlane, k), dv);
        if (GATE) Word<E>::get(words.get(stage + 2 * kPlane, k), qv);
        const bool ok = full.value || (ws + k >= at.va && ws + k < at.vb);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float o = 1.f, oi = 0.f;
          if (GATE) gate_pair(qv[v], o, oi);
          const float od = GATE ? o * dv[v] : dv[v];
          const float dh = od + c[v];
          gz[v] = dh * i[k][v];
          gp[v] = gz[v] * (hb[k][v] - zv[v]) * f[k][v];
          if (GATE) gq[v] = od * oi * h[v];
          h[v] = hb[k][v];  // the state after the step before
          c[v] = ok ? f[k][v] * dh : c[v];
        }
        if (at.live && (full.value || ws + k < p.T)) {
          uint32_t* o = reinterpret_cast<uint32_t*>(d) + lane;
          __stcs(o, ok ? Word<E>::put(gp) : 0u);
          __stcs(reinterpret_cast<uint32_t*>(d + bytes_h) + lane, ok ? Word<E>::put(gz) : 0u);
          if (GATE) __stcs(reinterpret_cast<uint32_t*>(d + 2 * bytes_h) + lane, ok ? Word<E>::put(gq) : 0u);
        }
      }
    };
    if (all) gradients(Yes());
    else gradients(No());
  }
  if (p.dh0 && rank == 0 && warp == 0 && at.live) {
#pragma unroll
    for (int v = 0; v < V; ++v) p.dh0[at.state + v] = carry[v];
  }
  if (csize > 1) cluster_sync();
}

// A few steps: one thread four (or one) channels, all steps in turn.
template <typename E, int V, bool GATE>
__global__ void __launch_bounds__(kThreads) scan_steps_kernel(const ScanP p) {
  constexpr int G = GATE ? 3 : 2;
  const Lane l = lane_of(p, (int64_t)blockIdx.x * kThreads + threadIdx.x, V, G);
  if (!l.live) return;
  const E* gx = static_cast<const E*>(p.gx) + l.g0;
  E* y = static_cast<E*>(p.y) + l.y0;
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = p.h0 ? p.h0[l.state + v] : 0.f;
  if (p.states)
#pragma unroll
    for (int v = 0; v < V; ++v) p.states[l.gh + v] = h[v];
  for (int w = 0; w < (int)p.T; ++w) {
    const int64_t t = l.d ? p.T - 1 - w : w;
    float out[V];
#pragma unroll
    for (int v = 0; v < V; ++v) out[v] = 0.f;
    if (t < l.len) {
      const E* row = gx + t * p.N * p.ldg;
      const Raw<E, V> rp = load_raw<E, V>(row), rz = load_raw<E, V>(row + p.H);
      Raw<E, V> rq;
      if (GATE) rq = load_raw<E, V>(row + 2 * p.H);
      float pv[V], zv[V], qv[V];
      unpack(rp, pv);
      unpack(rz, zv);
      if (GATE) unpack(rq, qv);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float f, i, o, oi;
        gate_pair(pv[v], f, i);
        h[v] = fmaf(f, h[v], i * zv[v]);
        out[v] = h[v];
        if (GATE) {
          gate_pair(qv[v], o, oi);
          out[v] *= o;
        }
      }
    }
    store_v(y + t * p.N * p.ldy, out);
  }
  if (p.hy)
#pragma unroll
    for (int v = 0; v < V; ++v) p.hy[l.state + v] = h[v];
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

// TMA's conditions: 16-byte rows, blocks and bases; and channels for at least
// half a block's width
bool by_tiles(const ScanArgs& a) {
  const int64_t e = a.bf16 ? 2 : 4;
  auto ok = [&](const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; };
  return a.H * e % 16 == 0 && a.ldg * e % 16 == 0 && a.ldy * e % 16 == 0 && ok(a.gx) && ok(a.y) &&
         ok(a.dy) && ok(a.dgx) && a.H * e >= kRow / 2;
}

template <typename E, typename K>
cudaError_t run_tiles(K kernel, const ScanArgs& a, int planes, int stages, cudaStream_t st) {
  constexpr int kCh = Word<E>::V * 32;
  const int G = a.gate ? 3 : 2;
  TileP p = {};
  p.T = (int)a.T; p.N = (int)a.N; p.H = (int)a.H; p.D = (int)a.D;
  p.groups_h = (int)((a.H + kCh - 1) / kCh);
  p.ldg = a.ldg; p.ldy = a.ldy;
  p.lengths = a.lengths; p.h0 = a.h0; p.y = a.y; p.hy = a.hy; p.states = a.states;
  p.dhy = a.dhy; p.dgx = a.dgx; p.dh0 = a.dh0;
  p.status = a.status;
  const uint32_t box[3] = {(uint32_t)kCh, 1u, (uint32_t)kTileSteps};
  auto map = [&](CUtensorMap* m, const void* ptr, int64_t width, int64_t ld) {
    const uint64_t dims[3] = {(uint64_t)width, (uint64_t)a.N, (uint64_t)a.T};
    const uint64_t strides[2] = {(uint64_t)ld * sizeof(E), (uint64_t)(a.N * ld) * sizeof(E)};
    return tma_encode(m, 3, a.bf16, ptr, dims, strides, box);
  };
  if (!map(&p.gx, a.gx, a.D * G * a.H, a.ldg) || (a.dy && !map(&p.dy, a.dy, a.D * a.H, a.ldy)))
    return cudaErrorInvalidValue;
  // blocks of a cluster share a channel group's tiles where the groups alone
  // give the card less than two blocks an SM
  const int64_t groups = a.N * a.D * p.groups_h, tiles = (a.T + kTileSteps - 1) / kTileSteps;
  int csize = 1;
  while (csize < 16 && groups * csize < 2 * a.num_sms && csize < tiles) csize *= 2;
  const size_t smem = (size_t)stages * planes * kPlane + 1024 +
                      (csize > 1 ? 2 * csize * 32 * sizeof(MapV<Word<E>::V>) : 0);
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess && csize > 8)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(groups * csize));
  cfg.blockDim = dim3(32 * kWarps);
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

// Stages of the ring: two tiles in flight a block.  A third leaves room for
// two blocks an SM instead of three and measured slower (65536 x 1 x 1024
// forward 158 -> 222 us, 512 x 128 x 1024 training 353 -> 386 us).
template <typename E>
cudaError_t forward_tiles(const ScanArgs& a, cudaStream_t st) {
  return a.gate ? run_tiles<E>(scan_forward_tiles<E, true, 2>, a, 3, 2, st)
                : run_tiles<E>(scan_forward_tiles<E, false, 3>, a, 2, 3, st);
}
template <typename E>
cudaError_t backward_tiles(const ScanArgs& a, cudaStream_t st) {
  return a.gate ? run_tiles<E>(scan_backward_tiles<E, true, 2>, a, 4, 2, st)
                : run_tiles<E>(scan_backward_tiles<E, false, 2>, a, 3, 2, st);
}

template <typename E, int V>
cudaError_t forward_steps(const ScanArgs& a, cudaStream_t st) {
  const ScanP p = params(a, V);
  const unsigned blocks = (unsigned)((p.vecs + kThreads - 1) / kThreads);
  if (a.gate) scan_steps_kernel<E, V, true><<<blocks, kThreads, 0, st>>>(p);
  else scan_steps_kernel<E, V, false><<<blocks, kThreads, 0, st>>>(p);
  g_kernel_launches.fetch_add(1, std::memory_order_relaxed);
  return cudaGetLastError();
}

}  // namespace

cudaError_t scan_forward(const ScanArgs& a, cudaStream_t st) {
  const bool four = by_four(a);
  if (a.T <= 8) {
    if (four) return a.bf16 ? forward_steps<bf16, 4>(a, st) : forward_steps<float, 4>(a, st);
    return a.bf16 ? forward_steps<bf16, 1>(a, st) : forward_steps<float, 1>(a, st);
  }
  if (by_tiles(a)) return a.bf16 ? forward_tiles<bf16>(a, st) : forward_tiles<float>(a, st);
  if (four)
    return a.bf16 ? run<bf16, 4, 16, 8, false>(a, st) : run<float, 4, 16, 8, false>(a, st);
  return a.bf16 ? run<bf16, 1, 32, 16, false>(a, st) : run<float, 1, 32, 16, false>(a, st);
}

cudaError_t scan_backward(const ScanArgs& a, cudaStream_t st) {
  if (by_tiles(a)) return a.bf16 ? backward_tiles<bf16>(a, st) : backward_tiles<float>(a, st);
  if (by_four(a))
    return a.bf16 ? run<bf16, 4, 16, 8, true>(a, st) : run<float, 4, 16, 4, true>(a, st);
  return a.bf16 ? run<bf16, 1, 32, 8, true>(a, st) : run<float, 1, 32, 8, true>(a, st);
}

}  // namespace lr
