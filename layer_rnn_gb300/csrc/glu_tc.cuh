// What the tensor-core kernels of the gated feed-forward share (bfloat16:
// glu.cu, float32: glu_f32.cu): pairs of blocks that walk tiles of a result,
// some of them cut along the contraction, TMA loads and tcgen05 MMAs over both
// blocks of a pair.
#pragma once

#include <cuda.h>

#include <algorithm>

#include "glu.cuh"
#include "launch.cuh"
#include "ops.h"
#include "wait.cuh"

namespace lr {
namespace glu {

constexpr int kHalf = 128;  // rows of a tile that one block of the pair holds

enum Product { kForward = 0, kDgu = 1, kDx = 2, kDw = 3 };

struct P {
  int m_tiles, n_tiles, planes;  // tiles of a plane of the result; planes (kDw: 2)
  int nkb, kb_plane;             // 64-element blocks of the contraction; per plane (kDx)
  int whole;                     // tiles done whole, in turn; the rest is cut
  int head;                      // blocks of a cut tile that one pair does first
  int rows, cols;                // of a plane of the result
  int group;                     // row tiles walked together (reuse in L2)
  int tma_out, tma_dy;
  void* out;                     // plain stores: row pitch ld_out, planes `rows` rows apart
  int64_t ld_out;
  const void* dy;                // plain loads
  int64_t ld_dy;
  float* part;                   // partial tiles of the pairs, two each
  const unsigned* amax;          // float32 operands as scaled fp16 pairs: the largest
  const unsigned* bmax;          // magnitudes (float bit patterns)
  unsigned* omax;                // kDgu: that of the result
  int* status;
};

__device__ __forceinline__ uint32_t map_rank(uint32_t addr, unsigned rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// box at {x, y, z} into this block's shared memory; the bytes count on `bar`,
// which may be the pair's other block's
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void store_box(const CUtensorMap* map, uint32_t src, int x, int y,
                                          int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(x), "r"(y), "r"(z), "r"(src)
      : "memory");
}

__device__ __forceinline__ void mma2(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                     uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// arrive on the barrier at this offset in both blocks once the MMAs are done
__device__ __forceinline__ void commit2(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(bar),
      "h"((unsigned short)3)
      : "memory");
}
// Arrive on a barrier of either block.  What it orders is reads of tensor memory
// (tcgen05.fence before it), not stores: a release at cluster scope would wait for
// the thread's stores as well, 3000 cycles at times.
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// operand tile of 128 rows (or columns) x 64 k, 128-byte swizzle.  K-major:
// rows of 128 bytes, groups of 8 rows 1024 bytes apart; 16 k further on is 32
// bytes.  MN-major: two boxes of 64 elements x 64 k (8192 bytes apart), groups
// of 8 k 1024 bytes apart; 16 k further on is 2048 bytes.
template <bool MN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(MN ? 8192 >> 4 : 1) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// What a pair works on, in order: whole tiles in turn, then its share of the
// `left` tiles that are cut along the contraction.  Pair r < left takes the first
// `head` blocks of cut tile r; the other pairs share the tiles' ends, laid end to
// end, evenly.  (Heads run side by side through the same part of the contraction
// and share its operands in L2.  Cutting all of it evenly instead had every pair
// in another part: dW of 65536 x 1024 x 4096 read 3.4 GB that way.)
struct Walk {
  int tile, kb0, kb1;
  int slot;          // of the partial sums, or -1: the whole tile
  int64_t pos, to;   // in the ends; heads: pos = -1, done: pos = to
};
struct Cut {
  int left, ends;    // cut tiles; blocks of an end
  __device__ __forceinline__ explicit Cut(const P& p)
      : left(p.m_tiles * p.n_tiles * p.planes - p.whole), ends(p.nkb - p.head) {}
  // where tail pair j (pair left + j) begins
  __device__ __forceinline__ int64_t begin(int64_t j, int pairs) const {
    return pairs > left ? j * ((int64_t)left * ends) / (pairs - left) : 0;
  }
};
__device__ __forceinline__ void walk_start(const P& p, Walk& w, int pair, int pairs) {
  w.tile = pair - pairs;
  const Cut c(p);
  w.pos = w.to = 0;
  if (c.left == 0) return;
  if (pair < c.left) {
    w.pos = -1;
  } else {
    w.pos = c.begin(pair - c.left, pairs);
    w.to = c.begin(pair - c.left + 1, pairs);
  }
}
__device__ __forceinline__ bool walk_next(const P& p, Walk& w, int pair, int pairs) {
  if (w.tile + pairs < p.whole) {
    w.tile += pairs;
    w.kb0 = 0;
    w.kb1 = p.nkb;
    w.slot = -1;
    return true;
  }
  w.tile = p.whole;  // whole tiles are done
  const Cut c(p);
  if (w.pos < 0) {
    w.tile = p.whole + pair;
    w.kb0 = 0;
    w.kb1 = p.head;
    w.slot = pair;
    w.pos = w.to = 0;
    return true;
  }
  if (w.pos >= w.to) return false;
  const int rel = (int)(w.pos / c.ends), at = (int)(w.pos - (int64_t)rel * c.ends);
  const int n = (int)min((int64_t)(c.ends - at), w.to - w.pos);
  w.tile = p.whole + rel;
  w.kb0 = p.head + at;
  w.kb1 = w.kb0 + n;
  w.slot = pair + rel;  // left + (pair - left) + rel: unique, since both only rise
  w.pos += n;
  return true;
}
// tile number -> plane, row tile, column tile: `group` row tiles at a time,
// rows fastest, so that pairs at work together share columns of one operand
// and a few rows of the other
__device__ __forceinline__ void tile_at(const P& p, int tile, int& z, int& mt, int& nt) {
  const int plane = p.m_tiles * p.n_tiles;
  z = tile / plane;
  tile -= z * plane;
  const int span = p.group * p.n_tiles, g = tile / span;
  tile -= g * span;
  const int rows = min(p.group, p.m_tiles - g * p.group);
  nt = tile / rows;
  mt = g * p.group + tile - nt * rows;
}

__device__ __forceinline__ void store4(bf16* o, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(o) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
}
__device__ __forceinline__ void store4(float* o, const float (&v)[4]) {
  *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
}

// A partial tile of TN columns: float4 of 4 columns, [block][row quarter][TN / 4]
// [row], so that the 32 lanes of a warp store and load 512 bytes in a line.
template <int TN>
__device__ __forceinline__ float4* part_at(const P& p, int64_t slot, int part) {
  return reinterpret_cast<float4*>(p.part) + (slot * 8 + part) * (TN / 4 * 32);
}

// Joins the partial tiles: block x handles four columns of 32 rows for each of its
// warps, in one cut tile's eighth (block of the pair * 4 + row quarter).  Pairs in
// rising order.
template <typename E, int TN>
__global__ void __launch_bounds__(256) glu_join_kernel(const P p, int pairs) {
  constexpr int kBlocks = TN / 4 * 32 / 256;  // of an eighth
  const int part = blockIdx.x / kBlocks & 7;
  const int rel = blockIdx.x / kBlocks >> 3, tile = p.whole + rel;
  int z, mt, nt;
  tile_at(p, tile, z, mt, nt);
  const Cut c(p);
  // the pairs that hold parts of this tile's end
  const int64_t t0 = (int64_t)rel * c.ends, t1 = t0 + c.ends;
  int first = (int)(t0 * (pairs - c.left) / ((int64_t)c.left * c.ends));
  while (first > 0 && c.begin(first, pairs) > t0) --first;
  while (c.begin(first + 1, pairs) <= t0) ++first;
  const int row0 = mt * 2 * kHalf + (part >> 2) * kHalf + (part & 3) * 32;
  E* out = static_cast<E*>(p.out);
  const bool by_four = p.ld_out % 4 == 0 && reinterpret_cast<uintptr_t>(out) % (4 * sizeof(E)) == 0;
  const int i = blockIdx.x % kBlocks * 256 + threadIdx.x;
  next_may_start();
  wait_for_last();
  float4 s = __ldcs(part_at<TN>(p, rel, part) + i);
  for (int j = first; j < pairs - c.left && c.begin(j, pairs) < t1; ++j) {
    if (c.begin(j + 1, pairs) == c.begin(j, pairs)) continue;
    const float4 v = __ldcs(part_at<TN>(p, c.left + j + rel, part) + i);
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
  }
  const int row = row0 + (i & 31), col = nt * TN + (i >> 5) * 4;
  if (row >= p.rows || col >= p.cols) return;
  E* o = out + ((int64_t)z * p.rows + row) * p.ld_out + col;
  const float v[4] = {s.x, s.y, s.z, s.w};
  if (by_four && col + 4 <= p.cols) {
    store4(o, v);
  } else {
    for (int u = 0; u < 4 && col + u < p.cols; ++u) o[u] = from_f<E>(v[u]);
  }
}
template <typename E, int TN>
cudaError_t launch_join(const P& p, int64_t cut_tiles, int pairs, cudaStream_t st) {
  return launch_kernel(glu_join_kernel<E, TN>, (unsigned)(cut_tiles * 8 * (TN / 4 * 32 / 256)), 256, 0, 0,
                       st, p, pairs);
}

// Pairs of blocks at work, and how many tiles (p.whole) they do whole.  Tiles
// of a last, unfilled round are cut along the contraction, all pairs taking an
// equal part, where that frees more than `least` blocks of 64 k: what a
// partial tile costs to write and read again.  A round that is more than four
// fifths full is left as it is: it would be cut into many small ends.
inline int plan_pairs(P* p, int num_sms, int least) {
  const int64_t tiles = (int64_t)p->m_tiles * p->n_tiles * p->planes;
  int pairs = std::max(1, std::min(num_sms / 2, kGluMaxPairs));
  p->whole = (int)tiles;
  p->head = p->nkb;
  const int64_t over = tiles % pairs;
  if (p->part && over && 5 * over <= 4 * pairs) {
    const int64_t each = (over * p->nkb + pairs - 1) / pairs;
    if (p->nkb - each > least) {
      p->whole = (int)(tiles - over);
      p->head = (int)each;
    }
  }
  if (p->whole == tiles) pairs = (int)std::min<int64_t>(pairs, tiles);
  return pairs;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round256(int64_t v) { return ceil_div(v, 256) * 256; }
inline int64_t pad8(int64_t v) { return ceil_div(v, 8) * 8; }

// three-dimensional map of 16-bit rows: boxes of 64 columns
inline bool map3(CUtensorMap* m, const void* ptr, int64_t cols, int64_t rows, int64_t planes,
                 int64_t ld, int64_t plane_rows, uint32_t box_rows) {
  const uint64_t dims[3] = {(uint64_t)cols, (uint64_t)rows, (uint64_t)planes};
  const uint64_t strides[2] = {(uint64_t)ld * 2, (uint64_t)(ld * plane_rows) * 2};
  const uint32_t box[3] = {64u, box_rows, 1u};
  return tma_encode(m, 3, true, ptr, dims, strides, box);
}

}  // namespace glu
}  // namespace lr
