// What the kernels of a warp per key step share (few rows of bf16, fp32): a finished row's output and
// the join of a block's warps and of a cluster's blocks.
#pragma once

#include <cooperative_groups.h>

#include "lla_paged.cuh"
#include "lla_tc_ptx.cuh"

namespace lla {
namespace paged {
namespace {

using tc::cp_async16;
using tc::cp_async_commit;
using tc::cp_async_wait;
using tc::smem_u32;

constexpr int KT = 16;  // keys per tile: within one page, since pages hold a multiple of 16
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// The rows of a block: row r is token t0 + (r0 + r) / width (positions from p0 on) and head h0 + (r0 + r) % width.
struct Rows {
  int t0, p0, p1, width, h0, r0 = 0;
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The nodes of a sequence of at most 64: of each the nodes that it sees (its parent, its parent's, .. and itself,
// less those that fell out of the window) as bits, and its position. One warp, lane l has nodes l and l + 32;
// parents come from the other lanes, so a tree costs one load and no launch before this one's.
__device__ __forceinline__ void small_tree(const Params& p, const Seq& sq, uint64_t* bits_of, int* pos_of) {
  const int lane = threadIdx.x & 31, n = min(sq.n, 64);
  int parent[2];
  bool bad = false;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = lane + 32 * h, a = i < n ? __ldg(p.parents + sq.t0 + i) : -1;
    bad |= a < -1 || a >= i;
    parent[h] = a < i ? max(a, -1) : -1;
  }
  if (bad) atomicOr(p.status, kStatusBadIndex);
  auto up = [&](int a) {  // whole warps call
    const int x = __shfl_sync(0xffffffffu, parent[0], a & 31), y = __shfl_sync(0xffffffffu, parent[1], a & 31);
    return a < 0 ? -1 : a < 32 ? x : y;
  };
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = lane + 32 * h;
    uint64_t bits = 1ull << i;
    int d = 0;
    for (int a = parent[h]; __any_sync(0xffffffffu, a >= 0); a = up(a)) {
      if (a >= 0) {
        bits |= 1ull << a;
        ++d;
      }
    }
    if (p.window < n) {
      int steps = 1;
      for (int a = parent[h]; __any_sync(0xffffffffu, a >= 0); a = up(a), ++steps)
        if (a >= 0 && steps >= p.window && sq.first + d - steps >= p.sinks) bits &= ~(1ull << a);
    }
    bits_of[i] = bits;
    pos_of[i] = sq.first + d;
  }
}

// A finished row's sums {m, d1, d2, d1 of the rounded weights} (the last one used where weights are
// rounded and differences of sums taken: bf16 with a probe), o1[c] and o2[c] its unnormalised columns
// lane * VC + c: writes out and lse.
template <typename T, bool PROBE>
constexpr bool kRoundedSum = PROBE && sizeof(T) == 2;
template <typename T, int D, bool PROBE>
__device__ __forceinline__ void write_row(const Params& p, const Seq& sq, int b, const Rows& rows, int r, float4 st,
                                           const float (&o1)[D / 32], const float (&o2)[D / 32]) {
  constexpr int VC = D / 32;
  const int lane = threadIdx.x & 31;
  const int token = rows.t0 + (rows.r0 + r) / rows.width, head = rows.h0 + (rows.r0 + r) % rows.width;
  const float s1 = st.y, norm = kRoundedSum<T, PROBE> ? st.w : s1;
  const float inv = norm == 0.f ? 0.f : 1.f / norm, f1 = (1.f + st.z * inv) * inv;
  T* dst = static_cast<T*>(p.out) + ((long long)token * p.Hq + head) * p.dv + lane * VC;
  float bad = 0.f, y[VC];
#pragma unroll
  for (int c = 0; c < VC; ++c) {
    y[c] = PROBE ? fmaf(o1[c], f1, -o2[c] * inv) : o1[c] * inv;
    bad += y[c] * 0.f;
  }
  if (lane * VC < p.dv) {
    if constexpr (sizeof(T) == 4) {
      if constexpr (VC == 4) *reinterpret_cast<float4*>(dst) = make_float4(y[0], y[1], y[2], y[3]);
      else *reinterpret_cast<float2*>(dst) = make_float2(y[0], y[1]);
    } else {
      uint32_t w[VC / 2];
#pragma unroll
      for (int c = 0; c < VC; c += 2) w[c / 2] = pack_bf16(y[c], y[c + 1]);
      if constexpr (VC == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
      else *reinterpret_cast<uint32_t*>(dst) = w[0];
    }
  }
  if (p.lse && lane == 0)
    p.lse[(long long)token * p.Hq + head] =
        s1 == 0.f ? -CUDART_INF_F : (st.x * (p.inv_h * kLog2e) + log2f(s1)) * kLn2;
  if (__any_sync(0xffffffffu, !(bad == 0.f))) {
    repair_row<T, KT>(p, sq, b, rows.p0, rows.p1, token, head, s1);
  }
}

// Adds a part's sums, taken against another reference (factor f).
template <bool ROUNDED>
__device__ __forceinline__ void add_sums(float4& sum, const float4& st, float f) {
  sum.y = fmaf(st.y, f, sum.y);
  sum.z = fmaf(st.z, f, sum.z);
  if (ROUNDED) sum.w = fmaf(st.w, f, sum.w);
}

// The join of a block's NW warps, and of the cluster's blocks where a pair's blocks are one
// (CLUSTER): O [warp][OROWS][D + 4] in `os` (a row's O2 ROWS rows behind its O1), its sums in `stats`; the block's own sums go to `fin` [OROWS][D] and `fin_stats`, to the scratch (more splits than
// a cluster has: row at(r), `cols` floats to a row's O), or finished to the output. All threads, behind a
// barrier.
template <typename T, int D, bool PROBE, bool CLUSTER, int NW, int ROWS, int OROWS, typename At>
__device__ __forceinline__ void join_block(const Params& p, const Seq& sq, int b, const Rows& rows, int part,
                                           int nrows, At at, int cols, const float* os, const float4 (&stats)[NW][16], float* fin,
                                           float4* fin_stats) {
  constexpr int VC = D / 32, OP = D + 4;  // columns per lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float c2 = p.inv_h * kLog2e;
  for (int r = warp; r < nrows; r += NW) {
    float top = -CUDART_INF_F;
#pragma unroll
    for (int i = 0; i < NW; ++i) top = fmaxf(top, stats[i][r].x);
    const float ref = top == -CUDART_INF_F ? 0.f : top * c2;
    float4 sum = make_float4(top, 0.f, 0.f, 0.f);
    float o1[VC] = {}, o2[VC] = {};
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const float4 st = stats[i][r];
      const float f = ex2(fmaf(st.x, c2, -ref));
      add_sums<kRoundedSum<T, PROBE>>(sum, st, f);
#pragma unroll
      for (int c = 0; c < VC; ++c) {
        o1[c] = fmaf(os[(i * OROWS + r) * OP + lane * VC + c], f, o1[c]);
        if (PROBE) o2[c] = fmaf(os[(i * OROWS + r + ROWS) * OP + lane * VC + c], f, o2[c]);
      }
    }
    if (CLUSTER) {
      if (lane == 0) fin_stats[r] = sum;
      float* dst = fin + r * D + lane * VC;
#pragma unroll
      for (int c = 0; c < VC; ++c) {
        dst[c] = o1[c];
        if (PROBE) dst[ROWS * D + c] = o2[c];
      }
    } else if (p.split > 1) {
      const long long id = at(r);
      if (lane == 0) p.part_s[id] = sum;
      if (lane * VC < cols) {
        float* dst = p.part_o + id * (PROBE ? 2 : 1) * cols + lane * VC;
#pragma unroll
        for (int c = 0; c < VC; ++c) {
          dst[c] = o1[c];
          if (PROBE) dst[cols + c] = o2[c];
        }
      }
    } else {
      write_row<T, D, PROBE>(p, sq, b, rows, r, sum, o1, o2);
    }
  }
  if constexpr (CLUSTER) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    for (int r = warp * p.split + part; r < nrows; r += NW * p.split) {  // this warp's rows
      float4 st[kRowsCluster];
      float top = -CUDART_INF_F;
#pragma unroll
      for (int i = 0; i < kRowsCluster; ++i)
        if (i < p.split) {
          st[i] = *cluster.map_shared_rank(&fin_stats[r], i);
          top = fmaxf(top, st[i].x);
        }
      const float ref = top == -CUDART_INF_F ? 0.f : top * c2;
      float4 sum = make_float4(top, 0.f, 0.f, 0.f);
      float o1[VC] = {}, o2[VC] = {};
#pragma unroll
      for (int i = 0; i < kRowsCluster; ++i)
        if (i < p.split) {
          const float f = ex2(fmaf(st[i].x, c2, -ref));
          add_sums<kRoundedSum<T, PROBE>>(sum, st[i], f);
          const float* src = cluster.map_shared_rank(fin, i) + r * D + lane * VC;
#pragma unroll
          for (int c = 0; c < VC; ++c) {
            o1[c] = fmaf(src[c], f, o1[c]);
            if (PROBE) o2[c] = fmaf(src[ROWS * D + c], f, o2[c]);
          }
        }
      write_row<T, D, PROBE>(p, sq, b, rows, r, sum, o1, o2);
    }
    cluster.sync();  // this block's sums have been read
  }
}

}  // namespace
}  // namespace paged
}  // namespace lla
