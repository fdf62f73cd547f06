// Eviction from a paged cache by accumulated attention weight. For every (sequence, key/value
// head): of its n positions keep m = min(n, budget): the first `sinks`, the last `recent`, and of
// the others those with the largest mass (equal mass: the lower position; NaN counts as the
// lowest), in their order; their keys, values and mass go to slots 0 .. m-1 of the destination's
// pages.
//
// Selection is a search for the need-th largest value, by radix: the fp32 mass maps to an unsigned
// key of the same order, and three histograms (11, 11 and 10 bits from the top) of the candidates
// that agree with the digits found so far give the threshold T and how many positions equal to T
// are still wanted; a prefix sum over positions then numbers the kept ones. One cluster of up to
// 8 CTAs serves a (sequence, head): each holds its share of the keys in shared memory (the mass is
// read from HBM once) and the CTAs add up their histograms through distributed shared memory, so a
// single long sequence still spreads over several SMs and no scratch or second launch is needed.
// The kept rows are then gathered by a copy kernel (16-byte accesses, 32 rows a warp): HBM-bound,
// each kept row read once and written once. Measured: 16 sequences of 9k to 33k, 8 heads of 128, to
// 8192: selection 30 us, gather 161 us (6.6 TB/s, 97 % of the copy bandwidth); one sequence of 4000, 8
// heads of 64, to 1000: 13 us, the barriers of three radix passes and two launches.
#include <cooperative_groups.h>

#include "lla_paged.cuh"

namespace lla {
namespace paged {
namespace {

namespace cg = cooperative_groups;

constexpr int NT = 512;
constexpr int BINS = 2048;

struct Evict {
  void* k;            // destination pages
  void* v;
  float* mass;
  const int* table;
  int* lens;
  int* kept;          // [B, Hkv, budget]
  int max_pages, num_pages;
  int budget, sinks, recent;
};

// Unsigned key of the same order as the float; NaN lowest, -0 equal to +0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// Inclusive prefix sums of x over the block (every thread calls); *total gets the block's sum.
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the previous call's readers are done
  if (lane == 31) warp_sums[w] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) {
    const int y = warp_sums[i];
    if (i < w) before += y;
    all += y;
  }
  *total = all;
  return x + before;
}

// STAGED: the CTA's keys fit its dynamic shared memory; otherwise they are read again per pass.
template <bool STAGED>
__global__ void __launch_bounds__(NT) select_kernel(Params p, Evict e) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(16) int hist[BINS];
  __shared__ int warp_sums[NT / 32];
  __shared__ int2 warp_counts[NT / 32], totals;  // positions above T, equal to T
  __shared__ int found_bin, found_above;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = cluster.num_blocks(), rank = cluster.block_rank();
  auto sync = [&]() {
    if (C == 1) __syncthreads();
    else cluster.sync();
  };
  const int pair = blockIdx.x / C, b = pair / p.Hkv, hk = pair % p.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cap = p.max_pages << p.page_shift;
  const int raw = p.lens[b], n = raw < 0 || raw > cap ? 0 : raw;  // impossible: nothing is kept
  if (raw != n && tid == 0) atomicOr(p.status, kStatusBadIndex);
  const int m = min(n, e.budget);
  // this CTA's positions c0 .. c1-1, and each warp's share of them (multiples of 32 and 128)
  const int share = ((n + C - 1) / C + 127) / 128 * 128;
  const int c0 = min(n, rank * share), c1 = min(n, c0 + share);
  if (hk == 0 && rank == 0 && tid == 0) e.lens[b] = m;

  // Keys of positions j .. j+3 (j a multiple of 4: one page, one 16-byte load).
  auto read4 = [&](int j) -> uint4 {
    const int pg = load_page(p, b, j >> p.page_shift);
    if (pg < 0) return make_uint4(0u, 0u, 0u, 0u);
    const float4 x = *reinterpret_cast<const float4*>(p.mass + ((long long)pg * p.Hkv + hk) * p.page + (j & (p.page - 1)));
    return make_uint4(order_key(x.x), order_key(x.y), order_key(x.z), order_key(x.w));
  };
  // candidates: positions lo .. hi-1; `need` of them are kept
  const bool all = n <= e.budget;
  const int lo = all ? 0 : e.sinks, hi = all ? n : n - e.recent;
  int need = all ? n : m - e.sinks - e.recent;
  if (STAGED && !all) {
#pragma unroll 4
    for (int j = c0 + tid * 4; j < c1; j += NT * 4) *reinterpret_cast<uint4*>(keys + j - c0) = read4(j);
    __syncthreads();
  }
  auto keys4 = [&](int j) { return STAGED ? *reinterpret_cast<const uint4*>(keys + j - c0) : read4(j); };

  uint32_t T = 0xFFFFFFFFu;  // above every key: no candidate is kept
  if (!all && need > 0) {    // uniform over the cluster
    T = 0;
    int shift = 32;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass == 2 ? 10 : 11;
      for (int i = tid; i < BINS; i += NT) hist[i] = 0;
      __syncthreads();
      const int down = shift - bits;
#pragma unroll 2
      for (int j = c0 + tid * 4; j < c1; j += NT * 4) {
        const uint4 k = keys4(j);
        const uint32_t u[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (j + i >= lo && j + i < hi && (pass == 0 || (u[i] >> shift) == (T >> shift)))
            atomicAdd(&hist[(u[i] >> down) & ((1u << bits) - 1u)], 1);
      }
      sync();
      // thread t sums bins 4t' .. 4t'+3 over the cluster, t' = NT-1-t: prefix sums run from the top
      const int top = (NT - 1 - tid) * 4;
      int c[4] = {};
      for (int r = 0; r < C; ++r) {
        const int4 x = *reinterpret_cast<const int4*>((C == 1 ? hist : cluster.map_shared_rank(hist, r)) + top);
        c[0] += x.x; c[1] += x.y; c[2] += x.z; c[3] += x.w;
      }
      int sum;
      const int upto = block_scan(c[0] + c[1] + c[2] + c[3], warp_sums, &sum);
      const int above = upto - (c[0] + c[1] + c[2] + c[3]);
      if (above < need && need <= upto) {  // exactly one thread: the need-th largest is here
        int a = above, bin = 3;
        while (a + c[bin] < need) a += c[bin--];
        found_bin = top + bin;
        found_above = a;
      }
      sync();  // found_* set; every CTA has read the histograms
      T |= (uint32_t)found_bin << down;
      need -= found_above;
      shift = down;
    }
  }
  // Kept: protected positions and candidates above T, and the first `need` candidates equal to T
  // (`all`: every position counts as protected). A warp counts its positions, the block and the
  // cluster add up the counts before it, and the warp numbers its kept positions by ballots.
  const int own = (share / (NT / 32) + 31) / 32 * 32;
  const int w0 = min(c1, c0 + warp * own), w1 = min(c1, w0 + own);
  auto kinds = [&](int j, unsigned& gt, unsigned& eq) {  // of positions j .. j+31, this lane's j + lane
    const int i = j + lane;
    bool g = false, q = false;
    if (i < w1) {
      if (all || i < lo || i >= hi) {
        g = true;
      } else {
        uint32_t u;
        if (STAGED) {
          u = keys[i - c0];
        } else {
          const int pg = load_page(p, b, i >> p.page_shift);
          u = pg < 0 ? 0u : order_key(p.mass[((long long)pg * p.Hkv + hk) * p.page + (i & (p.page - 1))]);
        }
        g = u > T;
        q = u == T && T != 0xFFFFFFFFu;
      }
    }
    gt = __ballot_sync(0xffffffffu, g);
    eq = __ballot_sync(0xffffffffu, q);
  };
  int2 mine_ = make_int2(0, 0);
  for (int j = w0; j < w1; j += 32) {
    unsigned gt, eq;
    kinds(j, gt, eq);
    mine_.x += __popc(gt);
    mine_.y += __popc(eq);
  }
  if (lane == 0) warp_counts[warp] = mine_;
  __syncthreads();
  int2 before = make_int2(0, 0), total = before;
  for (int w = 0; w < NT / 32; ++w) {
    const int2 x = warp_counts[w];
    if (w < warp) before = make_int2(before.x + x.x, before.y + x.y);
    total = make_int2(total.x + x.x, total.y + x.y);
  }
  if (tid == 0) totals = total;
  if (C > 1) {
    cluster.sync();
    for (int r = 0; r < rank; ++r) {
      const int2 x = *cluster.map_shared_rank(&totals, r);
      before = make_int2(before.x + x.x, before.y + x.y);
    }
  }
  let_next();
  const int want = all ? 0 : need;  // positions equal to T to keep
  int* kept = e.kept + (long long)pair * e.budget;
  const unsigned lower = (1u << lane) - 1u;
  for (int j = w0; j < w1; j += 32) {
    unsigned gt, eq;
    kinds(j, gt, eq);
    const int g = before.x + __popc(gt & lower), q = before.y + __popc(eq & lower);
    if (((gt >> lane) & 1u) || (((eq >> lane) & 1u) && q < want)) {
      const int at = g + min(q, want);
      if (at < m) kept[at] = j + lane;
    }
    before = make_int2(before.x + __popc(gt), before.y + __popc(eq));
  }
  for (int i = m + rank * NT + tid; i < e.budget; i += C * NT) kept[i] = -1;
  if (C > 1) cluster.sync();  // `totals` stays readable until every CTA is done
}

// A warp moves 32 kept rows of one (sequence, head): keys of kw and values of vw 16-byte words.
__global__ void __launch_bounds__(256) gather_kernel(Params p, Evict e, int kw, int vw, int blocks) {
  const int lane = threadIdx.x & 31;
  wait_previous();
  const int pair = blockIdx.x / blocks, b = pair / p.Hkv, hk = pair % p.Hkv;
  const int i0 = (blockIdx.x % blocks) * 256 + (threadIdx.x & ~31);
  const int i = i0 + lane;
  const int j = i < e.budget ? e.kept[(long long)pair * e.budget + i] : -1;
  long long src = -1, dst = -1;
  if (j >= 0) {
    const int pg = load_page(p, b, j >> p.page_shift);
    const int slot = i >> p.page_shift;
    const int to = slot < e.max_pages ? __ldg(e.table + (long long)b * e.max_pages + slot) : -1;
    if ((unsigned)to >= (unsigned)e.num_pages) atomicOr(p.status, kStatusBadIndex);
    else if (pg >= 0) {
      src = ((long long)pg * p.Hkv + hk) * p.page + (j & (p.page - 1));
      dst = ((long long)to * p.Hkv + hk) * p.page + (i & (p.page - 1));
      e.mass[dst] = p.mass[src];
    }
  }
  if (!__any_sync(0xffffffffu, src >= 0)) return;
  auto move = [&](const void* from, void* to, int words) {
    const uint4* f = static_cast<const uint4*>(from);
    uint4* t = static_cast<uint4*>(to);
    const int lw = __ffs(words) - 1;  // words is a power of two: head sizes are
    // 32 rows x words, 32 words a step: `words` steps, four loads in flight per lane
    for (int s0 = 0; s0 < words; s0 += 4) {
      uint4 x[4];
      long long at[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int w = (s0 + u) * 32 + lane, row = w >> lw, col = w & (words - 1);
        const long long sr = __shfl_sync(0xffffffffu, src, row & 31), ds = __shfl_sync(0xffffffffu, dst, row & 31);
        at[u] = -1;
        if (s0 + u < words && sr >= 0) {
          x[u] = __ldcs(f + sr * words + col);
          at[u] = ds * words + col;
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (at[u] >= 0) t[at[u]] = x[u];
    }
  };
  move(p.k, e.k, kw);
  move(p.v, e.v, vw);
}

}  // namespace

cudaError_t launch_evict(const Params& p, void* k, void* v, float* mass, const int* table, int* lens,
                         int max_pages, int num_pages, int budget, int sinks, int recent, int* kept,
                         int d, int dv, int dtype, cudaStream_t s) {
  const Evict e{k, v, mass, table, lens, kept, max_pages, num_pages, budget, sinks, recent};
  const long long pairs = (long long)p.B * p.Hkv;
  const long long cap = (long long)p.max_pages << p.page_shift;
  // A cluster per (sequence, head), large enough to give every SM a CTA but no CTA fewer than 4096
  // positions (below that the cluster's barriers cost more than it shares: 11 sequences of 28k, 2 heads,
  // 72 us in all with 3600 a CTA, 65 with 7200).
  int C = 1;
  while (C < 8 && pairs * C < 152 && cap / (2 * C) >= 4096) C *= 2;
  const long long share = ((cap + C - 1) / C + 127) / 128 * 128;
  const bool staged = share * 4 <= 160 * 1024;
  if (pairs * C > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaError_t err = launch(staged ? select_kernel<true> : select_kernel<false>, dim3((unsigned)(pairs * C)), NT,
                           staged ? (size_t)share * 4 : 0, C, false, s, p, e);
  if (err != cudaSuccess) return err;
  const int eb = dtype == LLA_F32 ? 4 : 2;
  const long long most = budget < cap ? budget : cap;
  const int blocks = (int)((most + 255) / 256);
  if (blocks == 0) return cudaSuccess;  // tables without pages: nothing is kept
  if (pairs * blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch(gather_kernel, dim3((unsigned)(pairs * blocks)), 256, 0, 1, true, s, p, e, d * eb / 16, dv * eb / 16,
                blocks);
}

}  // namespace paged
}  // namespace lla
