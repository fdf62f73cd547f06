// Sharing, growing and releasing the pages of a cache, and moving what is in them.
//
// refs[page] counts the table entries that hold a page; a sequence holds its first ceil(lens / page) entries; a
// page is free when nobody does. Fork, free and grow change tables, lengths and counts alone: a model's layers
// share them, and copy and compact then move each layer's keys and values.
//
// What bounds them: the bookkeeping its launch and the chain lens - table - refs; copy and compact HBM,
// each byte read once and written once. Counts are integers and pages are taken lowest first, in the order of
// sequences, so results do not depend on scheduling.
// Measured, warm caches: fork 1.9, free 1.9, grow 4.6 us for 8 sequences (grow: two passes over the counts with a barrier of
// the cluster between them; 7.5 for 64); 60 pages of 524 KB (keys and values) copied in 4.8 us, within L2; kept paths of 8 in
// 64 drafts of 64, 8 heads of 128, 4.0 us.
#include <cooperative_groups.h>

#include "lla_paged.cuh"

namespace lla {
namespace paged {
namespace {

namespace cg = cooperative_groups;

__device__ __forceinline__ int pages_of(const Params& p, int n) { return (n + p.page - 1) >> p.page_shift; }
// A sequence's length, or -1 (reported) where the table cannot hold it.
__device__ __forceinline__ int load_len(const Params& p, int b) {
  const int n = p.lens[b];
  if (n >= 0 && n <= p.max_pages << p.page_shift) return n;
  atomicOr(p.status, kStatusBadIndex);
  return -1;
}

// ------------------------------------------------------------------------------------ fork
// A block per new sequence.
__global__ void __launch_bounds__(256) fork_kernel(Params p, const int* parents, int* table, int* lens, int max_pages,
                                                   int* refs) {
  const int c = blockIdx.x, from = parents[c];
  int n = 0;
  if (from < -1 || from >= p.B) {
    if (threadIdx.x == 0) atomicOr(p.status, kStatusBadIndex);
  } else if (from >= 0) {
    n = load_len(p, from);
    if (n > max_pages << p.page_shift) {
      if (threadIdx.x == 0) atomicOr(p.status, kStatusBadIndex);
      n = 0;
    }
    n = max(n, 0);
  }
  bool bad = false;
  for (int i = threadIdx.x; i < pages_of(p, n); i += 256) bad |= load_page(p, from, i) < 0;
  if (__syncthreads_or(bad)) n = 0;
  for (int i = threadIdx.x; i < pages_of(p, n); i += 256) {
    const int pg = p.table[(long long)from * p.max_pages + i];
    table[(long long)c * max_pages + i] = pg;
    atomicAdd(refs + pg, 1);
  }
  if (threadIdx.x == 0) lens[c] = n;
}

// ------------------------------------------------------------------------------------ free
// A block per sequence (its threads have read the length before one of them writes it).
__global__ void __launch_bounds__(256) free_kernel(Params p, const int* keep, int* lens, int* refs) {
  const int b = blockIdx.x, n = load_len(p, b);
  if (n < 0) return;
  const int k = keep ? min(n, max(keep[b], 0)) : 0;
  for (int i = pages_of(p, k) + threadIdx.x; i < pages_of(p, n); i += 256) {
    const int pg = load_page(p, b, i);
    if (pg >= 0 && atomicSub(refs + pg, 1) <= 0) {  // nobody held it
      atomicAdd(refs + pg, 1);
      atomicOr(p.status, kStatusBadIndex);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) lens[b] = k;
}

// ------------------------------------------------------------------------------------ grow
// One cluster. Every block finds what the sequences need (a few words each); the pages' counts are shared out
// over the blocks' warps, whose numbers of free pages meet in distributed shared memory; then a warp knows the
// rank of each of its free pages and whose it becomes. The counts are read twice (the second time from L2) and
// no further than they are needed.
constexpr int kGrowBlocks = 8, kGrowThreads = 1024, kGrowWarps = kGrowThreads / 32;

struct Grow {
  int off[kMaxGrow + 1];  // pages that sequences 0 .. b-1 take
  int more[kMaxGrow];     // new positions; 0: b stays as it is; -1: and is left out
  int held[kMaxGrow];     // pages that b has
  int last[kMaxGrow];     // the page that b copies because others hold it too; -1: none
  int sums[kGrowWarps];   // free pages of the warps before
  int free;               // and of this block
  long long need;         // of all sequences; `off` holds where it does not pass what is free
  unsigned long long over;  // table entries that full rows lack
};

template <typename T>
__device__ __forceinline__ T warp_incl(T x) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if ((threadIdx.x & 31) >= o) x += y;
  }
  return x;
}

__global__ void __launch_bounds__(kGrowThreads) grow_kernel(Params p, int* table, int* lens, int* refs, int2* copies,
                                                            int* left) {
  extern __shared__ __align__(16) uint8_t smem[];
  Grow& g = *reinterpret_cast<Grow*>(smem);
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // The pages of this warp: steps of 128, four counts to a lane.
  const long long steps = ((long long)p.num_pages + 127) / 128, warps = kGrowBlocks * kGrowWarps;
  const long long each = (steps + warps - 1) / warps, id = (long long)rank * kGrowWarps + warp;
  const int s0 = (int)min(steps, id * each), s1 = (int)min(steps, (id + 1) * each);
  auto load = [&](int s) {  // pages past the end are not free
    const int at = s * 128 + lane * 4;
    if (at + 3 < p.num_pages) return *reinterpret_cast<const int4*>(refs + at);
    int4 x = make_int4(1, 1, 1, 1);
    if (at < p.num_pages) x.x = refs[at];
    if (at + 1 < p.num_pages) x.y = refs[at + 1];
    if (at + 2 < p.num_pages) x.z = refs[at + 2];
    return x;
  };
  auto zeros = [](const int4& x) { return (x.x == 0) + (x.y == 0) + (x.z == 0) + (x.w == 0); };
  int mine = 0;
#pragma unroll 4
  for (int s = s0; s < s1; ++s) mine += zeros(load(s));

  // What the sequences need: of pages up to the end of their row of the table, and beyond it of entries.
  if (tid == 0) g.over = 0;
  unsigned long long over = 0;
  for (int b = tid; b < p.B; b += kGrowThreads) {
    const int n = load_len(p, b), t0 = p.starts[b], t1 = p.starts[b + 1], cap = p.max_pages << p.page_shift;
    const bool bad = t0 < 0 || t1 < t0 || t1 - t0 > cap;
    if (bad) atomicOr(p.status, kStatusBadIndex);
    int more = n < 0 || bad ? -1 : t1 - t0;
    if (more > cap - n) {
      over += (((long long)n + more + p.page - 1) >> p.page_shift) - p.max_pages;
      more = cap - n;
    }
    int last = -1;
    if (more > 0 && n & (p.page - 1)) last = load_page(p, b, n >> p.page_shift);
    if (last >= 0 && refs[last] <= 1) last = -1;
    g.more[b] = more;
    g.held[b] = pages_of(p, max(n, 0));
    g.last[b] = last;
  }
  __syncthreads();
  if (over) atomicAdd(&g.over, over);
  // Of the sequences that share a last page and grow, the last keeps it if nobody else holds it.
  unsigned keeps = 0;  // bit i: this thread's i-th sequence
  static_assert(kMaxGrow <= 32 * kGrowThreads, "bits");
  for (int b = tid, i = 0; b < p.B; b += kGrowThreads, ++i) {
    const int last = g.last[b];
    if (last < 0) continue;
    int before = 0;
    for (int a = 0; a < b; ++a) before += g.last[a] == last;
    if (refs[last] - before <= 1) keeps |= 1u << i;
  }
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) g.sums[warp] = mine;
  __syncthreads();
  for (int b = tid, i = 0; b < p.B; b += kGrowThreads, ++i)
    if (keeps >> i & 1u) g.last[b] = -1;
  __syncthreads();
  if (warp == 0) {
    // (in 64 bits: starts that go up and down may ask for more than there can be)
    long long before = 0;
    for (int base = 0; base < p.B; base += 32) {
      const int b = base + lane;
      long long x = 0;
      if (b < p.B && g.more[b] > 0)
        x = (g.last[b] >= 0) + pages_of(p, lens[b] + g.more[b]) - g.held[b];
      const long long incl = warp_incl(x);
      if (b < p.B) g.off[b] = (int)(before + incl - x);
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      g.off[p.B] = (int)before;
      g.need = before;
    }
  } else if (warp == 1) {
    const int x = g.sums[lane], incl = warp_incl(x);
    __syncwarp();
    g.sums[lane] = incl - x;
    if (lane == 31) g.free = incl;
  }
  cluster.sync();  // what is written from here on has been read by every block
  int first = g.sums[warp], all = 0;
  for (int i = 0; i < kGrowBlocks; ++i) {
    const int x = *cluster.map_shared_rank(&g.free, i);
    if (i < rank) first += x;
    all += x;
  }
  const bool enough = g.need <= all && g.over == 0;
  const int need = enough ? (int)g.need : 0;
  cluster.sync();  // no block leaves before its sum has been read
  if (rank == 0) {
    if (tid == 0)
      *left = (int)max(enough ? all - g.need : -(max(g.need - all, 0LL) + (long long)g.over), -2147483647LL);
    for (int b = tid; b < p.B; b += kGrowThreads) {
      if (!enough || g.last[b] < 0) copies[b] = enough && g.more[b] < 0 ? make_int2(-2, -2) : make_int2(-1, -1);
      if (!enough) continue;
      if (g.last[b] >= 0) atomicSub(refs + g.last[b], 1);
      if (g.more[b] > 0) lens[b] += g.more[b];
    }
  }
  if (!enough) return;
  for (int s = s0; s < s1 && first < need; ++s) {
    const int4 x = load(s);
    const int count = zeros(x), incl = warp_incl(count), at = s * 128 + lane * 4;
    int k = first + incl - count;  // the rank of the lane's next free page
    const int c[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (c[i] != 0) continue;
      if (k < need) {
        int b = 0, e = p.B;  // whose it becomes: off[b] <= k < off[b + 1]
        while (e - b > 1) {
          const int mid = (b + e) / 2;
          if (g.off[mid] <= k) b = mid;
          else e = mid;
        }
        int nth = k - g.off[b], slot = g.held[b] + nth;
        if (g.last[b] >= 0) {  // the first one takes the shared page's place
          --slot;
          if (nth == 0) copies[b] = make_int2(g.last[b], at + i);
        }
        table[(long long)b * p.max_pages + slot] = at + i;
        refs[at + i] = 1;
      }
      ++k;
    }
    first += __shfl_sync(0xffffffffu, incl, 31);
  }
}

// ------------------------------------------------------------------------------------ copy
// A block moves kCopyBytes of one pair's pages, taken as one stretch: keys, values, mass. Its words are counted in
// 32 bits (copy_fits).
struct Pools {
  const uint4* from[3];
  uint4* to[3];
  int words[3];  // 16-byte words of a page: keys, values, mass
  int from_pages, to_pages, chunks;
};
__global__ void __launch_bounds__(256) copy_kernel(const __grid_constant__ Pools a, const int2* pairs, int* status) {
  const int pair = blockIdx.x / a.chunks, chunk = blockIdx.x % a.chunks;
  const int2 x = pairs[pair];
  if (x.x < 0 || x.y < 0) return;
  if (x.x >= a.from_pages || x.y >= a.to_pages) {
    if (threadIdx.x == 0) atomicOr(status, kStatusBadIndex);
    return;
  }
  constexpr int N = kCopyBytes / 16 / 256;
  uint4 w[N];
  const int first = chunk * (kCopyBytes / 16) + threadIdx.x;
  auto at = [&](int i, int& which) {  // word i of the stretch: which array, and the word of its page (-1: past the end)
    which = 0;
    for (; which < 3 && i >= a.words[which]; ++which) i -= a.words[which];
    return which < 3 ? i : -1;
  };
#pragma unroll
  for (int u = 0; u < N; ++u) {
    int p, i = at(first + u * 256, p);
    if (i >= 0) w[u] = a.from[p][(long long)x.x * a.words[p] + i];
  }
#pragma unroll
  for (int u = 0; u < N; ++u) {
    int p, i = at(first + u * 256, p);
    if (i >= 0) a.to[p][(long long)x.y * a.words[p] + i] = w[u];
  }
}

// ------------------------------------------------------------------------------------ compact
// A block moves the kept nodes of one sequence and key/value head. Destinations come at or before their
// sources and both rise, so rounds in order, each read whole before it is written, lose nothing.
constexpr int kCompactThreads = 256, kCompactWords = 4;  // 16-byte words of a thread in a round
__global__ void __launch_bounds__(kCompactThreads) compact_kernel(Params p, const int* path, int max_path, int* keep, int kw,
                                                                  int vw) {
  const int b = blockIdx.x / p.Hkv, hk = blockIdx.x % p.Hkv, tid = threadIdx.x;
  const Seq sq = load_seq(p, b);
  const int* mine = path + (long long)b * max_path;
  // The path: entries before the first that is negative, rising, below the number of nodes; it moves between pages of
  // the pool.
  int count = max_path;
  for (int i = tid; i < max_path; i += kCompactThreads)
    if (mine[i] < 0) count = min(count, i);
  __shared__ int shared_count;
  if (tid == 0) shared_count = max_path;
  __syncthreads();
  if (count < max_path) atomicMin(&shared_count, count);
  __syncthreads();
  count = shared_count;
  bool bad = sq.first < 0;
  for (int i = tid; i < count; i += kCompactThreads) {
    const int a = mine[i];
    bad |= a >= sq.n || a < i || (i > 0 && a <= mine[i - 1]);  // (what rises from 0 on stays at or above its index)
    if (!bad && a != i)  // both slots are the sequence's: are their pages the pool's
      bad = load_page(p, b, (sq.first + a) >> p.page_shift) < 0 || load_page(p, b, (sq.first + i) >> p.page_shift) < 0;
  }
  bad = __syncthreads_or(bad);
  if (tid == 0 && hk == 0) {
    if (bad) atomicOr(p.status, kStatusBadIndex);
    // load_seq gives a sequence with impossible starts or length no nodes: it stays as it is
    const int t0 = p.starts[b], t1 = p.starts[b + 1], len = p.lens[b];
    const bool sane = t0 >= 0 && t1 >= t0 && t1 <= p.tokens && t1 - t0 <= len;
    keep[b] = sane ? len - (t1 - t0) + (bad ? 0 : count) : len;
  }
  if (bad) return;
  const int words = kw + vw, each = kCompactThreads * kCompactWords / words;  // positions of a round
  for (int i0 = 0; i0 < count; i0 += each) {
    uint4 x[kCompactWords];
    uint4* to[kCompactWords];
    float mass[kCompactWords];
    float* mass_to[kCompactWords];
    const int i1 = min(count, i0 + each);
    auto slot = [&](int j) -> long long {
      const int pg = load_page(p, b, j >> p.page_shift);
      return pg < 0 ? -1 : ((long long)pg * p.Hkv + hk) * p.page + (j & (p.page - 1));
    };
#pragma unroll
    for (int u = 0; u < kCompactWords; ++u) {
      const int e = tid + u * kCompactThreads, i = i0 + e / words, w = e % words;
      to[u] = nullptr;
      mass_to[u] = nullptr;
      if (i >= i1 || mine[i] == i) continue;
      const long long src = slot(sq.first + mine[i]), dst = slot(sq.first + i);
      if (src < 0 || dst < 0) continue;
      const bool key = w < kw;
      uint4* base = static_cast<uint4*>(key ? p.k : p.v);
      const int row = key ? kw : vw, c = key ? w : w - kw;
      x[u] = base[src * row + c];
      to[u] = base + dst * row + c;
      if (w == 0 && p.mass) {
        mass[u] = p.mass[src];
        mass_to[u] = p.mass + dst;
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kCompactWords; ++u) {
      if (to[u]) *to[u] = x[u];
      if (mass_to[u]) *mass_to[u] = mass[u];
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_fork(const Params& p, const int* parents, int* table, int* lens, int num_seqs, int max_pages, int* refs,
                        cudaStream_t s) {
  fork_kernel<<<num_seqs, 256, 0, s>>>(p, parents, table, lens, max_pages, refs);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_free(const Params& p, const int* keep, int* lens, int* refs, cudaStream_t s) {
  free_kernel<<<p.B, 256, 0, s>>>(p, keep, lens, refs);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_grow(const Params& p, int* table, int* lens, int* refs, int* copies, int* left, cudaStream_t s) {
  return launch(grow_kernel, dim3(kGrowBlocks), kGrowThreads, sizeof(Grow), kGrowBlocks, false, s, p, table, lens, refs,
                reinterpret_cast<int2*>(copies), left);
}

bool copy_fits(long long page_bytes, int count) {
  const long long chunks = (page_bytes + kCopyBytes - 1) / kCopyBytes;
  return page_bytes <= (1LL << 35) - kCopyBytes && count * chunks <= 0x7fffffffLL;
}

cudaError_t launch_copy(const Params& from, const Params& to, const int* pairs, int count, int dtype, cudaStream_t s) {
  const int eb = dtype == LLA_F32 ? 4 : 2;
  Pools a = {};
  const void* f[3] = {from.k, from.v, from.mass};
  void* t[3] = {to.k, to.v, to.mass};
  const bool mass = from.mass && to.mass;
  const int bytes[3] = {from.d * eb, from.dv * eb, mass ? 4 : 0};  // of a slot
  long long words = 0;
  for (int i = 0; i < 3; ++i) {
    a.from[i] = static_cast<const uint4*>(f[i]);
    a.to[i] = static_cast<uint4*>(t[i]);
    a.words[i] = (int)((long long)from.Hkv * from.page * bytes[i] / 16);
    words += a.words[i];
  }
  a.from_pages = from.num_pages;
  a.to_pages = to.num_pages;
  a.chunks = (int)((words * 16 + kCopyBytes - 1) / kCopyBytes);
  copy_kernel<<<(unsigned)(count * (long long)a.chunks), 256, 0, s>>>(a, reinterpret_cast<const int2*>(pairs), from.status);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_compact(const Params& p, const int* path, int max_path, int* keep, int dtype, cudaStream_t s) {
  const int eb = dtype == LLA_F32 ? 4 : 2;
  compact_kernel<<<(unsigned)p.B * p.Hkv, kCompactThreads, 0, s>>>(p, path, max_path, keep, p.d * eb / 16, p.dv * eb / 16);
  count_launch();
  return cudaGetLastError();
}

}  // namespace paged
}  // namespace lla
