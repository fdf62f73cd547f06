// Attention over a paged cache for sequences with many rows (prompts and chunks), bf16, head sizes up
// to D = 64 or 128 (smaller ones padded with zeros: the tensor maps fill them in), on the tensor
// cores (tcgen05, tensor memory, TMA).
//
// One pass over the keys. Per tile of KT keys and block of 128 rows (tokens x grouped heads of one
// key/value head): S = Q K^T, P = exp(S - m), O += P V; with a probe also T = R K^T, P2 = P .* T,
// O2 += P2 V. "Operand" below: Q of a block, or R.
//   D = 128: one CTA per SM with two operands (512 tensor-memory columns: two S, two O; with a probe S and
//     T, O and O2). Softmax attention takes two row blocks, whose softmax and matrix products alternate: while one
//     block's weights are computed the tensor core works for the other, and both read one key tile.
//   D = 64: two CTAs per SM of 256 columns each, which alternate by themselves: one row block with
//     128-key tiles, or with a probe Q and R with 64-key tiles.
// Warps: softmax (a thread is a row and KT / NG of a tile's keys, NG groups of four warps to a row
// block), then a TMA loader (one lane per page fragment; rows past the sequence's end and bad pages
// are loaded as zeros by an out-of-range coordinate) and one MMA issuer. Its code is warp-uniform
// with only the instructions under elect_one(): issued from a branch on the lane index, an MMA took
// 75 cycles of operand moves against 64 of tensor pipe, and that was the bound (chunk of 2048 at
// 32768, D = 128: 1.06 -> 0.85 ms). One issuer serves both blocks in turn; with an issuer each, their
// products interleave, finish together and the two softmax phases run in step instead of alternating.
// bf16 P overwrites its S (P2 its T, its lower part S behind P), and the next score product is issued behind
// the value product that reads P (MMAs run in order). (At D = 64 there is room for P beside S; using it measured 108 against 106
// us on softmax prompts B4 T4096, 8 heads.)
// The accumulators are rescaled only when a row's maximum outgrows its reference by more than 2^8;
// after the first tiles this hardly happens.
// Rounding: p enters the value product as bf16; d1, the sum of the unrounded fp32 weights, goes into lse
// and divides softmax attention's O. With a probe o is the difference of two sums that grow with the mean
// of t, so both are taken with the same weights, the rounded ones (in p t, d2 and a second d1), and p t as
// the sum of two bf16 (16 bits): P2 is a high and a low part, each with a value product. With p and p t
// rounded each for itself the error grew with the mean of t (2e-3 of the output at 0.1, 5e-2 at 25).
// What bounds it: at D = 128 the chain softmax - value product - next scores of a block, about 3,100
// cycles a 128-key step against 2,048 of MMA for the two blocks (chunk of 2048 at 32768, 32 heads
// over 8: 1.4 PFLOP/s in a row of calls); at D = 64 the N = 64 products (about 59 cycles for 32 of work) and
// the same chain, which is longer with a probe (prompts B4 T4096, 8 heads of 64: 99 us, with a probe 186); at
// D = 128 with a probe the chain of the one block a CTA has (8 heads of 128: 361 us, tensor pipe 42 % active).
// Trees of drafted tokens (TREE) run here too: a masked step looks a row's nodes up as bits that the launch before
// this one finds. With at most 128 rows to a sequence a CTA takes two key tiles at a time (STREAMS): 19 trees of
// 32 nodes at 10240, 32 heads over 8 of 128: 134 us, 89 % of the copy bandwidth (152 with an empty second row
// block); 16 of 4k to 16k 141 us in three launches, of which the cut tiles' join is the last 13; 256 nodes at 32768, where
// the same chain as a chunk's bounds it, 122 us.
// All mbarrier waits are bounded.
#include <type_traits>

#include "lla_paged.cuh"
#include "lla_tc_ptx.cuh"
#include "lla_tmap.cuh"

namespace lla {
namespace paged {
namespace {

using namespace tc;

constexpr int BM = 128;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kTooFar = 100.f;  // a weight of 2^100: its products and sums may leave fp32

// STREAMS: a CTA has one row block and takes its key tiles two at a time, each with scores, weights and an
// accumulator of its own, which alternate like two row blocks; they are joined at a piece's end. For trees of at
// most 128 rows, which would leave a second row block empty (softmax attention at D = 128).
template <int D, bool PROBE, bool STREAMS>
struct Cfg {
  static_assert(!STREAMS || (D == 128 && !PROBE), "streams");
  static constexpr int kt = D == 64 && PROBE ? 64 : 128;       // keys per tile
  static constexpr int blocks = D == 128 && !PROBE && !STREAMS ? 2 : 1;  // row blocks
  static constexpr int halves = STREAMS ? 2 : blocks;          // row blocks or streams, with softmax warps of their own
  static constexpr int ops = halves * (PROBE ? 2 : 1);         // scores at once: of Q of each half, or of Q and R
  static constexpr int operands = STREAMS ? 1 : ops;           // of these in shared memory
  // Groups of four warps per row block. One, a thread taking a whole row of the tile, where the
  // registers allow it: nothing is exchanged then (chunk of 2048 at 32768, D = 128: 779 us with two,
  // 729 with one; prompts B4 T4096 D = 64: 121 and 108, with a probe 462 and 186, the threads of two short of
  // registers). At D = 128 with a probe a step's weights are a long way for one: two (chunk of 2048 at
  // 8192, 32 heads over 8: 675 us with one, 590 with two).
  static constexpr int groups = D == 128 && PROBE ? 2 : 1;
  static_assert(groups <= 2, "a group's weights are one half of a step's, or all");
  static constexpr int nsoft = halves * groups * 4;            // softmax warps
  static constexpr int ctas = D == 64 ? 2 : 1;                 // per SM
  static constexpr int threads = (nsoft + 2) * 32;
  // tensor memory: S [ops][kt] with P in it, O [ops][D]
  static constexpr uint32_t t_o = ops * kt;
  // Column of key j's weight (j even) within S: each group's weights stay within the columns of its
  // own scores, which it has read.
  static constexpr int nc = kt / groups;
  static constexpr uint32_t p_col(int j) { return j / nc * nc + j % nc / 2; }
  static constexpr uint32_t p_low = nc / 2;  // from there (in S, behind the weights): the lower part of p t
  static constexpr uint32_t cols = D == 64 ? 256 : 512;
  static_assert(t_o + ops * D <= cols, "tensor memory");
  // shared memory: operands [ops][D/64][128 rows][128 B], ring of key and value tiles
  // [D/64][kt rows][128 B], barriers, row exchange [6 buffers][nsoft/4 groups][128], tile counts
  static constexpr int op_bytes = BM * D * 2, tile = kt * D * 2, half = kt * 128;
  static constexpr int stages = STREAMS ? 5 : D == 128 ? 4 : PROBE ? 8 : 5;
  static constexpr int items = STREAMS ? 4 : 2;                // ring stages of a step
  static constexpr int sm_ring = operands * op_bytes;
  static constexpr int sm_bar = sm_ring + stages * tile;
  static constexpr int sm_x = sm_bar + 512;
  static constexpr int sm_tiles = sm_x + 6 * (nsoft / 4) * BM * 4, tiles_bytes = 2048 * 4;
  static constexpr int bytes = sm_tiles + tiles_bytes + 1024;  // 1024: aligning the base
  static_assert(ctas * (bytes + 1024) <= 227 * 1024, "shared memory");
};

struct Barriers {
  uint64_t full[8], empty[8];
  uint64_t sfull[2], pfull[2][2], pvdone[2];
  uint64_t rowx[2][4], opfull, opempty, workfull[2], workempty[2], done;
};
static_assert(sizeof(Barriers) <= 512, "barrier region");

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 32 contiguous bytes: a whole sector in one access where they are aligned to it.
__device__ __forceinline__ void store32(void* dst, const uint32_t (&x)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(x[0]), "r"(x[1]),
                 "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
  } else {
    static_cast<uint4*>(dst)[0] = make_uint4(x[0], x[1], x[2], x[3]);
    static_cast<uint4*>(dst)[1] = make_uint4(x[4], x[5], x[6], x[7]);
  }
}

// ------------------------------------------------------------------------------------ schedule
// The work is a line of steps: sequence after sequence, row tile after row tile, key/value head after
// head, key tile after key tile, and before each row tile kStart steps for what it costs to begin
// and end it. Each CTA takes an equal share of the line, so that neither ragged lengths nor a number
// of tiles just above a multiple of the SMs leaves SMs idle (chunk of 2048 at 32768: 256 tiles on
// 152 SMs). A share may begin or end inside a tile; the pieces of such a tile are joined by
// join_tc_kernel. No piece is shorter than kPiece steps: ends that would cut one off move to the
// tile's edge.
// Cutting has a price (partial results of 128 or 256 rows written and read again, about kCut steps of
// time), so where the tiles are many and their tail is short (prompts: the last tiles of a causal
// prompt are the longest, its first the shortest), each CTA takes whole tiles instead: longest
// first, in rows of one per CTA that run back and forth, which levels out a steady decline.
constexpr int kMaxSeqs = 2048;  // their costs wait in the ring's shared memory (larger batches: CUDA cores)
template <int D, bool PROBE, bool STREAMS>
struct Sched {
  using C = Cfg<D, PROBE, STREAMS>;
  static constexpr int kStart = STREAMS ? 6 : C::kt == 64 ? 4 : 3, kPiece = C::kt == 64 ? 8 : 4;
  static constexpr int kCut = C::kt == 64 || STREAMS ? 18 : 12;
  static constexpr int rows = C::blocks * BM;
};
struct Place {  // step s of a tile; b = number of sequences: the end
  int b, tile, hk, s;
};
// TREE: the positions of a tile's nodes lie between the first node's and p1.
struct Tile {
  int tok0, ntok, p0, p1;
  __device__ __forceinline__ Tile(const Seq& sq, int tile, int tokens, bool tree)
      : tok0(tile * tokens), ntok(min(tokens, sq.n - tok0)), p0(tree ? sq.first : sq.first + tok0),
        p1(sq.first + tok0 + ntok - 1) {}
};
// Steps of sequence b's tiles (one head), kStart included, and the shortest's; all lanes of the warp
// return them.
template <int D, bool PROBE, bool TREE, bool STREAMS>
__device__ __forceinline__ long long seq_cost(const Params& p, int b, int tokens, int* tiles, int* shortest) {
  using S = Sched<D, PROBE, STREAMS>;
  const Seq sq = load_seq<TREE>(p, b);
  long long c = 0;
  int least = 0x7fffffff, nt = 0;
  if (mine(p, sq.n)) {
    nt = (sq.n + tokens - 1) / tokens;
    for (int t = threadIdx.x & 31; t < nt; t += 32) {
      const Tile x(sq, t, tokens, TREE);
      const int n = TileRange<S::C::kt>(p, x.p0, x.p1).count + S::kStart;
      c += n;
      least = min(least, n);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    c += __shfl_xor_sync(0xffffffffu, c, o);
    least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
  }
  *tiles = nt;
  *shortest = least;
  return c;
}
__device__ __forceinline__ long long scan_incl(long long x) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if ((threadIdx.x & 31) >= o) x += y;
  }
  return x;
}
// The place at step u of the line, from the sequences' costs (a whole warp calls and agrees).
template <int D, bool PROBE, bool TREE, bool STREAMS>
__device__ __forceinline__ Place locate(const Params& p, const long long* cost, long long u, int tokens) {
  using S = Sched<D, PROBE, STREAMS>;
  const int lane = threadIdx.x & 31;
  for (int base = 0; base < p.B; base += 32) {
    const long long c = base + lane < p.B ? cost[base + lane] * p.Hkv : 0;
    const long long incl = scan_incl(c);
    const unsigned hit = __ballot_sync(0xffffffffu, u < incl);
    if (!hit) {
      u -= __shfl_sync(0xffffffffu, incl, 31);
      continue;
    }
    const int l = __ffs(hit) - 1, b = base + l;
    u -= __shfl_sync(0xffffffffu, incl - c, l);
    const Seq sq = load_seq<TREE>(p, b);
    const int nt = (sq.n + tokens - 1) / tokens;
    for (int tb = 0; tb < nt; tb += 32) {
      int count = 0;
      long long tc = 0;
      if (tb + lane < nt) {
        const Tile x(sq, tb + lane, tokens, TREE);
        count = TileRange<S::C::kt>(p, x.p0, x.p1).count;
        tc = (long long)(count + S::kStart) * p.Hkv;
      }
      const long long ti = scan_incl(tc);
      const unsigned th = __ballot_sync(0xffffffffu, u < ti);
      if (!th) {
        u -= __shfl_sync(0xffffffffu, ti, 31);
        continue;
      }
      const int tl = __ffs(th) - 1;
      const long long rem = u - __shfl_sync(0xffffffffu, ti - tc, tl);
      const int n = __shfl_sync(0xffffffffu, count, tl);
      int step = max(0, (int)(rem % (n + S::kStart)) - S::kStart);
      if (step < S::kPiece) step = 0;
      else if (n - step < S::kPiece) step = n;
      return {b, tb + tl, (int)(rem / (n + S::kStart)), step};
    }
  }
  return {p.B, 0, 0, 0};
}
// Whole tile x in the order last tiles of the sequences, last but one, .. (heads innermost): its place,
// from the sequences' tile counts (a whole warp calls and agrees; tiles x heads stay below 2^31).
__device__ __forceinline__ Place by_rank(const Params& p, const int* tiles, int most, unsigned x) {
  const int lane = threadIdx.x & 31;
  const unsigned row = x / p.Hkv;
  const int hk = (int)(x - row * p.Hkv);
  auto upto = [&](int r) {  // tiles of rank below r
    unsigned n = 0;
    for (int i = 0; i < p.B; i += 32)
      n += __reduce_add_sync(0xffffffffu, i + lane < p.B ? (unsigned)min(tiles[i + lane], r) : 0u);
    return n;
  };
  int lo = 0, hi = most;  // the rank r with upto(r) <= row < upto(r + 1)
  unsigned below = 0;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    const unsigned n = upto(mid);
    if (n <= row) {
      lo = mid;
      below = n;
    } else {
      hi = mid;
    }
  }
  int k = (int)(row - below);  // the k-th sequence with more than lo tiles
  for (int base = 0; base < p.B; base += 32) {
    const bool mine_ = base + lane < p.B && tiles[base + lane] > lo;
    const unsigned has = __ballot_sync(0xffffffffu, mine_);
    const unsigned it = __ballot_sync(0xffffffffu, mine_ && __popc(has & ((1u << lane) - 1u)) == k);
    if (it) {
      const int b = base + __ffs(it) - 1;
      return {b, tiles[b] - 1 - lo, hk, 0};
    }
    k -= __popc(has);
  }
  return {p.B, 0, 0, 0};
}
// A piece of a CTA's share: steps i0 .. i0 + n - 1 of a tile. The loader works the pieces out and the
// other warps read them from shared memory (two entries), so that a CTA has one view of the lengths
// whatever becomes of them meanwhile; it runs ahead, with the next piece's operands and first keys
// in flight while the softmax warps still write the last one's output.
struct Work {
  int b, tile, hk, i0, n, whole, none;
  int t0, seq_n, len, first;  // of the sequence (Seq)
  int n1, w0;                 // of the tile's key tiles (TileRange)
};
// The first of this launch's sequences from b on (a whole warp calls and agrees).
template <bool TREE>
__device__ __forceinline__ int next_seq(const Params& p, int b) {
  for (; b < p.B; b += 32) {
    const int i = b + (threadIdx.x & 31);
    const unsigned hit = __ballot_sync(0xffffffffu, i < p.B && mine(p, load_seq<TREE>(p, i).n));
    if (hit) return b + __ffs(hit) - 1;
  }
  return p.B;
}

// TREE: the new tokens are nodes of trees, whose bits and depths the launch before this one writes.
template <int D, bool PROBE, bool TREE, bool STREAMS>
__global__ void __launch_bounds__((Cfg<D, PROBE, STREAMS>::threads), (Cfg<D, PROBE, STREAMS>::ctas))
attend_tc_kernel(Params p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                 const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap rmap) {
  using C = Cfg<D, PROBE, STREAMS>;
  constexpr int KT = C::kt;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Barriers& bar = *reinterpret_cast<Barriers*>(smem + C::sm_bar);
  __shared__ uint32_t tmem_base_s;
  __shared__ int abort_flag;
  __shared__ Place bounds[2];
  __shared__ int whole_s;              // whole tiles: the most of a sequence; 0: a stretch of the line
  __shared__ long long whole_tiles_s;  // and how many there are
  int* const tiles_s = reinterpret_cast<int*>(smem + C::sm_tiles);  // [B] tiles of each sequence
  __shared__ Work work_s[2];
  // Of each step, by the loader: its first key, and in the low bits (it is a multiple of 64) whether
  // row blocks 0 and 1 need a mask and whether the sequence ends inside it; with streams of each of a
  // step's tiles, and whether there is none.
  __shared__ int step_s[4 * C::items];
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  let_next();  // the few-rows kernel of the same call, which does not depend on this one
  const int per = BM / p.g, width = per * p.g;  // tokens and rows of a row block
  const int tokens = C::blocks * per;           // tokens of a tile

  if (tid == 0) {
    for (int s = 0; s < C::stages; ++s) { mbar_init(&bar.full[s], 1); mbar_init(&bar.empty[s], 1); }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar.sfull[s], 1);
      mbar_init(&bar.pfull[s][0], C::groups * 4);  // (with two groups the second's rescaling too, see there)
      mbar_init(&bar.pfull[s][1], 4);
      mbar_init(&bar.pvdone[s], 1);
      for (int q = 0; q < 4; ++q) mbar_init(&bar.rowx[s][q], STREAMS ? 2 : C::groups);
      mbar_init(&bar.workfull[s], 1);
      mbar_init(&bar.workempty[s], C::nsoft + 1);
    }
    mbar_init(&bar.opfull, 1);
    mbar_init(&bar.opempty, 1);
    mbar_init(&bar.done, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::nsoft + 1) {
    tmem_alloc(&tmem_base_s, C::cols);
    tmem_relinquish();
  }
  // The operands' rows past `width` are never loaded: zeros.
  for (int e = tid; e < C::operands * (D / 64) * (BM - width) * 8; e += C::threads) {
    const int c = e & 7, row = width + (e >> 3) % (BM - width), half = (e >> 3) / (BM - width);
    *reinterpret_cast<uint4*>(smem + half * 16384 + row * 128 + c * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  if (tid == 0) {
    tma_prefetch_map(&kmap);
    tma_prefetch_map(&vmap);
    tma_prefetch_map(&qmap);
    if (PROBE) tma_prefetch_map(&rmap);
  }
  {  // this CTA's share: a stretch of the line, or whole tiles
    long long* cost = reinterpret_cast<long long*>(smem + C::sm_ring);
    int* shortest = reinterpret_cast<int*>(cost + kMaxSeqs);
    static_assert(kMaxSeqs * 12 <= C::stages * C::tile && kMaxSeqs * 4 <= C::tiles_bytes, "the sequences' costs");
    for (int i = warp; i < p.B; i += C::threads / 32) {
      int nt, least;
      const long long c = seq_cost<D, PROBE, TREE, STREAMS>(p, i, tokens, &nt, &least);
      if (lane == 0) {
        cost[i] = c;
        shortest[i] = least;
        tiles_s[i] = nt;
      }
    }
    __syncthreads();
    if (warp < 2) {
      long long w = 0, nt = 0, longest = 0;
      int least = 0x7fffffff, most = 0;
      for (int i = lane; i < p.B; i += 32) {
        w += cost[i];
        nt += tiles_s[i];
        if (TREE && tiles_s[i] > 0) longest = max(longest, cost[i] / tiles_s[i]);  // (alike but for a few nodes)
        least = min(least, shortest[i]);
        most = max(most, tiles_s[i]);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        w += __shfl_xor_sync(0xffffffffu, w, o);
        nt += __shfl_xor_sync(0xffffffffu, nt, o);
        least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
        most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        if (TREE) longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
      }
      w *= p.Hkv;
      nt *= p.Hkv;
      // Whole tiles: the CTAs that the last row leaves out wait for about the shortest tile.
      const long long rows = (nt + gridDim.x - 1) / gridDim.x;
      // (Trees: a sequence's tiles all see its whole prefix, so few sequences of unlike lengths leave CTAs idle
      // behind the longest. 16 of 4k to 16k, 8 heads of 128, a tile each: 201 us whole, 141 cut.)
      const bool whole = TREE ? (rows * longest - Sched<D, PROBE, STREAMS>::kCut) * gridDim.x <= w
                              : (rows * gridDim.x - nt) * least <= (long long)Sched<D, PROBE, STREAMS>::kCut * gridDim.x;
      if (whole) {
        if (tid == 0) whole_s = most;
        if (lane == 0) bounds[warp] = {p.B, 0, 0, 0};
      } else {
        const long long share = max((w + gridDim.x - 1) / gridDim.x, (long long)(Sched<D, PROBE, STREAMS>::kPiece));
        const Place x = locate<D, PROBE, TREE, STREAMS>(p, cost, (blockIdx.x + warp) * share, tokens);
        if (lane == 0) bounds[warp] = x;
        if (tid == 0) whole_s = 0;
      }
      if (tid == 0) whole_tiles_s = nt;
    }
    if (tid < 2) p.pieces[blockIdx.x * 2 + tid] = make_int4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = __shfl_sync(0xffffffffu, tmem_base_s, 0);
  volatile int* abort_p = &abort_flag;
  int* const status = p.status;
  constexpr int TO = kStatusTimeout;
  auto wait = [&](uint64_t* x, uint32_t par) { return warp_wait(x, par, status, TO, abort_p); };
  // From one lane to all: the compiler then knows the value uniform, which the MMA issuer lives on.
  auto uni = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
  // The k-th piece of work, as the loader published it (nullptr: there is none); whoever took it gives
  // it back (whole warps call).
  auto take = [&](int k) -> const volatile Work* {
    if (!wait(&bar.workfull[k & 1], (k >> 1) & 1)) return nullptr;
    return uni(work_s[k & 1].none) ? nullptr : &work_s[k & 1];
  };
  auto give_back = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar.workempty[k & 1]);
  };


  if (warp == C::nsoft + 1) {
    // ------------------------------------------------------------------ MMA issuer
    const uint64_t xd = smem_desc_sw128(smem_u32(smem), 1024);
    const uint64_t kd = smem_desc_sw128(smem_u32(smem + C::sm_ring), 1024);
    const uint64_t vd = smem_desc_sw128_mn(smem_u32(smem + C::sm_ring), C::half, 1024);
    constexpr uint32_t id_s = idesc_bf16(BM, KT, false, false);
    constexpr uint32_t id_o = idesc_bf16(BM, D, false, true);
    constexpr uint32_t tile16 = C::tile >> 4;
    auto stage = [](int x) { return (uint32_t)(x % C::stages); };
    auto parity = [](int x) { return (uint32_t)((x / C::stages) & 1); };
    int base = 0;  // steps before this piece: stages and phases go on from piece to piece
    // S_o = operand o x K^T for operands o0 .. o0 + count - 1 at step gi; the last of a step frees its
    // stage, the last of a piece its operands
    auto scores = [&](auto o0, auto count, int gi, bool last) {
      const uint32_t st = stage(STREAMS ? 4 * gi + 2 * o0 : 2 * gi);
      const uint64_t k = kd + (uint64_t)(st * tile16);
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int o = o0; o < o0 + count; ++o) {
#pragma unroll
          for (int s = 0; s < D / 16; ++s)
            mma_ss(tbase + o * KT, xd + (uint64_t)((STREAMS ? 0 : o) * (C::op_bytes >> 4) + (s >> 2) * 1024 + (s & 3) * 2),
                   k + (uint64_t)((s >> 2) * (C::half >> 4) + (s & 3) * 2), id_s, s > 0);
          mma_commit(&bar.sfull[o]);
        }
        if (STREAMS || o0 + count == C::ops) mma_commit(&bar.empty[st]);
        if (o0 + count == C::ops && last) mma_commit(&bar.opempty);
      }
      __syncwarp();
    };
    // O_o += P_o V over one half of the step's keys
    auto values = [&](auto o0, auto count, int gi, bool first, auto half) {
      const uint32_t st = stage(STREAMS ? 4 * gi + 2 * o0 + 1 : 2 * gi + 1);
      const uint64_t v = vd + (uint64_t)(st * tile16);
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int o = o0; o < o0 + count; ++o) {
#pragma unroll
          for (int u = 0; u < KT / 32; ++u) {
            const int s = half * (KT / 32) + u;
            mma_ts(tbase + C::t_o + o * D, tbase + o * KT + C::p_col(s * 16),
                   v + (uint64_t)(s * (2048 >> 4)), id_o, (!first || s > 0) ? 1u : 0u);
            if (PROBE && o == 1)
              mma_ts(tbase + C::t_o + o * D, tbase + C::p_col(s * 16) + C::p_low,
                     v + (uint64_t)(s * (2048 >> 4)), id_o, 1u);
          }
          if (half) mma_commit(&bar.pvdone[o]);
        }
        if (half && (STREAMS || o0 + count == C::ops)) mma_commit(&bar.empty[st]);
      }
      __syncwarp();
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using Per = std::integral_constant<int, PROBE ? 2 : 1>;  // operands of a row block
    using All = std::integral_constant<int, C::ops>;
    using Second = std::integral_constant<int, C::halves - 1>;
    bool ok = true;
    int pieces = 0;
    for (int k = 0; ok; ++k) {
      const volatile Work* w = take(k);
      if (!w) break;
      const int n = STREAMS ? (uni(w->n) + 1) / 2 : uni(w->n);
      give_back(k);
      if (n == 0) continue;
      // A row block's value products, half a step's weights at a time (the first product runs while
      // the others are computed), and the next scores behind them.
      auto block = [&](auto h, auto o, int i) {
        const int gi = base + i;
        bool d = wait(&bar.pfull[h][0], gi & 1);
        if (d) values(o, Per{}, gi, i == 0, I0{});
        d = d && wait(&bar.pfull[h][1], gi & 1);
        if (d) values(o, Per{}, gi, i == 0, I1{});
        if (STREAMS && d && i + 1 < n) d = wait(&bar.full[stage(4 * gi + 4 + 2 * h)], parity(4 * gi + 4 + 2 * h));
        if (d && i + 1 < n) scores(o, Per{}, gi + 1, i + 2 == n);
        return d;
      };
      ok = wait(&bar.opfull, pieces++ & 1) && wait(&bar.full[stage(C::items * base)], parity(C::items * base));
      if (STREAMS) {
        if (ok) scores(I0{}, I1{}, base, false);
        ok = ok && wait(&bar.full[stage(4 * base + 2)], parity(4 * base + 2));
        if (ok) scores(Second{}, I1{}, base, n == 1);
      } else if (ok) {
        scores(I0{}, All{}, base, n == 1);
      }
      for (int i = 0; STREAMS && i < n && ok; ++i) {
        const int x = 4 * (base + i);
        ok = wait(&bar.full[stage(x + 1)], parity(x + 1)) && block(I0{}, I0{}, i);
        ok = ok && wait(&bar.full[stage(x + 3)], parity(x + 3)) && block(Second{}, Second{}, i);
      }
      for (int i = 0; !STREAMS && i < n && ok; ++i) {
        const int x = 2 * (base + i);
        if (i + 1 < n) ok = wait(&bar.full[stage(x + 2)], parity(x + 2));
        ok = ok && wait(&bar.full[stage(x + 1)], parity(x + 1));
        ok = ok && block(I0{}, I0{}, i);
        if (C::blocks == 2) ok = ok && block(I1{}, Second{}, i);
      }
      base += n;
    }
    if (!ok) *abort_p = 1;
    if (elect_one()) mma_commit(&bar.done);  // after an abort there may be products in flight
    __syncwarp();
    volatile int never = 0;
    mbar_wait(&bar.done, 0, status, TO, &never);
    __syncwarp();
  } else if (warp == C::nsoft) {
    // ------------------------------------------------------------------ work list, loader
    const int frag = min(p.page, KT), nfrag = KT / frag;
    const int most = whole_s;
    const long long ntiles = whole_tiles_s;
    Place cur = bounds[0];
    const Place end = bounds[1];
    int base = 0, pieces = 0, issued = 0;
    bool ok = true, over = false;
    for (int k = 0; ok; ++k) {
      // the piece at `cur`, which moves past it
      Work w = {};
      w.none = 1;
      if (most > 0) {
        const long long at = (long long)k * gridDim.x + (k & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        const Place t = at < ntiles ? by_rank(p, tiles_s, most, (unsigned)at) : Place{p.B, 0, 0, 0};
        if (t.b < p.B) {
          const Seq sq = load_seq<TREE>(p, t.b);
          const Tile x(sq, t.tile, tokens, TREE);
          const TileRange<KT> range(p, x.p0, x.p1);
          w = {t.b, t.tile, t.hk, 0, range.count, 1, 0, sq.t0, sq.n, sq.len, sq.first, range.n1, range.w0};
        }
      }
      while (most == 0 && !over && cur.b < p.B) {
        const Seq sq = load_seq<TREE>(p, cur.b);
        const Tile x(sq, cur.tile, tokens, TREE);
        const TileRange<KT> range(p, x.p0, x.p1);
        const int count = range.count;
        over = cur.b == end.b && cur.tile == end.tile && cur.hk == end.hk;
        if (over && end.s <= cur.s) break;
        const int n = (over ? end.s : count) - cur.s;
        if (n > 0 || n == count)
          w = {cur.b, cur.tile, cur.hk, cur.s, n, n == count, 0, sq.t0, sq.n, sq.len, sq.first, range.n1, range.w0};
        cur.s = 0;
        if (++cur.hk >= p.Hkv) {
          cur.hk = 0;
          if (++cur.tile >= (sq.n + tokens - 1) / tokens) {
            cur.tile = 0;
            cur.b = next_seq<TREE>(p, cur.b + 1);
          }
        }
        if (!w.none) break;
      }
      if (k >= 2) ok = wait(&bar.workempty[k & 1], ((k >> 1) - 1) & 1);
      if (!ok) break;
      if (lane == 0) {
        work_s[k & 1] = w;
        mbar_arrive(&bar.workfull[k & 1]);
      }
      __syncwarp();
      if (w.none) break;
      if (w.n == 0) continue;
      const Tile x(Seq{w.t0, w.seq_n, w.len, w.first}, w.tile, tokens, TREE);
      // Step i's first key, and this lane's page fragment of it: the page number is read a step ahead.
      auto first_key = [&](int i) {
        const int it = w.i0 + i;
        return (it < w.n1 ? it : w.w0 + it - w.n1) * KT;
      };
      auto page_row = [&](int i) {  // row of the tensor map; out of range: zeros
        const int j = first_key(i) + lane * frag;
        const int pg = i < w.n && lane < nfrag && j < w.len ? load_page(p, w.b, j >> p.page_shift) : -1;
        return pg >= 0 ? pg * p.Hkv + w.hk : p.num_pages * p.Hkv;
      };
      int c2_next = page_row(0);
      if (pieces > 0) ok = wait(&bar.opempty, (pieces - 1) & 1);
      if (!ok) break;
      ++pieces;
      if (lane == 0) {  // boxes of [per tokens][g heads][64 features]
        mbar_arrive_expect_tx(&bar.opfull, C::operands * width * D * 2);
        for (int o = 0; o < C::operands; ++o)
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(smem + o * C::op_bytes + c * 16384, PROBE && o ? &rmap : &qmap, c * 64, w.hk * p.g,
                        w.t0 + w.tile * tokens + (PROBE ? 0 : o * per), &bar.opfull);
      }
      __syncwarp();
      const int tiles = STREAMS ? (w.n + 1) / 2 * 2 : w.n;  // (the last step's second may be none: zeros)
      for (int i = 0; i < tiles && ok; ++i) {
        const int k0 = first_key(i), j = k0 + lane * frag, c2 = c2_next;
        c2_next = page_row(i + 1);
        int info = k0 | (k0 + KT > w.len ? 4 : 0);
#pragma unroll
        for (int h = 0; h < C::blocks; ++h) {
          const int q0 = TREE ? x.p0 : min(x.p0 + h * per, x.p1);
          if (TREE ? !tree_all_visible(p, x.p0, x.p1, k0, k0 + KT)
                   : !all_visible(p, q0, min(q0 + per - 1, x.p1), k0, k0 + KT))
            info |= 1 << h;
        }
        if (STREAMS && i >= w.n) info = 1 | 8;
        for (int kv = 0; kv < 2 && ok; ++kv) {
          const int y = 2 * (C::items / 2 * base + i) + kv, st = y % C::stages;
          if (y >= C::stages) ok = wait(&bar.empty[st], ((y / C::stages) - 1) & 1);
          if (!ok) break;
          if (lane == 0) {
            if (kv == 0) step_s[(C::items / 2 * base + i) % (4 * C::items)] = info;
            mbar_arrive_expect_tx(&bar.full[st], C::tile);
          }
          __syncwarp();
          if (lane < nfrag) {
            uint8_t* dst = smem + C::sm_ring + st * C::tile + lane * frag * 128;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(dst + c * C::half, kv ? &vmap : &kmap, c * 64, j & (p.page - 1), c2, &bar.full[st]);
          }
          issued = y + 1;
        }
      }
      base += STREAMS ? tiles / 2 : w.n;
    }
    // Nothing may land in this CTA's shared memory after it exits (the last copies; after an abort
    // nobody else has waited for them).
    if (lane == 0) {
      volatile int never = 0;
      if (pieces > 0) mbar_wait(&bar.opfull, (pieces - 1) & 1, status, TO, &never);
      for (int x = issued > C::stages ? issued - C::stages : 0; x < issued; ++x)
        mbar_wait(&bar.full[x % C::stages], (x / C::stages) & 1, status, TO, &never);
    }
    __syncwarp();
  } else if (warp < C::nsoft) {
    // ------------------------------------------------------------------ softmax + output
    // A group is four warps, one per tensor-memory lane quarter.
    constexpr int NG = C::groups;                  // groups that share a row block
    constexpr int NC = KT / NG;                    // keys of a tile per thread: 64 or 32
    const int r = (warp & 3) * 32 + lane;
    const int h = (warp >> 2) / NG, sub = (warp >> 2) % NG;  // row block, group within it
    const uint32_t lanes = tbase + ((uint32_t)((warp & 3) * 32) << 16);
    const float c2 = p.inv_h * kLog2e, slack = 8.f / c2;
    const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
    // Exchange among the groups of a row: x[buffer][group][row], buffers 0 to 2 for the maxima of steps in
    // turn, 3 to 5 for a piece's sums; between warps of the same rows.
    float* const xm = reinterpret_cast<float*>(smem + C::sm_x);
    auto slot = [&](int buf, int g) -> float& {
      return STREAMS ? xm[(buf * 2 + g) * BM + r] : xm[((buf * C::blocks + h) * NG + g) * BM + r];
    };
    int xphase = 0;  // phases of rowx used so far
    auto exchange = [&]() {
      if (NG == 1 && !STREAMS) return true;
      __syncwarp();
      const int of = STREAMS ? 0 : h;
      if (lane == 0) mbar_arrive(&bar.rowx[of][warp & 3]);
      return wait(&bar.rowx[of][warp & 3], (xphase++) & 1);
    };
    // The groups that share a piece's output, of a row block or the streams, and this one's place among them.
    constexpr int NS = STREAMS ? 2 : NG;
    const int share = STREAMS ? h : sub;
    const int r_tok = r < width ? (STREAMS ? 0 : h * per) + r / p.g : 1 << 30, r_head = r % p.g;  // this row: token of the tile, grouped head
    int base = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
    const volatile Work* w = take(k);  // read again where it is needed: registers are what is short here
    if (!w) break;
    const int n = STREAMS ? (uni(w->n) + 1) / 2 : uni(w->n);
    auto tile_of = [&]() {
      Seq sq;
      sq.n = w->seq_n;
      sq.first = w->first;
      return Tile(sq, w->tile, tokens, TREE);
    };
    float m = -CUDART_INF_F, d1 = 0.f, d2 = 0.f, d1r = 0.f, before = -CUDART_INF_F;  // d1r: of the rounded weights (PROBE)
    for (int i = 0; i < n; ++i) {
      const int gi = base + i;
      ok = wait(&bar.sfull[h], gi & 1);
      if (PROBE) ok = ok && wait(&bar.sfull[1], gi & 1);
      if (!ok) break;
      tc_fence_after();
      // Probe scores come 16 at a time, the next ones under way while these are used: held all at once
      // beside the scores they left too few registers to overlap anything (prompts B4 T4096, 8 heads of 64:
      // 214 us, 186 so).
      uint32_t s[NC / 32][32], tt[PROBE ? 2 : 1][16];
      unsigned seen[NC / 32];
#pragma unroll
      for (int c = 0; c < NC / 32; ++c) tmem_ld32(lanes + h * KT + sub * NC + c * 32, s[c]);
      tmem_ld_wait();
      if constexpr (PROBE) tmem_ld16(lanes + KT + sub * NC, tt[0]);
      const int info = uni(*(volatile int*)&step_s[(STREAMS ? 2 * gi + h : gi) % (4 * C::items)]);
      const int k0 = info & ~63, kb = k0 + sub * NC;
      const bool masked = (info >> (STREAMS ? 0 : h)) & 1;
      if (masked) {
        const Tile tile = tile_of();
        int pos = r_tok < tile.ntok ? tile.p0 + r_tok : tile.p1;  // rows that do not exist are not written
        int past = pos + 1, token = 0;
        if constexpr (TREE) {
          wait_previous();  // (at once but the first time)
          token = w->t0 + tile.tok0 + min(r_tok, tile.ntok - 1);
          past = w->first;
          pos = past + p.depth[token];
        }
        // column c is visible when c < past and (c > lo or c < first), a node's by its bit: as bits, then a
        // select each (a branch per column made such a tile five times as long as a full one)
        const int hi = past - kb, lo = pos - p.window - kb, first = p.sinks - kb;
        auto below = [](int x) { return x <= 0 ? 0u : x >= 32 ? 0xFFFFFFFFu : (1u << x) - 1u; };
#pragma unroll
        for (int c = 0; c < NC / 32; ++c) {
          seen[c] = below(hi - c * 32) & (~below(lo + 1 - c * 32) | below(first - c * 32));
          if (TREE && hi < (c + 1) * 32) seen[c] |= node_bits(p, token, c * 32 - hi);
          if (STREAMS && info & 8) seen[c] = 0u;
#pragma unroll
          for (int e = 0; e < 32; ++e) s[c][e] = seen[c] & (1u << e) ? s[c][e] : 0xFF800000u;
        }
      }
      auto own_max = [&]() {  // over this thread's keys
        float t4[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
        for (int c = 0; c < NC; c += 2)
          t4[(c >> 1) & 3] = max3(t4[(c >> 1) & 3], __uint_as_float(s[c >> 5][c & 31]), __uint_as_float(s[c >> 5][(c & 31) + 1]));
        return fmaxf(max3(t4[0], t4[1], t4[2]), t4[3]);
      };
      // The reference that weights are taken against. The first step of a piece and masked ones take
      // the row's maximum over all groups. The others do not wait for a maximum: they keep the
      // reference, or raise it to the maximum of two steps ago where that had outgrown it by 2^8, and
      // find their own maximum once their weights are on the way. (Of two steps ago, because it was
      // written before the arrivals that the scores of this step come after.) A weight is then at most
      // 2^(growth over three steps); past 2^100 the row is given up here and taken again by itself.
      // With the exchange in every step and the maximum in front of the weights, 1100 of a step's 3400
      // cycles went there (d = 128).
      const bool exact = i == 0 || masked || __any_sync(0xffffffffu, m == -CUDART_INF_F);
      float tm = -CUDART_INF_F, top = m;
      if (exact) {
        top = tm = own_max();
        if (NG > 1) {
          slot(gi % 3, sub) = tm;
          ok = exchange();
          if (!ok) break;
#pragma unroll
          for (int g = 0; g < NG; ++g) top = fmaxf(top, slot(gi % 3, g));
        }
      } else if (NG == 1) {
        top = before;
      } else if (i > 1) {
#pragma unroll
        for (int g = 0; g < NG; ++g) top = fmaxf(top, slot((gi + 1) % 3, g));
      }
      const bool grow = top > m + slack || (m == -CUDART_INF_F && top > m);  // alike in every group
      if (__any_sync(0xffffffffu, grow)) {
        float sc = 1.f;
        if (grow) {
          const float m_old = m;
          sc = ex2((m - top) * c2);  // 0 from -infinity
          m = top;
          // beyond what the last step's weights could hold: the row is taken again at the end
          d1 = (top - m_old) * c2 > kTooFar && m_old != -CUDART_INF_F ? CUDART_INF_F : d1 * sc;
          d2 *= sc;
          d1r *= sc;
        }
        if (i > 0) {
          // (the products that went into them precede this step's scores in the pipe)
          // the row block's accumulators, an equal part per group
          constexpr int part_cols = (PROBE ? 2 : 1) * D / NG;
          const uint32_t o = lanes + C::t_o + h * D + sub * part_cols;
#pragma unroll
          for (int c = 0; c < part_cols; c += 16) {
            uint32_t x[16];
            tmem_ld16(o + c, x);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * sc);
            tmem_st16(o + c, x);
          }
        }
      }
      if (NG > 1 && sub > 0) {
        // The product with the first half's weights goes into the columns that this group has rescaled
        // as well, so it waits for this arrival besides those of the first group.
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.pfull[h][0]);
      }
      if (info & 4) {
        // the last page's slots past the sequence's end may hold anything: their weight is zero,
        // and so must be the values
        const int len = w->len;
        const int x = STREAMS ? 4 * gi + 2 * h + 1 : 2 * gi + 1, st = x % C::stages;
        ok = wait(&bar.full[st], (x / C::stages) & 1);
        if (!ok) break;
        // every warp zeroes every row: its own arrival below is then enough for the products it lets go
        for (int e = lane; e < (k0 + KT - len) * (D / 8); e += 32) {
          const int row = len - k0 + e / (D / 8), c = e % (D / 8);
          *reinterpret_cast<uint4*>(smem + C::sm_ring + st * C::tile + (c >> 3) * C::half + row * 128 + (c & 7) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      const float ref = m == -CUDART_INF_F ? 0.f : m * c2;
      const uint64_t c22 = pair(c2, c2), ref2 = pair(-ref, -ref), minus = pair(-1.f, -1.f);
      uint64_t sum[2] = {}, sumt = 0, sumr = 0;  // pairs of partial sums
      constexpr int CW = PROBE ? 16 : 32;  // keys at once
#pragma unroll
      for (int c = 0; c < NC; c += CW) {
        uint32_t wp[CW / 2], wt[CW / 2], wl[CW / 2];
        uint32_t(&t)[16] = tt[PROBE ? (c / CW) & 1 : 0];
        if constexpr (PROBE) {
          tmem_ld_wait();
          if (c + CW < NC) tmem_ld16(lanes + KT + sub * NC + c + CW, tt[((c / CW) & 1) ^ 1]);
          if (masked) {
#pragma unroll
            for (int e = 0; e < 16; ++e) t[e] = seen[c >> 5] & (1u << ((c & 31) + e)) ? t[e] : 0u;  // of a slot that may hold anything
          }
        }
#pragma unroll
        for (int e = 0; e < CW; e += 2) {
          const uint32_t(&sc)[32] = s[(c + e) >> 5];
          const int at = (c + e) & 31;
          float y0, y1;
          unpair(fma2(pair(__uint_as_float(sc[at]), __uint_as_float(sc[at + 1])), c22, ref2), y0, y1);
          y0 = ex2(y0);
          y1 = ex2(y1);
          sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], pair(y0, y1));
          wp[e / 2] = pack_bf16(y0, y1);
          if constexpr (PROBE) {
            const uint64_t yr = pair(bf16_lo(wp[e / 2]), bf16_hi(wp[e / 2]));
            sumr = add2(sumr, yr);
            const uint64_t z = mul2(yr, pair(__uint_as_float(t[e]), __uint_as_float(t[e + 1])));
            sumt = add2(sumt, z);
            float z0, z1;
            unpair(z, z0, z1);
            wt[e / 2] = pack_bf16(z0, z1);
            unpair(fma2(pair(bf16_lo(wt[e / 2]), bf16_hi(wt[e / 2])), minus, z), z0, z1);
            wl[e / 2] = pack_bf16(z0, z1);
          }
        }
        if constexpr (PROBE) {
          tmem_st8(lanes + C::p_col(sub * NC) + c / 2, wp);
          tmem_st8(lanes + KT + C::p_col(sub * NC) + c / 2, wt);
          tmem_st8(lanes + C::p_col(sub * NC) + C::p_low + c / 2, wl);
        } else {
          tmem_st16(lanes + h * KT + C::p_col(sub * NC) + c / 2, wp);
        }
        // half of the step's weights are there: with this group's last, or, alone, halfway
        if (c + CW == NC || (NG == 1 && c + CW == NC / 2)) {
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.pfull[h][NG == 1 ? c / (NC / 2) : sub]);
        }
      }
      if (!ok) break;
      float a0, a1;
      unpair(add2(sum[0], sum[1]), a0, a1);
      d1 += a0 + a1;
      unpair(sumt, a0, a1);
      d2 += a0 + a1;
      unpair(sumr, a0, a1);
      d1r += a0 + a1;
      if (!exact) {
        tm = own_max();
        if (NG > 1) slot(gi % 3, sub) = tm;
      }
      before = tm;
      if ((tm - m) * c2 > kTooFar) d1 = CUDART_INF_F;  // weights too large to go on with (see repair_row)
    }

    if (PROBE) tmem_ld_wait();  // after a break: nothing may arrive in a register late
    if (NG > 1 && ok) {  // the groups' sums
      slot(3, sub) = d1;
      slot(4, sub) = d2;
      slot(5, sub) = d1r;
      ok = exchange();
      d1 = d2 = d1r = 0.f;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        d1 += slot(3, g);
        d2 += slot(4, g);
        d1r += slot(5, g);
      }
    }
    [[maybe_unused]] float scale[2] = {};  // of the streams' accumulators
    if constexpr (STREAMS) {  // the streams' sums, taken against the larger reference
      if (ok) {
        slot(3, h) = d1;
        slot(4, h) = m;
        ok = exchange();
        m = fmaxf(slot(4, 0), slot(4, 1));
        d1 = 0.f;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const float x = slot(3, g);
          scale[g] = slot(4, g) == -CUDART_INF_F ? 0.f : ex2((slot(4, g) - m) * c2);
          d1 = isinf(x) || isinf(d1) ? CUDART_INF_F : fmaf(x, scale[g], d1);  // (infinite: see repair_row)
        }
      }
    }
    if (ok && n > 0) {
      ok = wait(&bar.pvdone[h], (base + n - 1) & 1);
      if (PROBE || STREAMS) ok = ok && wait(&bar.pvdone[STREAMS ? h ^ 1 : 1], (base + n - 1) & 1);
      tc_fence_after();
    }
    if (!ok) break;
    base += n;
    const Tile tile = tile_of();
    const int t0 = w->t0, hk = w->hk;
    const bool there = r_tok < tile.ntok, whole = w->whole;
    const float norm = PROBE ? d1r : d1;
    const float inv = norm == 0.f ? 0.f : 1.f / norm, f1 = (1.f + d2 * inv) * inv;
    const long long id = (long long)(t0 + tile.tok0 + r_tok) * p.Hq + hk * p.g + r_head;
    // a piece of a tile: slot 0 when it begins inside the tile, else 1
    const int piece = blockIdx.x * 2 + (w->i0 == 0);
    const long long pid = (long long)piece * Sched<D, PROBE, STREAMS>::rows + (STREAMS ? 0 : h * BM) + r;
    float bad = (d1 + d2) * 0.f;  // NaN when something is not finite
    constexpr int NO = D / NS;  // output columns per thread
#pragma unroll 1
    for (int c0 = share * NO; c0 < (share + 1) * NO; c0 += 32) {
      uint32_t a[32], e[PROBE || STREAMS ? 32 : 1];
      if (n > 0) {
        tmem_ld32(lanes + C::t_o + (STREAMS ? 0 : h * D) + c0, a);
        if constexpr (PROBE || STREAMS) tmem_ld32(lanes + C::t_o + D + c0, e);
        tmem_ld_wait();
        if constexpr (STREAMS) {
#pragma unroll
          for (int u = 0; u < 32; ++u)
            a[u] = __float_as_uint(fmaf(__uint_as_float(a[u]), scale[0], __uint_as_float(e[u]) * scale[1]));
        }
      } else {
#pragma unroll
        for (int u = 0; u < 32; ++u) {
          a[u] = 0u;
          if constexpr (PROBE) e[u] = 0u;
        }
      }
#pragma unroll
      for (int q = 0; q < 32; q += 16) {
        const int c = c0 + q;
        if (!there || c >= p.dv) continue;
        if (!whole) {
          float* dst = p.part_o + pid * (PROBE ? 2 : 1) * D + c;
#pragma unroll
          for (int u = 0; u < 16; u += 8) {
            store32(dst + u, *reinterpret_cast<const uint32_t(*)[8]>(a + q + u), true);
            if constexpr (PROBE) store32(dst + D + u, *reinterpret_cast<const uint32_t(*)[8]>(e + q + u), true);
          }
          continue;
        }
        uint32_t o[8];
#pragma unroll
        for (int u = 0; u < 16; u += 2) {
          float y0 = __uint_as_float(a[q + u]) * (PROBE ? f1 : inv);
          float y1 = __uint_as_float(a[q + u + 1]) * (PROBE ? f1 : inv);
          if constexpr (PROBE) {
            y0 = fmaf(-__uint_as_float(e[q + u]), inv, y0);
            y1 = fmaf(-__uint_as_float(e[q + u + 1]), inv, y1);
          }
          bad += (y0 + y1) * 0.f;
          o[u / 2] = pack_bf16(y0, y1);
        }
        store32(static_cast<__nv_bfloat16*>(p.out) + id * p.dv + c, o, wide);
      }
    }
    tc_fence_before();  // these reads, before the arrivals that let the next piece's products go
    if (there && share == 0) {
      if (!whole) p.part_s[pid] = make_float4(m, d1, d2, d1r);
      else if (p.lse) p.lse[id] = d1 == 0.f ? -CUDART_INF_F : (m * c2 + log2f(d1)) * kLn2;
    }
    if (!whole) {
      if (tid == 0) p.pieces[piece] = make_int4(w->b, w->tile, hk, 1);
      give_back(k);
      if (NS > 1) ok = exchange();  // the sums have been read, and the accumulators
      continue;
    }
    // Rows that are not finite, again by themselves: once every group has written its columns, by the
    // first.
    if (NS > 1) {
      ok = exchange();  // the sums have been read, and the accumulators
      if (!ok) break;
      slot(3, share) = bad;
      ok = exchange();
      bad = 0.f;
#pragma unroll
      for (int g = 0; g < NS; ++g) bad += slot(3, g);
    }
    unsigned again = __ballot_sync(0xffffffffu, ok && there && !(bad == 0.f) && share == 0);
    while (again) {
      const int l = __ffs(again) - 1, row = (warp & 3) * 32 + l, tk = (STREAMS ? 0 : h * per) + row / p.g;
      again &= again - 1;
      const Seq sq{t0, w->seq_n, w->len, w->first};
      repair_row<__nv_bfloat16, KT>(p, sq, w->b, tile.p0, tile.p1, t0 + tile.tok0 + tk, hk * p.g + row % p.g,
                                    __shfl_sync(0xffffffffu, d1, l));
    }
    give_back(k);
    if (NS > 1 && ok) ok = exchange();  // and these
    }
  }

  if (TREE && tid == 0) wait_previous();  // the end of this grid is the end of both, whatever it had to do
  tc_fence_before();
  __syncthreads();
  if (warp == C::nsoft + 1) {
    tc_fence_after();
    tmem_dealloc(tbase, C::cols);
  }
}

// The pieces of a tile that was cut: blocks y join the tile whose first piece CTA y has (slot 1); the
// next CTAs' slots 0 continue it. A thread has COLS columns of a row, so that what a row costs whatever its
// size (its place, the pieces' factors) is paid by few threads, and blocks x apart of a tile go to different SMs. (16 trees
// at 4k to 16k, nearly every tile cut: 14.4 us with a warp to a row, 9.3 so.)
// COLS is 16, or 4 where the tiles are few and each has many pieces: then the pieces' loads in flight count.
// Three blocks an SM, with few loads a thread in flight each: with twice those and one or two blocks, a call without cut
// tiles waited 1.5 us for waves of blocks that find nothing (24 mixed sequences 110.1 us, 109.1 so; chunk of 64 at 32768
// 55.6 and 53.9, of 256 at 16000 with heads of 64 58.1 and 56.7; four blocks, with spills, took 256 nodes at 32768 from 122
// to 125).
template <int D, bool PROBE, bool STREAMS, int COLS>
__global__ void __launch_bounds__(256, 3) join_tc_kernel(Params p) {
  using C = Cfg<D, PROBE, STREAMS>;
  constexpr int ROWS = Sched<D, PROBE, STREAMS>::rows, TR = D / COLS;  // threads of a row
  wait_previous();
  const int lane = threadIdx.x & 31;
  auto piece = [&](int c) { return c < gridDim.y ? p.pieces[c * 2] : make_int4(0, 0, 0, 0); };
  const int4 first = p.pieces[blockIdx.y * 2 + 1];
  int4 next = piece(blockIdx.y + 1 + lane);  // with the first: one latency
  if (!first.w) return;
  int n = 1;
  for (;;) {  // the CTAs that continue it, 32 looked at together
    const unsigned on =
        __ballot_sync(0xffffffffu, next.w && next.x == first.x && next.y == first.y && next.z == first.z);
    if (on != 0xffffffffu) {
      n += __ffs(~on) - 1;
      break;
    }
    n += 32;
    next = piece(blockIdx.y + n + lane);
  }
  // The pieces' results of this row, the next ones on their way beside the sequence's lengths.
  const int row = blockIdx.x * (256 / TR) + threadIdx.x / TR, col = threadIdx.x % TR * COLS;
  auto at = [&](int i) { return (long long)((blockIdx.y + i) * 2 + (i == 0)) * ROWS + row; };
  constexpr int CH = (COLS == 4 ? 4 : 2) / (PROBE ? 2 : 1);  // pieces at once
  const bool cols = col < p.dv;
  float4 st[CH], o[CH][COLS / 4], e[PROBE ? CH : 1][COLS / 4];
  auto load = [&](int c) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (c + i >= n) break;
      st[i] = p.part_s[at(c + i)];
      if (!cols) continue;
      const float4* src = reinterpret_cast<const float4*>(p.part_o + at(c + i) * (PROBE ? 2 : 1) * D + col);
#pragma unroll
      for (int u = 0; u < COLS / 4; ++u) {
        o[i][u] = src[u];
        if constexpr (PROBE) e[i][u] = src[D / 4 + u];
      }
    }
  };
  load(0);
  float top = -CUDART_INF_F;
  for (int i = threadIdx.x % TR; i < n; i += TR) top = fmaxf(top, p.part_s[at(i)].x);
#pragma unroll
  for (int i = 1; i < TR; i <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
  const int per = BM / p.g, tokens = C::blocks * per, b = first.x, hk = first.z;
  const Seq sq = load_seq(p, b);
  const Tile tile(sq, first.y, tokens, p.parents != nullptr);
  const float c2 = p.inv_h * kLog2e;
  const int r = row % BM, t = row / BM * per + r / p.g;
  const bool there = r < per * p.g && t < tile.ntok;  // the other rows hold anything
  float s1 = 0.f, s2 = 0.f, s1r = 0.f, bad = 0.f;
  const int token = sq.t0 + tile.tok0 + t, head = hk * p.g + r % p.g;
  if (there) {
    const float ref = top == -CUDART_INF_F ? 0.f : top * c2;
    float o1[COLS] = {}, o2[PROBE ? COLS : 1] = {};
    for (int c = 0; c < n; c += CH) {
      if (c) load(c);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        if (c + i >= n) break;
        const float f = ex2(fmaf(st[i].x, c2, -ref));
        s1 = isinf(st[i].y) ? st[i].y : fmaf(st[i].y, f, s1);  // (infinite: see repair_row; times f it might be NaN)
        s2 = fmaf(st[i].z, f, s2);
        s1r = fmaf(st[i].w, f, s1r);
        if (!cols) continue;
#pragma unroll
        for (int u = 0; u < COLS; u += 4) {
          const float4 x = o[i][u / 4];
          o1[u] = fmaf(x.x, f, o1[u]);
          o1[u + 1] = fmaf(x.y, f, o1[u + 1]);
          o1[u + 2] = fmaf(x.z, f, o1[u + 2]);
          o1[u + 3] = fmaf(x.w, f, o1[u + 3]);
          if constexpr (PROBE) {
            const float4 y = e[i][u / 4];
            o2[u] = fmaf(y.x, f, o2[u]);
            o2[u + 1] = fmaf(y.y, f, o2[u + 1]);
            o2[u + 2] = fmaf(y.z, f, o2[u + 2]);
            o2[u + 3] = fmaf(y.w, f, o2[u + 3]);
          }
        }
      }
    }
    const float norm = PROBE ? s1r : s1;
    const float inv = norm == 0.f ? 0.f : 1.f / norm, f1 = (1.f + s2 * inv) * inv;
    bad = (s1 + s2) * 0.f;
    uint32_t w[COLS / 2];
#pragma unroll
    for (int c = 0; c < COLS; c += 2) {
      const float y0 = PROBE ? fmaf(o1[c], f1, -o2[PROBE ? c : 0] * inv) : o1[c] * inv;
      const float y1 = PROBE ? fmaf(o1[c + 1], f1, -o2[PROBE ? c + 1 : 0] * inv) : o1[c + 1] * inv;
      bad += (y0 + y1) * 0.f;
      w[c / 2] = pack_bf16(y0, y1);
    }
    if (cols) {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + ((long long)token * p.Hq + head) * p.dv + col;
      if constexpr (COLS == 4) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
      } else {
#pragma unroll
        for (int u = 0; u < COLS / 2; u += 4)
          reinterpret_cast<uint4*>(dst)[u / 4] = make_uint4(w[u], w[u + 1], w[u + 2], w[u + 3]);
      }
    }
    if (p.lse && col == 0)
      p.lse[(long long)token * p.Hq + head] = s1 == 0.f ? -CUDART_INF_F : (top * c2 + log2f(s1)) * kLn2;
  }
  // Rows that are not finite, again by themselves, once the warp has written all of their columns.
  unsigned again = __ballot_sync(0xffffffffu, there && !(bad == 0.f));
  while (again) {
    const int l = (__ffs(again) - 1) / TR * TR;  // a row's first lane
    again &= ~((TR == 32 ? 0xffffffffu : (1u << (TR & 31)) - 1u) << l);
    repair_row<__nv_bfloat16, C::kt>(p, sq, b, tile.p0, tile.p1, __shfl_sync(0xffffffffu, token, l),
                                     __shfl_sync(0xffffffffu, head, l), __shfl_sync(0xffffffffu, s1, l));
  }
}

template <int D, bool PROBE, bool TREE, bool STREAMS = false>
cudaError_t launch_tc_t(const Params& p, cudaStream_t s) {
  using C = Cfg<D, PROBE, STREAMS>;
  CUtensorMap kmap, vmap, qmap, rmap;
  cudaError_t err = encode_page_map(p, p.k, p.d, C::kt, &kmap);
  if (err == cudaSuccess) err = encode_page_map(p, p.v, p.dv, C::kt, &vmap);
  if (err == cudaSuccess) err = encode_query_map(p, p.q, &qmap);
  if (err == cudaSuccess) err = encode_query_map(p, PROBE ? p.r : p.q, &rmap);
  if (err != cudaSuccess) return err;
  return launch(attend_tc_kernel<D, PROBE, TREE, STREAMS>, dim3((unsigned)p.split), C::threads, C::bytes, 1, TREE, s, p, kmap,
                vmap, qmap, rmap);
}

template <int D, bool PROBE, bool STREAMS = false>
TcPlan plan_t(long long tokens, int B, int Hkv, int g, long long keys) {
  using C = Cfg<D, PROBE, STREAMS>;
  using S = Sched<D, PROBE, STREAMS>;
  // No more CTAs than pieces there can be.
  const long long tiles = (tokens / (BM / g * C::blocks) + B) * Hkv;
  const long long steps = (keys + C::kt - 1) / C::kt + 3;  // first tokens and window may begin and end inside tiles
  const long long most = tiles * ((steps + S::kPiece - 1) / S::kPiece);
  TcPlan t;
  t.ctas = (int)(most < 152 * C::ctas ? most : 152 * C::ctas);
  t.rows = (size_t)t.ctas * 2 * S::rows;
  t.row_floats = (PROBE ? 2 : 1) * D;
  t.cuts = steps >= 2 * S::kPiece;  // (see locate: both sides of a cut have kPiece steps)
  return t;
}

}  // namespace

// Tensor map of the pages ([num_pages * Hkv][page][d] bf16; boxes of one page fragment, at most
// kt rows, x 64 features, 128-byte swizzled; features past d are zeros).
cudaError_t encode_page_map(const Params& p, void* pages, int d, int kt, CUtensorMap* map) {
  auto encode = tensor_map_encoder();
  if (!encode) return cudaErrorNotSupported;
  const cuuint32_t ones[3] = {1, 1, 1};
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)p.page, (cuuint64_t)p.num_pages * p.Hkv};
  const cuuint64_t str[2] = {(cuuint64_t)d * 2, (cuuint64_t)p.page * d * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)(p.page < kt ? p.page : kt), 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, pages, dims, str, box, ones,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

// Tensor map of q or r ([tokens][Hq][d] bf16; boxes of the 128 / g tokens and g heads of a row block,
// 64 features).
cudaError_t encode_query_map(const Params& p, const void* q, CUtensorMap* map) {
  auto encode = tensor_map_encoder();
  if (!encode) return cudaErrorNotSupported;
  const cuuint32_t ones[3] = {1, 1, 1};
  const cuuint64_t dims[3] = {(cuuint64_t)p.d, (cuuint64_t)p.Hq, (cuuint64_t)p.tokens};
  const cuuint64_t str[2] = {(cuuint64_t)p.d * 2, (cuuint64_t)p.Hq * p.d * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)p.g, (cuuint32_t)(128 / p.g)};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, str, box, ones,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

TcPlan plan_tc(int D, bool probe, bool streams, long long tokens, int B, int Hkv, int g, long long keys) {
  if (B > kMaxSeqs || g > BM) return {};
  if (streams) return plan_t<128, false, true>(tokens, B, Hkv, g, keys);
  if (probe) return D == 128 ? plan_t<128, true>(tokens, B, Hkv, g, keys) : plan_t<64, true>(tokens, B, Hkv, g, keys);
  return D == 128 ? plan_t<128, false>(tokens, B, Hkv, g, keys) : plan_t<64, false>(tokens, B, Hkv, g, keys);
}

template <bool TREE>
static cudaError_t pick(const Params& p, int D, cudaStream_t s) {
  if (p.r) return D == 128 ? launch_tc_t<128, true, TREE>(p, s) : launch_tc_t<64, true, TREE>(p, s);
  return D == 128 ? launch_tc_t<128, false, TREE>(p, s) : launch_tc_t<64, false, TREE>(p, s);
}
cudaError_t launch_attend_tc(const Params& p, int D, cudaStream_t s) {
  if (p.streams) return launch_tc_t<128, false, true, true>(p, s);
  return p.parents ? pick<true>(p, D, s) : pick<false>(p, D, s);
}

template <int COLS>
static cudaError_t join(const Params& p, int D, cudaStream_t s) {
  auto kern = p.r ? (D == 128 ? join_tc_kernel<128, true, false, COLS> : join_tc_kernel<64, true, false, COLS>)
                  : (D == 128 ? join_tc_kernel<128, false, false, COLS> : join_tc_kernel<64, false, false, COLS>);
  if (p.streams) kern = join_tc_kernel<128, false, true, COLS>;
  const int rows = p.streams || p.r || D == 64 ? BM : 2 * BM;
  return launch(kern, dim3(rows * (D / COLS) / 256, (unsigned)p.split), 256, 0, 1, true, s, p);
}
cudaError_t launch_join_tc(const Params& p, int D, cudaStream_t s) {
  // Few tiles: fewer than a quarter of the CTAs, so that most have many more pieces than a thread of 16 columns loads
  // at once (32 nodes at 16000, 32 heads over 8 of 64 with a probe, 38 pieces to a tile: 73 us in all with 16
  // columns, 44 with 4; of 128 without: 37 and 31).
  const int tokens = BM / p.g * (D == 128 && !p.r && !p.streams ? 2 : 1);
  const long long tiles = ((long long)p.tokens / tokens + p.B) * p.Hkv;
  return tiles * 4 <= p.split ? join<4>(p, D, s) : join<16>(p, D, s);
}

}  // namespace paged
}  // namespace lla
