// Attention over a paged cache for sequences with few rows (new tokens x grouped heads): a decode
// step, or a few speculated tokens. bf16, head sizes up to D = 64 or 128 (smaller ones padded with
// zeros as they are copied to shared memory).
//
// What bounds it: HBM. Each cached key and value is read once for all rows of its key/value head
// and takes part in at most 32 row products per element, an order below the ridge point, so what
// counts is bytes in flight: two steps of 8 KB a warp, 12 warps an SM at D = 128. Measured: 32
// sequences of 4k to 16k, 32 heads over 8 of 128, 230 us for the attention, 6.2 TB/s (91 % of the
// copy bandwidth); Parallax, 8 heads of 64, 2k to 16k, 103 us, 6.3 TB/s; one token of 8 heads at 1000
// positions, 6.3 us, most of it the launch and the chain lengths - page - keys. Why not tcgen05: its M is
// 64 or 128 rows and a decode step has 1 to 16, so the smaller mma.sync (m16n8k16) wastes less, keeps scores, weights and accumulators in
// registers (no tensor-memory round trip between the two products of a 16-key step), and lets
// every warp run by itself.
//
// Layout: a block of 4 warps takes a contiguous share of a (sequence, key/value head)'s keys; its
// warps take 16-key steps in turn, each warp with a ring of STAGES steps of its own (keys and
// values, 16-byte asynchronous copies, chunk c of row r at c ^ (r & 7): ldmatrix without bank
// conflicts) and its own running maximum, so the main loop has no block-wide barrier. The warps'
// results are joined through shared memory. Up to 8 blocks of a pair form a cluster and join
// through distributed shared memory: one launch, no scratch. Where a few long sequences need more
// blocks than that, their partial results go through scratch to join_rows_kernel. Either way the
// order is fixed, so results do not depend on scheduling.
// Weight tracking: the attention leaves its logits in scratch and mass_rows_kernel adds up
// exp(s - lse) once the rows' lse is known. (Done by the attention's own blocks after their join,
// the same pass took 60 us longer at B32 L16384 d128: 128 threads a block waiting for scratch.)
// Trees of drafted tokens (TREE, up to 64 nodes): masks come from the tree, which a warp finds between its lanes, and
// more than 16 rows are several tiles. Measured: 12 nodes at 1000 positions, 8 heads of 64 with a probe, 7.0 us; 32
// nodes at 4000, 32 heads over 8 of 64, 17 us.
// Rows: 16 without a probe. With one, rows 0-7 of the MMA are q and rows 8-15 the same rows' r:
// the accumulator fragment gives a thread s and t of one row, p goes back as row i and p t as row
// i + 8, and O1, O2 come out of one product.
// Rounding: p enters the second product as bf16 (the values are bf16 already; fp32 operands have no
// matrix path at this rate); d1, an fp32 sum of the unrounded weights, goes into lse and divides softmax
// attention's O. With a probe o is the difference of two sums that grow with the mean of t, so both are
// taken with the same weights: the rounded ones in p t, d2 and a second d1, and p t as the sum of two
// bf16 (16 bits), the lower parts by a product of their own. With p and p t rounded each for itself
// the error grew with the mean of t (2e-3 of the output at 0.1, 5e-2 at 25; now 2e-3 at either).
#include "lla_paged_rows.cuh"

namespace lla {
namespace paged {
namespace {

constexpr int NW = 4;

template <int D>
struct Cfg {
  // Fewer stages let a third block (D = 128) or a fourth (D = 64) onto an SM, which is worth more:
  // window of 1024 on 48 sequences, D = 128: 29 us with 3 stages, 22 with 2; 8 heads of 64: 107 us
  // with 4, 99 with 3, 106 with 2.
  static constexpr int stages = D == 128 ? 2 : 3;
  static constexpr int step_bytes = KT * D * 2;            // keys, or values
  static constexpr int warp_bytes = stages * 2 * step_bytes;
  static constexpr int join_bytes = NW * 16 * (D + 4) * 4; // the warps' O, reusing the rings,
  static constexpr int fin = join_bytes;                   // and the block's, [16][D]
  static constexpr int bytes = NW * warp_bytes;
  static_assert(fin + 16 * D * 4 <= bytes, "join regions");
};

// CLUSTER: the blocks of a pair (and tile) are one cluster and join there.
// TREE: the new tokens are a tree's nodes (64 at most), their rows in tiles of a block's, which find the keys again in L2.
template <int D, bool PROBE, bool LOGITS, bool CLUSTER, bool TREE>
__global__ void __launch_bounds__(NW * 32) attend_rows_kernel(Params p) {
  using C = Cfg<D>;
  constexpr int ROWS = PROBE ? 8 : 16, NR = PROBE ? 1 : 2;  // rows; rows per thread
  constexpr int CH = D / 8;                                 // 16-byte chunks per key
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ float4 stats[NW][16];
  __shared__ float4 fin_stats[16];  // the block's sums
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ uint64_t node_bits_s[TREE ? kRowsNodes : 1];
  __shared__ int node_pos_s[TREE ? kRowsNodes : 1];
  // the parts of a pair (and tile) follow one another: clusters are made of neighbours
  const int part = blockIdx.x % p.split, index = blockIdx.x / p.split, pair = TREE ? index / p.row_tiles : index;
  const int b = pair / p.Hkv, hk = pair % p.Hkv;
  let_next();
  // Set up behind the tiled kernel of the same call, this one may run beside its last blocks (they
  // share no output); one thread's wait makes the end of this grid the end of both.
  if (p.beside && blockIdx.x == 0 && threadIdx.x == 0) wait_previous();
  const Seq sq = load_seq<TREE>(p, b);
  if (!mine(p, sq.n)) {
    if (sq.n > 0 && sq.n * p.g > p.max_rows) atomicOr(p.status, kStatusBadIndex);  // beyond max_new
    return;
  }
  const int r0 = TREE ? index % p.row_tiles * ROWS : 0, nrows = TREE ? min(ROWS, sq.n * p.g - r0) : sq.n * p.g;
  if (TREE && nrows <= 0) return;
  const int p0 = sq.first, p1 = TREE ? p0 + (r0 + nrows - 1) / p.g : sq.len - 1;
  const TileRange<KT> range(p, p0, p1);
  const int chunk = (range.count + p.split - 1) / p.split;
  const int i0 = min(range.count, part * chunk), i1 = min(range.count, i0 + chunk);
  const __nv_bfloat16* kg = static_cast<const __nv_bfloat16*>(p.k);
  const __nv_bfloat16* vg = static_cast<const __nv_bfloat16*>(p.v);
  uint8_t* const ring = smem + warp * C::warp_bytes;

  // Pages of this warp's next 32 steps, one per lane: one load's latency for all of them.
  int pages = 0, page_at = 0;
  auto load_pages = [&](int first) {
    const int it = first + lane * NW, j = it < i1 ? range.tile(it) * KT : sq.len;
    pages = j < sq.len ? load_page(p, b, j >> p.page_shift) : -1;
    page_at = 0;
  };
  // Copies step `it` (page pg) into a stage: positions past the sequence's end, and those of a bad
  // page, become zeros.
  auto issue = [&](int it, int pg, int stage) {
    if (it < i1) {
      const int j0 = range.tile(it) * KT;
      const long long slot = ((long long)max(pg, 0) * p.Hkv + hk) * p.page + (j0 & (p.page - 1));
      const int live = pg < 0 ? 0 : sq.len - j0;
      const __nv_bfloat16* ks = kg + slot * p.d;
      const __nv_bfloat16* vs = vg + slot * p.dv;
      uint8_t* dst = ring + stage * 2 * C::step_bytes;
#pragma unroll
      for (int e = lane; e < KT * CH; e += 32) {
        const int row = e / CH, c = e % CH;
        const bool k_in = row < live && c * 8 < p.d, v_in = row < live && c * 8 < p.dv;
        const int off = row * (D * 2) + ((c ^ (row & 7)) * 16);
        cp_async16(dst + off, k_in ? ks + row * p.d + c * 8 : kg, k_in ? 16u : 0u);
        cp_async16(dst + C::step_bytes + off, v_in ? vs + row * p.dv + c * 8 : vg, v_in ? 16u : 0u);
      }
    }
    cp_async_commit();
  };
  int it_next = i0 + warp;
  load_pages(it_next);
  auto advance = [&](int stage) {
    if (page_at == 32) load_pages(it_next);
    issue(it_next, __shfl_sync(0xffffffffu, pages, page_at++), stage);
    it_next += NW;
  };
#pragma unroll
  for (int s = 0; s < C::stages - 1; ++s) advance(s);

  // A operand of the first product: rows of q (and r) of this thread.
  uint32_t a[D / 16][4];
  {
    const int i = lane >> 2, cc = (lane & 3) * 2;
    auto row = [&](const void* base, int r) -> const uint32_t* {
      r += r0;
      return reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(base) +
             ((long long)(sq.t0 + r / p.g) * p.Hq + hk * p.g + r % p.g) * p.d + cc);
    };
    const uint32_t* x = i < nrows ? row(p.q, i) : nullptr;
    const uint32_t* y = PROBE ? (i < nrows ? row(p.r, i) : nullptr)
                              : (i + 8 < nrows ? row(p.q, i + 8) : nullptr);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      const bool in = ks * 16 < p.d;
      a[ks][0] = in && x ? x[ks * 8] : 0u;
      a[ks][2] = in && x ? x[ks * 8 + 4] : 0u;
      a[ks][1] = in && y ? y[ks * 8] : 0u;
      a[ks][3] = in && y ? y[ks * 8 + 4] : 0u;
    }
  }
  int pos[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int r = (lane >> 2) + 8 * i;
    pos[i] = r < nrows ? p0 + r / p.g : p1;  // rows past the end are not written
  }
  if constexpr (TREE) {
    if (warp == 0) small_tree(p, sq, node_bits_s, node_pos_s);
    __syncthreads();
  }
  const float c2 = p.inv_h * kLog2e;
  float m[NR], d1[NR], d2 = 0.f, d1r = 0.f, o[D / 8][4];  // d1r: of the rounded weights (PROBE)
#pragma unroll
  for (int i = 0; i < NR; ++i) { m[i] = -CUDART_INF_F; d1[i] = 0.f; }
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[n][i] = 0.f;

  // ldmatrix row addresses of this lane within a stage (before the swizzle's xor)
  const int mi = lane >> 3, mr = lane & 7;
  const int k_row = (mi >> 1) * 8 + mr, k_c = mi & 1;   // keys: [n-tile][k half]
  const int v_row = (mi & 1) * 8 + mr, v_c = mi >> 1;   // values: [k half][n-tile]
  int stage = 0;
  for (int it = i0 + warp; it < i1; it += NW) {
    cp_async_wait<C::stages - 2>();
    __syncwarp();
    {
      const int fill = stage == 0 ? C::stages - 1 : stage - 1;  // the stage read last time
      advance(fill);
    }
    const uint32_t ks_addr = smem_u32(ring + stage * 2 * C::step_bytes);
    const uint32_t vs_addr = ks_addr + C::step_bytes;
    float s[2][2][4] = {};  // [n-tile][even, odd k-steps]: two chains
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t f[4];
      ldmatrix4(f, ks_addr + k_row * (D * 2) + (((ks * 2 + k_c) ^ (k_row & 7)) * 16));
      mma16816(s[0][ks & 1], a[ks], f[0], f[1]);
      mma16816(s[1][ks & 1], a[ks], f[2], f[3]);
    }
    const int j0 = range.tile(it) * KT + (lane & 3) * 2;
    const bool full = TREE ? tree_all_visible(p, p0, p1, j0 & ~15, (j0 & ~15) + KT)
                           : all_visible(p, p0, p1, j0 & ~15, (j0 & ~15) + KT);
    float x[NR][4], t[4];  // logits q.k of this thread's rows and 4 keys (t: probe scores)
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        x[0][n * 2 + e] = s[n][0][e] + s[n][1][e];
        const float y = s[n][0][2 + e] + s[n][1][2 + e];
        if (PROBE) t[n * 2 + e] = y;
        else x[NR - 1][n * 2 + e] = y;
      }
    if (!full) {
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const int node = TREE ? (r0 + min((lane >> 2) + 8 * i, nrows - 1)) / p.g : 0, at = TREE ? node_pos_s[node] : pos[i];
        const uint64_t bits = TREE ? node_bits_s[node] : 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = j0 + (e >> 1) * 8 + (e & 1);
          const bool see = !TREE ? visible(p, at, j)
                           : j < p0 ? j > at - p.window || j < p.sinks : j - p0 < kRowsNodes && (bits >> (j - p0) & 1u);
          if (!see) x[i][e] = -CUDART_INF_F;
        }
      }
    }
    if (LOGITS) {
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const int r = (lane >> 2) + 8 * i;
        if (r < nrows) {
          float* dst = p.logits + ((long long)pair * p.row_cap + r) * p.keys_cap + it * KT + (lane & 3) * 2;
          *reinterpret_cast<float2*>(dst) = make_float2(x[i][0], x[i][1]);
          *reinterpret_cast<float2*>(dst + 8) = make_float2(x[i][2], x[i][3]);
        }
      }
    }
    uint32_t w[4], low[4] = {};  // weights; with a probe, the lower parts of p t as rows 8-15
    bool grew = false;
    float sc[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      float tm = fmaxf(fmaxf(x[i][0], x[i][1]), fmaxf(x[i][2], x[i][3]));
      tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 1));
      tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 2));
      const float mn = fmaxf(m[i], tm);
      const float ref = mn == -CUDART_INF_F ? 0.f : mn * c2;
      grew |= mn > m[i];
      sc[i] = ex2(fmaf(m[i], c2, -ref));
      m[i] = mn;
      float e4[4], sum = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        e4[e] = ex2(fmaf(x[i][e], c2, -ref));
        sum += e4[e];
      }
      d1[i] = fmaf(d1[i], sc[i], sum);
      w[i] = pack_bf16(e4[0], e4[1]);
      w[i + 2] = pack_bf16(e4[2], e4[3]);
      if (PROBE) {
        const float pr[4] = {bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[2]), bf16_hi(w[2])};
        float z[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = x[0][e] == -CUDART_INF_F ? 0.f : pr[e] * t[e];
        d1r = fmaf(d1r, sc[0], (pr[0] + pr[1]) + (pr[2] + pr[3]));
        d2 = fmaf(d2, sc[0], (z[0] + z[1]) + (z[2] + z[3]));
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          w[e + 1] = pack_bf16(z[e], z[e + 1]);
          low[e + 1] = pack_bf16(z[e] - bf16_lo(w[e + 1]), z[e + 1] - bf16_hi(w[e + 1]));
        }
      }
    }
    if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        o[n][0] *= sc[0];
        o[n][1] *= sc[0];
        o[n][2] *= sc[NR - 1];
        o[n][3] *= sc[NR - 1];
      }
    }
#pragma unroll
    for (int n = 0; n < D / 16; ++n) {
      uint32_t f[4];
      ldmatrix4_t(f, vs_addr + v_row * (D * 2) + (((n * 2 + v_c) ^ (v_row & 7)) * 16));
      mma16816(o[2 * n], w, f[0], f[1]);
      mma16816(o[2 * n + 1], w, f[2], f[3]);
      if (PROBE) {
        mma16816(o[2 * n], low, f[0], f[1]);
        mma16816(o[2 * n + 1], low, f[2], f[3]);
      }
    }
    if (++stage == C::stages) stage = 0;
  }
  cp_async_wait<0>();
  __syncthreads();  // the rings are free

  // Join of the four warps through shared memory: O [warp][16][D + 4] and the sums.
  float* os = reinterpret_cast<float*>(smem);
  constexpr int OP = D + 4;
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    d1[i] += __shfl_xor_sync(0xffffffffu, d1[i], 1);
    d1[i] += __shfl_xor_sync(0xffffffffu, d1[i], 2);
  }
  d2 += __shfl_xor_sync(0xffffffffu, d2, 1);
  d2 += __shfl_xor_sync(0xffffffffu, d2, 2);
  d1r += __shfl_xor_sync(0xffffffffu, d1r, 1);
  d1r += __shfl_xor_sync(0xffffffffu, d1r, 2);
  if ((lane & 3) == 0) {
#pragma unroll
    for (int i = 0; i < NR; ++i) stats[warp][(lane >> 2) + 8 * i] = make_float4(m[i], d1[i], d2, d1r);
  }
#pragma unroll
  for (int n = 0; n < D / 8; ++n) {
    float* dst = os + (warp * 16 + (lane >> 2)) * OP + n * 8 + (lane & 3) * 2;
    *reinterpret_cast<float2*>(dst) = make_float2(o[n][0], o[n][1]);
    *reinterpret_cast<float2*>(dst + 8 * OP) = make_float2(o[n][2], o[n][3]);
  }
  __syncthreads();
  const Rows rows{sq.t0, p0, p1, p.g, hk * p.g, r0};
  auto at = [&](int r) { return ((long long)part * p.B * p.Hkv + pair) * p.row_cap + r0 + r; };
  join_block<__nv_bfloat16, D, PROBE, CLUSTER, NW, ROWS, 16>(p, sq, b, rows, part, nrows, at, D, os, stats,
                                                             reinterpret_cast<float*>(smem + C::fin), fin_stats);
}

// One warp per row of the few-rows launch: joins the splits in order.
template <int D, bool PROBE>
__global__ void __launch_bounds__(128) join_rows_kernel(Params p) {
  constexpr int VC = D / 32;
  const int lane = threadIdx.x & 31;
  const long long id = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int pairs = p.B * p.Hkv;
  wait_previous();  // by every thread: this kernel ends after the attention has
  const int pair = (int)(id / p.row_cap), r = (int)(id % p.row_cap);
  if (pair >= pairs) return;
  const int b = pair / p.Hkv, hk = pair % p.Hkv;
  const Seq sq = load_seq_or_tree(p, b);
  if (!mine(p, sq.n) || r >= sq.n * p.g) return;
  const float c2 = p.inv_h * kLog2e;
  auto at = [&](int s) { return ((long long)s * pairs + pair) * p.row_cap + r; };
  float top = -CUDART_INF_F;
  for (int s = 0; s < p.split; ++s) top = fmaxf(top, p.part_s[at(s)].x);
  const float ref = top == -CUDART_INF_F ? 0.f : top * c2;
  float4 sum = make_float4(top, 0.f, 0.f, 0.f);
  float o1[VC] = {}, o2[VC] = {};
  for (int s = 0; s < p.split; ++s) {
    const float4 st = p.part_s[at(s)];
    const float f = ex2(fmaf(st.x, c2, -ref));
    add_sums<PROBE>(sum, st, f);
    const float* src = p.part_o + at(s) * (PROBE ? 2 : 1) * D + lane * VC;
#pragma unroll
    for (int c = 0; c < VC; ++c) {
      o1[c] = fmaf(src[c], f, o1[c]);
      if (PROBE) o2[c] = fmaf(src[D + c], f, o2[c]);
    }
  }
  write_row<__nv_bfloat16, D, PROBE>(p, sq, b, Rows{sq.t0, sq.first, sq.len - 1, p.g, hk * p.g}, r, sum, o1, o2);
}

// mass += the rows' weights, from the logits that the attention wrote (4 bytes a row and key,
// against 2 d bytes a key to read the keys again and the products) and the finished lse. A thread
// takes four keys, whose loads (a row's four logits are one 16-byte word) are all in flight at once.
__global__ void __launch_bounds__(256) mass_rows_kernel(Params p) {
  __shared__ float lse[16];
  wait_previous();
  const int pair = blockIdx.x, b = pair / p.Hkv, hk = pair % p.Hkv;
  const Seq sq = load_seq(p, b);
  if (!mine(p, sq.n)) return;
  const TileRange<KT> range(p, sq.first, sq.len - 1);
  const int nrows = sq.n * p.g, count = range.count * KT;
  if (blockIdx.y * 1024 >= count) return;
  if (threadIdx.x < nrows) {
    const int r = threadIdx.x;
    lse[r] = p.lse[(long long)(sq.t0 + r / p.g) * p.Hq + hk * p.g + r % p.g] * kLog2e;
  }
  __syncthreads();
  const float c2 = p.inv_h * kLog2e;
  for (int i = (blockIdx.y * 256 + threadIdx.x) * 4; i < count; i += gridDim.y * 1024) {
    const int j = range.tile(i / KT) * KT + i % KT;
    if (j >= sq.len) continue;
    const int pg = load_page(p, b, j >> p.page_shift);
    if (pg < 0) continue;
    float4* dst = reinterpret_cast<float4*>(p.mass + ((long long)pg * p.Hkv + hk) * p.page + (j & (p.page - 1)));
    const float4 old = *dst;
    float got[4] = {};
    const float* src = p.logits + (long long)pair * p.row_cap * p.keys_cap + i;
#pragma unroll 4
    for (int r = 0; r < nrows; ++r) {
      const float4 x = *reinterpret_cast<const float4*>(src + (long long)r * p.keys_cap);
      const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (y[e] != -CUDART_INF_F) got[e] += ex2(fmaf(y[e], c2, -lse[r]));  // -inf: not visible
    }
    *dst = make_float4(old.x + got[0], old.y + got[1], old.z + got[2], old.w + got[3]);
  }
}

template <int D, bool PROBE, bool LOGITS, bool TREE = false>
cudaError_t launch_rows_t(Params p, cudaStream_t s) {
  const unsigned pairs = (unsigned)p.B * p.Hkv;
  p.row_tiles = TREE ? (p.row_cap + rows_limit(PROBE) - 1) / rows_limit(PROBE) : 1;
  const long long blocks = (long long)pairs * p.row_tiles * p.split;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const bool cluster = p.split > 1 && p.split <= kRowsCluster;
  auto kern = cluster ? attend_rows_kernel<D, PROBE, LOGITS, true, TREE> : attend_rows_kernel<D, PROBE, LOGITS, false, TREE>;
  cudaError_t err = launch(kern, dim3((unsigned)blocks), NW * 32, Cfg<D>::bytes, cluster ? p.split : 1, p.beside != 0, s, p);
  if (err == cudaSuccess && !cluster && p.split > 1) {
    const long long rows = (long long)pairs * p.row_cap;
    err = launch(join_rows_kernel<D, PROBE>, dim3((unsigned)((rows + 3) / 4)), 128, 0, 1, true, s, p);
  }
  if (err == cudaSuccess && LOGITS) {
    const int blocks = (p.keys_cap + 1023) / 1024;
    err = launch(mass_rows_kernel, dim3(pairs, blocks < 4096 ? blocks : 4096), 256, 0, 1, true, s, p);
  }
  return err;
}

template <int D>
cudaError_t pick(const Params& p, cudaStream_t s) {
  if (p.parents) return p.r ? launch_rows_t<D, true, false, true>(p, s) : launch_rows_t<D, false, false, true>(p, s);
  if (p.r) return p.logits ? launch_rows_t<D, true, true>(p, s) : launch_rows_t<D, true, false>(p, s);
  return p.logits ? launch_rows_t<D, false, true>(p, s) : launch_rows_t<D, false, false>(p, s);
}

}  // namespace

cudaError_t launch_attend_rows(const Params& p, int D, cudaStream_t s) {
  return D == 128 ? pick<128>(p, s) : pick<64>(p, s);
}

}  // namespace paged
}  // namespace lla
