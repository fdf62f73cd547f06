// Attention over a paged cache, fp32, head sizes up to D = 64 or 128 (smaller ones padded with zeros as
// they are copied to shared memory). fp32 operands have no matrix path that keeps their bits, so the
// products are packed fp32 FMAs.
//
// A tile is up to 16 rows (new tokens x grouped heads of one key/value head); larger chunks are many
// tiles, which find the keys again in L2. The code is built for RT = 4, 8 and 16 rows and a tile takes
// the least that holds it: the FMAs of rows that are not there cost as much as the others'.
// What bounds it: HBM up to 8 rows, above that the FMAs (a key of 128 + 128 floats is 1 KB, about 46
// cycles of an SM's share of the bandwidth, and 2 cycles of FMA per row, 4 with a probe).
// Shared memory must not come first, so both products are register tiles: in the first a lane has 4
// rows and RG = RT / 4 keys of a step's 32, in the second all RT rows and 4 value columns.
//
// Layout: a block of NW warps takes a contiguous share of a tile's keys; its warps take steps of 32 keys
// in turn, each with two 8 KB chunks of its own (asynchronous 16-byte copies, one chunk in flight
// behind the one in use; a third chunk a warp would leave an SM six warps instead of eight: 10 % slower): a step's keys by 64 features (16-byte piece c of row r at c ^ (r & 7): lanes read rows apart
// without bank conflicts), then its values. Every warp has its own running maximum, so the main loop
// has no block-wide barrier. Warps and clusters join as in the bf16 kernel of few rows, more splits than
// a cluster has through scratch.
// The accumulators are rescaled only when a row's maximum outgrows its reference by more than 2^8:
// sums and weights are fp32 either way, relative to the same reference.
// Measured: 62 single tokens at 12k to 18k, 16 heads each over 2 of 128, with a probe, 0.90 ms (35 TFLOP/s;
// 2.3 ms in the block-wide form of lla_paged_cc.cuh, with tiles of 16 rows); prompts of 7 sequences of
// 3.8k, 4 heads of 128, 0.71 ms (1.13, tiles of 64 rows); 3 sequences of up to 37 new tokens and 2047
// positions, 6 heads over 2, d 64, dv 32, with a probe and weights, 22 us (47) in two launches. Eight warps
// an SM (registers and shared memory) wait for their own instructions' results most of the time.
#include "lla_paged_rows.cuh"

namespace lla {
namespace paged {
namespace {

constexpr int NW = 4;       // two blocks on an SM with every RT
constexpr int STEP = 32;    // keys
constexpr int STAGES = 2;
constexpr int CHUNK = 8192; // bytes

template <int D, int RT, bool PROBE>
struct Cfg {
  static constexpr int kc = D / 64, vc = D / 64;      // chunks of a step's keys, and values
  static constexpr int vkeys = STEP / vc;             // keys of a chunk of values
  static constexpr int qp = D + 4;                    // row pitch of q and r
  static constexpr int pp = RT == 4 ? 4 : RT + 4;     // key pitch of the weights
  static constexpr int branches = PROBE ? 2 : 1;
  static constexpr int q = NW * STAGES * CHUNK;
  static constexpr int w = q + branches * RT * qp * 4;
  static constexpr int bytes = w + NW * branches * STEP * pp * 4;
  static constexpr int fin = NW * branches * kF32Rows * (D + 4) * 4;  // the join's regions reuse all of it
  static_assert(RT < kF32Rows || fin + branches * kF32Rows * D * 4 <= bytes, "join regions");
  static_assert(2 * (bytes + 3 * 1024) <= 227 * 1024, "two blocks");
};

__device__ __forceinline__ void load2(const void* at, uint64_t& a, uint64_t& b) {  // 16 bytes of shared memory
  const ulonglong2 x = *static_cast<const ulonglong2*>(at);
  a = x.x;
  b = x.y;
}

// A tile of nrows <= RT rows over this block's part of its keys: leaves the warps' sums for the join.
template <int D, int RT, bool PROBE>
__device__ __forceinline__ void attend_tile(const Params& p, const Seq& sq, const Rows& rows, int nrows, int b, int hk,
                                            int part, uint8_t* smem, float4 (&stats)[NW][16]) {
  using C = Cfg<D, RT, PROBE>;
  constexpr int RG = RT / 4, KL = 32 / RG;  // row groups; lanes of one
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, p0 = rows.p0, p1 = rows.p1;
  const TileRange<KT> range(p, p0, p1);
  const int chunk = (range.count + p.split - 1) / p.split;
  const int i0 = min(range.count, part * chunk), i1 = min(range.count, i0 + chunk);
  const int steps = (i1 - i0 + 1) / 2;  // two tiles each
  const float* kg = static_cast<const float*>(p.k);
  const float* vg = static_cast<const float*>(p.v);
  uint8_t* const ring = smem + warp * STAGES * CHUNK;
  float* const qs = reinterpret_cast<float*>(smem + C::q);
  float* const ws = reinterpret_cast<float*>(smem + C::w) + warp * C::branches * STEP * C::pp;

  // Pages of this warp's next 16 steps: lane l has tile l & 1 of the (l >> 1)-th.
  int pages = 0, page_at = 0;
  auto load_pages = [&](int st) {
    const int it = i0 + 2 * (st + (lane >> 1) * NW) + (lane & 1);
    const int j = it < i1 ? range.tile(it) * KT : sq.len;
    pages = j < sq.len ? load_page(p, b, j >> p.page_shift) : -1;
    page_at = 0;
  };
  // A step's two tiles: first position, live rows (the others become zeros: positions past the
  // sequence's end or this block's share, bad pages), first slot.
  struct Step {
    int j[2], live[2];
    long long slot[2];
  };
  int st_next = warp;
  load_pages(st_next);
  auto next_step = [&](Step& x) {
    if (page_at == 16) load_pages(st_next);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int pg = __shfl_sync(0xffffffffu, pages, page_at * 2 + t), it = i0 + 2 * st_next + t;
      x.j[t] = it < i1 ? range.tile(it) * KT : 0x7fffffff - KT;  // past the share: no row sees it
      x.live[t] = it < i1 && pg >= 0 ? sq.len - x.j[t] : 0;
      x.slot[t] = ((long long)max(pg, 0) * p.Hkv + hk) * p.page + (x.j[t] & (p.page - 1));
    }
    ++page_at;
    st_next += NW;
  };
  // A tile lies within a page, so the addresses are in range whatever is live; what is not becomes zeros.
  auto issue_keys = [&](const Step& x, int c, int stage) {  // 32 keys x 64 features
    const int piece = lane & 15, row0 = lane >> 4, at = c * 64 + piece * 4;
    const uint32_t size = at < p.d ? 16u : 0u;
    uint8_t* dst = ring + stage * CHUNK + row0 * 256;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const float* src = kg + (x.slot[t] + row0) * p.d + (size ? at : 0);
      const int live = x.live[t] - row0;
#pragma unroll
      for (int i = 0; i < 8; ++i, src += 2 * p.d)
        cp_async16(dst + (t * 16 + 2 * i) * 256 + ((piece ^ row0 ^ (2 * (i & 3))) * 16), src, 2 * i < live ? size : 0u);
    }
    cp_async_commit();
  };
  auto issue_values = [&](const Step& x, int c, int stage) {  // 16 keys x 128 columns, or 32 x 64
    constexpr int LR = D / 4, RI = 32 / LR;                    // lanes of a row, rows at once
    const int row0 = lane / LR, at = lane % LR * 4;
    const uint32_t size = at < p.dv ? 16u : 0u;
    uint8_t* dst = ring + stage * CHUNK + lane * 16;
#pragma unroll
    for (int u = 0; u < 2 / C::vc; ++u) {
      const bool second = C::vc == 2 ? c != 0 : u != 0;
      const float* src = vg + ((second ? x.slot[1] : x.slot[0]) + row0) * p.dv + (size ? at : 0);
      const int live = (second ? x.live[1] : x.live[0]) - row0;
#pragma unroll
      for (int i = 0; i < 16 / RI; ++i, src += RI * p.dv)
        cp_async16(dst + (u * (16 / RI) + i) * 512, src, RI * i < live ? size : 0u);
    }
    cp_async_commit();
  };
  Step cur, nxt;
  next_step(cur);
  issue_keys(cur, 0, 0);

  // q and r: [RT][D], zeros past nrows and past d
  for (int e = threadIdx.x; e < C::branches * RT * (D / 4); e += NW * 32) {
    const int r = e / (D / 4) % RT, c = e % (D / 4) * 4, br = e / (RT * (D / 4));
    const float* src = static_cast<const float*>(br ? p.r : p.q);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < nrows && c < p.d)
      x = *reinterpret_cast<const float4*>(src + ((long long)(rows.t0 + r / rows.width) * p.Hq + rows.h0 + r % rows.width) * p.d + c);
    *reinterpret_cast<float4*>(qs + (br * RT + r) * C::qp + c) = x;
  }
  __syncthreads();

  // Rows i * RG + rg of this lane, keys kl + KL kk of a step. The weights of a key lie as
  // [rg][i], so slot rg * 4 + i of the second product is row i * RG + rg.
  const int rg = lane / KL, kl = lane % KL;
  int pos[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * RG + rg;
    pos[i] = r < nrows ? p0 + r / rows.width : p1;  // rows past the end are not written
  }
  const float c2 = p.inv_h * kLog2e, slack = fminf(8.f / c2, 1e38f);
  float m[4], ref[4], d1[4], d2[4];
  uint64_t o1[RT / 2][4], o2[PROBE ? RT / 2 : 1][4];  // pairs of slots x 4 columns
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -CUDART_INF_F;
    ref[i] = d1[i] = d2[i] = 0.f;
  }
#pragma unroll
  for (int s = 0; s < RT / 2; ++s)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      o1[s][c] = 0;
      if (PROBE) o2[s][c] = 0;
    }

  const bool logits = p.logits && sq.n * p.g <= p.row_cap;
  const TileRange<KT> whole(p, sq.first, sq.len - 1);  // the sequence's: a logit's place is its key's there
  int stage = 0;
  // The next chunk is here; the one after it goes on its way, into the stage read last time.
  auto arrive = [&](bool keys, int c) {
    cp_async_wait<0>();
    __syncwarp();
    const uint8_t* at = ring + stage * CHUNK;
    stage ^= 1;
    if (keys) {
      if (c + 1 < C::kc) issue_keys(cur, c + 1, stage);
      else issue_values(cur, 0, stage);
    } else {
      if (c + 1 < C::vc) issue_values(cur, c + 1, stage);
      else issue_keys(nxt, 0, stage);
    }
    return at;
  };
  for (int st = warp; st < steps; st += NW) {
    next_step(nxt);
    uint64_t s2[4][RG], t2[PROBE ? 4 : 1][RG];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < RG; ++k) {
        s2[i][k] = 0;
        if (PROBE) t2[i][k] = 0;
      }
#pragma unroll 1
    for (int c = 0; c < C::kc; ++c) {
      const uint8_t* ks = arrive(true, c) + kl * 256;
      const float* qr = qs + rg * C::qp + c * 64;
#pragma unroll 4
      for (int f = 0; f < 16; ++f) {
        uint64_t a[RG], e[RG];
#pragma unroll
        for (int k = 0; k < RG; ++k) load2(ks + k * KL * 256 + ((f ^ (kl & 7)) * 16), a[k], e[k]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint64_t x, y;
          load2(qr + i * RG * C::qp + f * 4, x, y);
#pragma unroll
          for (int k = 0; k < RG; ++k) s2[i][k] = fma2(y, e[k], fma2(x, a[k], s2[i][k]));
          if constexpr (PROBE) {
            load2(qr + (RT + i * RG) * C::qp + f * 4, x, y);
#pragma unroll
            for (int k = 0; k < RG; ++k) t2[i][k] = fma2(y, e[k], fma2(x, a[k], t2[i][k]));
          }
        }
      }
    }
    float x[4][RG];
    const bool full = all_visible(p, p0, p1, cur.j[0], cur.j[0] + KT) && all_visible(p, p0, p1, cur.j[1], cur.j[1] + KT);
    bool grew = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float top = -CUDART_INF_F;
#pragma unroll
      for (int k = 0; k < RG; ++k) {
        float lo, hi;
        unpair(s2[i][k], lo, hi);
        x[i][k] = lo + hi;
        const int key = kl + KL * k, j = (key < KT ? cur.j[0] : cur.j[1]) + (key & (KT - 1));
        if (!full && !visible(p, pos[i], j)) x[i][k] = -CUDART_INF_F;
        top = fmaxf(top, x[i][k]);
      }
      grew |= top > m[i] + slack;
    }
    if (logits) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = i * RG + rg, row = (rows.t0 - sq.t0 + r / rows.width) * p.g + rows.h0 - hk * p.g + r % rows.width;
        float* dst = p.logits + (((long long)b * p.Hkv + hk) * p.row_cap + row) * p.keys_cap;
#pragma unroll
        for (int k = 0; k < RG; ++k) {
          const int key = kl + KL * k, t = key / KT, at = cur.j[t] / KT;
          if (r < nrows && i0 + 2 * st + t < i1)
            dst[(at < whole.n1 ? at : whole.n1 + at - whole.w0) * KT + key % KT] = x[i][k];
        }
      }
    }
    if (__any_sync(0xffffffffu, grew)) {
      float sc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float top = x[i][0];
#pragma unroll
        for (int k = 1; k < RG; ++k) top = fmaxf(top, x[i][k]);
#pragma unroll
        for (int o = KL / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float mn = fmaxf(m[i], top);
        ref[i] = mn == -CUDART_INF_F ? 0.f : mn * c2;
        sc[i] = ex2(fmaf(m[i], c2, -ref[i]));  // 0 where nothing was seen before
        m[i] = mn;
        d1[i] *= sc[i];
        d2[i] *= sc[i];
      }
#pragma unroll
      for (int s = 0; s < RT / 2; ++s) {
        const uint64_t f = pair(__shfl_sync(0xffffffffu, sc[s * 2 % 4], s / 2 * KL),
                                __shfl_sync(0xffffffffu, sc[s * 2 % 4 + 1], s / 2 * KL));
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          o1[s][c] = mul2(o1[s][c], f);
          if (PROBE) o2[s][c] = mul2(o2[s][c], f);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < RG; ++k) {
      float w[4], z[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = ex2(fmaf(x[i][k], c2, -ref[i]));
        d1[i] += w[i];
        if constexpr (PROBE) {
          float lo, hi;
          unpair(t2[i][k], lo, hi);
          z[i] = x[i][k] == -CUDART_INF_F ? 0.f : w[i] * (lo + hi);
          d2[i] += z[i];
        }
      }
      float* dst = ws + (kl + KL * k) * C::pp + rg * 4;
      *reinterpret_cast<float4*>(dst) = make_float4(w[0], w[1], w[2], w[3]);
      if constexpr (PROBE) *reinterpret_cast<float4*>(dst + STEP * C::pp) = make_float4(z[0], z[1], z[2], z[3]);
    }
#pragma unroll 1
    for (int c = 0; c < C::vc; ++c) {
      const uint8_t* vs = arrive(false, c);  // (its warp barrier is the weights' too)
#pragma unroll 8
      for (int k = 0; k < 16; ++k) {
        const int key = D == 128 ? k : 2 * k + (lane >> 4);
        const float4 v = *reinterpret_cast<const float4*>(vs + (D == 128 ? k * 512 + lane * 16 : key * 256 + (lane & 15) * 16));
        const uint64_t vv[4] = {pair(v.x, v.x), pair(v.y, v.y), pair(v.z, v.z), pair(v.w, v.w)};
        const float* w = ws + (c * C::vkeys + key) * C::pp;
#pragma unroll
        for (int s = 0; s < RT / 2; s += 2) {
          uint64_t a, e;
          load2(w + s * 2, a, e);
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            o1[s][f] = fma2(a, vv[f], o1[s][f]);
            o1[s + 1][f] = fma2(e, vv[f], o1[s + 1][f]);
          }
          if constexpr (PROBE) {
            load2(w + STEP * C::pp + s * 2, a, e);
#pragma unroll
            for (int f = 0; f < 4; ++f) {
              o2[s][f] = fma2(a, vv[f], o2[s][f]);
              o2[s + 1][f] = fma2(e, vv[f], o2[s + 1][f]);
            }
          }
        }
      }
    }
    cur = nxt;
  }
  cp_async_wait<0>();
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int o = KL / 2; o; o >>= 1) {
      d1[i] += __shfl_xor_sync(0xffffffffu, d1[i], o);
      d2[i] += __shfl_xor_sync(0xffffffffu, d2[i], o);
    }
  if (kl == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) stats[warp][i * RG + rg] = make_float4(m[i], d1[i], d2[i], 0.f);
  }
  __syncthreads();  // the rings, q and the weights have been read
  float* os = reinterpret_cast<float*>(smem);
  constexpr int OROWS = C::branches * kF32Rows;
  auto put = [&](const uint64_t (&o)[4], int s, int base) {  // slots 2 s and 2 s + 1
    float y[2][4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      unpair(o[c], y[0][c], y[1][c]);
      if (D == 64) {  // the half-warps took a key each
        y[0][c] += __shfl_xor_sync(0xffffffffu, y[0][c], 16);
        y[1][c] += __shfl_xor_sync(0xffffffffu, y[1][c], 16);
      }
    }
    if (lane * 4 < D) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int slot = 2 * s + u, row = slot % 4 * RG + slot / 4;
        *reinterpret_cast<float4*>(os + (warp * OROWS + base + row) * (D + 4) + lane * 4) =
            make_float4(y[u][0], y[u][1], y[u][2], y[u][3]);
      }
    }
  };
#pragma unroll
  for (int s = 0; s < RT / 2; ++s) {
    put(o1[s], s, 0);
    if constexpr (PROBE) put(o2[s], s, kF32Rows);
  }
}

template <int D, bool PROBE>
__global__ void __launch_bounds__(NW * 32, 2) attend_f32_kernel(Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ float4 stats[NW][16];
  __shared__ float4 fin_stats[16];
  // The parts of a tile follow one another: clusters are made of neighbours.
  const int index = blockIdx.x / p.split, part = blockIdx.x % p.split, hk = index % p.Hkv;
  const int per = max(1, kF32Rows / p.g), slices = (p.g + kF32Rows - 1) / kF32Rows;  // tokens a tile; tiles a token
  let_next();
  // Sequences of more rows than p.hi (beyond max_new) have no tiles here, since the grid was not sized for
  // them: they are reported.
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < p.B; i += NW * 32) {
      const int n = load_seq(p, i).n;
      if (n > 0 && !mine(p, n)) atomicOr(p.status, kStatusBadIndex);
    }
  int b, tile;
  if (!find_tile(p, per, index / p.Hkv / slices, &b, &tile)) return;
  const Seq sq = load_seq(p, b);
  if (sq.n == 0) return;  // an impossible length (find_tile counts by the starts)
  const int u0 = index / p.Hkv % slices * kF32Rows, tok0 = tile * per, ntok = min(per, sq.n - tok0);
  const int p0 = sq.first + tok0;
  const Rows rows{sq.t0 + tok0, p0, p0 + ntok - 1, min(p.g - u0, kF32Rows), hk * p.g + u0};
  const int nrows = ntok * rows.width;
  if (nrows <= 4) attend_tile<D, 4, PROBE>(p, sq, rows, nrows, b, hk, part, smem, stats);
  else if (nrows <= 8) attend_tile<D, 8, PROBE>(p, sq, rows, nrows, b, hk, part, smem, stats);
  else attend_tile<D, 16, PROBE>(p, sq, rows, nrows, b, hk, part, smem, stats);
  __syncthreads();
  using C = Cfg<D, kF32Rows, PROBE>;
  const float* os = reinterpret_cast<const float*>(smem);
  float* fin = reinterpret_cast<float*>(smem + C::fin);
  auto at = [&](int r) {
    return ((long long)part * p.tokens + rows.t0 + r / rows.width) * p.Hq + rows.h0 + r % rows.width;
  };
  constexpr int OROWS = C::branches * kF32Rows;
  if (p.split > 1 && p.split <= kRowsCluster)
    join_block<float, D, PROBE, true, NW, kF32Rows, OROWS>(p, sq, b, rows, part, nrows, at, p.dv, os, stats, fin, fin_stats);
  else
    join_block<float, D, PROBE, false, NW, kF32Rows, OROWS>(p, sq, b, rows, part, nrows, at, p.dv, os, stats, fin, fin_stats);
}

// mass += the rows' weights, from the logits that the attention wrote and the finished lse, as
// mass_rows_kernel does, for up to kF32MassRows rows. A warp's lane takes four keys; up to eight warps
// share a key's rows, and their sums are added in order.
__global__ void __launch_bounds__(256) mass_f32_kernel(Params p) {
  __shared__ float lse[kF32MassRows];
  __shared__ float4 sums[8][32];
  wait_previous();
  const int pair = blockIdx.x, b = pair / p.Hkv, hk = pair % p.Hkv, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Seq sq = load_seq(p, b);
  if (!mine(p, sq.n)) return;
  const TileRange<KT> range(p, sq.first, sq.len - 1);
  const int nrows = sq.n * p.g, count = range.count * KT;
  const int share = nrows > 4 ? 8 : nrows > 2 ? 4 : nrows, groups = 8 / share, span = groups * 128;
  if (blockIdx.y * span >= count) return;
  for (int r = threadIdx.x; r < nrows; r += 256)
    lse[r] = subtrahend(p.lse[(long long)(sq.t0 + r / p.g) * p.Hq + hk * p.g + r % p.g]) * kLog2e;
  __syncthreads();
  const float c2 = p.inv_h * kLog2e;
  for (int base = blockIdx.y * span; base < count; base += gridDim.y * span) {
    const int i = base + warp / share * 128 + lane * 4;
    const int j = i < count ? range.tile(i / KT) * KT + i % KT : 0x7ffffff0;  // past the end: not visible
    const float* src = p.logits + (long long)pair * p.row_cap * p.keys_cap + min(i, count - 4);
    float got[4] = {};
#pragma unroll 4
    for (int r = warp % share; r < nrows; r += share) {
      const float4 x = *reinterpret_cast<const float4*>(src + (long long)r * p.keys_cap);
      const float y[4] = {x.x, x.y, x.z, x.w};
      const int pos = sq.first + r / p.g;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (visible(p, pos, j + e)) got[e] += ex2(fmaf(y[e], c2, -lse[r]));
    }
    sums[warp][lane] = make_float4(got[0], got[1], got[2], got[3]);
    __syncthreads();
    if (warp % share == 0 && j < sq.len) {
      const int pg = load_page(p, b, j >> p.page_shift);
      if (pg >= 0) {
        float4* dst = reinterpret_cast<float4*>(p.mass + ((long long)pg * p.Hkv + hk) * p.page + (j & (p.page - 1)));
        float4 a = *dst;
        for (int w = 0; w < share; ++w) {
          const float4 x = sums[warp + w][lane];
          a.x += x.x;
          a.y += x.y;
          a.z += x.z;
          a.w += x.w;
        }
        *dst = a;
      }
    }
    __syncthreads();
  }
}

template <int D, bool PROBE>
cudaError_t launch_t(const Params& p, long long tiles, cudaStream_t s) {
  const long long blocks = tiles * p.Hkv * p.split;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const bool cluster = p.split > 1 && p.split <= kRowsCluster;
  return launch(attend_f32_kernel<D, PROBE>, dim3((unsigned)blocks), NW * 32, Cfg<D, kF32Rows, PROBE>::bytes,
                cluster ? p.split : 1, false, s, p);
}

}  // namespace

long long f32_tiles(long long tokens, long long max_new, int B, int g) {
  const long long per = g < kF32Rows ? kF32Rows / g : 1, slices = (g + kF32Rows - 1) / kF32Rows;
  const long long by_tokens = per == 1 ? tokens : tokens / per + B, by_seqs = (max_new + per - 1) / per * B;
  return (by_tokens < by_seqs ? by_tokens : by_seqs) * slices;
}

cudaError_t launch_attend_f32(const Params& p, long long tiles, int D, cudaStream_t s) {
  if (D == 128) return p.r ? launch_t<128, true>(p, tiles, s) : launch_t<128, false>(p, tiles, s);
  return p.r ? launch_t<64, true>(p, tiles, s) : launch_t<64, false>(p, tiles, s);
}
cudaError_t launch_mass_f32(const Params& p, cudaStream_t s) {
  const int blocks = (p.keys_cap + 127) / 128;
  return launch(mass_f32_kernel, dim3((unsigned)p.B * p.Hkv, blocks < 4096 ? blocks : 4096), 256, 0, 1, true, s, p);
}

}  // namespace paged
}  // namespace lla
