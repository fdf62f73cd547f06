// Attention over a paged cache for sequences with many rows (prompts and chunks), bf16, head sizes
// up to D = 64 or 128 (smaller ones padded with zeros: the tensor maps fill them in), on the tensor cores (tcgen05, tensor memory, TMA).
//
// One pass over the keys with a running row maximum. Per tile of KT keys and block of 128 rows
// (tokens x grouped heads of one key/value head): S = Q K^T, P = exp(S - m), O += P V; with a probe
// also T = R K^T, P2 = P .* T, O2 += P2 V. "Operand" below: Q of a block, or R.
//   d = 128: one CTA per SM with two operands (512 tensor-memory columns: two S, two O). Softmax
//     attention takes two row blocks, whose softmax and matrix products alternate: while one
//     block's weights are computed the tensor core works for the other, and both read one key tile.
//   d = 64: two CTAs per SM of 256 columns each, which alternate by themselves: one row block with
//     128-key tiles, or with a probe Q and R with 64-key tiles.
// Warps: softmax (a thread is a row and KT / NG of a tile's keys; the NG groups of four warps that
// share a row block pass the row maximum through shared memory), then a TMA loader (one lane per
// page fragment; rows past the sequence's end and bad pages are loaded as zeros by an out-of-range
// coordinate) and one MMA issuer. Its code is warp-uniform with only the instructions under
// elect_one(): issued from a branch on the lane index, an MMA took 75 cycles of operand moves
// against 64 of tensor pipe, and that was the bound (chunk of 2048 at 32768, d = 128: 1.06 -> 0.85
// ms). One issuer serves both blocks in turn; with an issuer each, their products interleave,
// finish together and the two softmax phases run in step instead of alternating.
// bf16 P has columns of its own where there is room (d = 64 without a probe: the next scores are
// issued as soon as these are read), else it overwrites its S and the next score product is issued
// behind the value product that reads P (MMAs run in order).
// The accumulators are rescaled only when a row's maximum grows by more than 2^8 (the weights then
// stay below 2^8, exact in scale; d1 is fp32): after the first tiles this hardly happens.
// Rounding: p and p t enter the value products as bf16, d1 and d2 sum the unrounded fp32 weights.
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

template <int D, bool PROBE>
struct Cfg {
  static constexpr int kt = D == 64 && PROBE ? 64 : 128;       // keys per tile
  static constexpr int blocks = D == 128 && !PROBE ? 2 : 1;    // row blocks
  static constexpr int ops = blocks * (PROBE ? 2 : 1);         // operands: Q of each block, or Q and R
  // groups of four warps per row block (d = 64, prompts of B4 T4096, 8 heads: 127 us with two, 138
  // with one; with a probe 222 with two of 32 keys a thread, 195 with one of 64 and no exchange)
  static constexpr int groups = D == 128 ? (PROBE ? 4 : 2) : (PROBE ? 1 : 2);
  static constexpr int nsoft = blocks * groups * 4;            // softmax warps
  static constexpr int threads = (nsoft + 2) * 32;
  static constexpr int ctas = D == 64 ? 2 : 1;                 // per SM
  static constexpr bool overlay = D == 128 || PROBE;           // P overwrites S
  // tensor memory: S [ops][kt], O [ops][D], and P [ops][kt/2] unless it overlays S
  static constexpr uint32_t t_o = ops * kt, t_p = overlay ? 0 : t_o + ops * D;
  static constexpr uint32_t p_stride = overlay ? kt : kt / 2;
  static constexpr uint32_t cols = D == 64 ? 256 : 512;
  static_assert((overlay ? t_o + ops * D : t_p + ops * kt / 2) <= cols, "tensor memory");
  // shared memory: operands [ops][D/64][128 rows][128 B], ring of key and value tiles
  // [D/64][kt rows][128 B], barriers, row exchange [2 buffers][nsoft/4 groups][128]
  static constexpr int op_bytes = BM * D * 2, tile = kt * D * 2, half = kt * 128;
  static constexpr int stages = D == 128 ? 4 : PROBE ? 8 : 5;
  static constexpr int sm_ring = ops * op_bytes;
  static constexpr int sm_bar = sm_ring + stages * tile;
  static constexpr int sm_x = sm_bar + 512;
  static constexpr int bytes = sm_x + 2 * (nsoft / 4) * BM * 4 + 1024;  // 1024: aligning the base
  static_assert(ctas * (bytes + 1024) <= 227 * 1024, "shared memory");
};

struct Barriers {
  uint64_t full[8], empty[8];
  uint64_t sfull[2], sfree[2], pfull[2][2], pvdone[2];
  uint64_t rowx[2], done;
};
static_assert(sizeof(Barriers) <= 512, "barrier region");

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <int D, bool PROBE>
__global__ void __launch_bounds__((Cfg<D, PROBE>::threads), (Cfg<D, PROBE>::ctas))
attend_tc_kernel(Params p, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap) {
  using C = Cfg<D, PROBE>;
  constexpr int KT = C::kt;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Barriers& bar = *reinterpret_cast<Barriers*>(smem + C::sm_bar);
  __shared__ uint32_t tmem_base_s;
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int hk = blockIdx.x % p.Hkv, part = blockIdx.y;
  let_next();  // the few-rows kernel of the same call, which does not depend on this one
  const int per = BM / p.g, tokens = C::blocks * per;  // tokens per row block and per CTA
  int b, tile;
  if (!find_tile(p, tokens, blockIdx.x / p.Hkv, &b, &tile)) return;
  const Seq sq = load_seq(p, b);
  const int tok0 = tile * tokens, ntok = min(tokens, sq.n - tok0);
  const int p0 = sq.first + tok0, p1 = p0 + ntok - 1;
  const TileRange<KT> range(p, p0, p1);
  const int chunk = (range.count + p.split - 1) / p.split;
  const int i0 = min(range.count, part * chunk), n = min(range.count, i0 + chunk) - i0;

  // Row r of row block h: its token within the CTA, -1 when there is none.
  auto token_of = [&](int h, int r) {
    const int t = h * per + r / p.g;
    return r < per * p.g && t < ntok ? t : -1;
  };
  auto rowid = [&](int t, int r) -> long long {
    return (long long)(sq.t0 + tok0 + t) * p.Hq + hk * p.g + r % p.g;
  };

  // Operands in the 128-byte swizzled layout (rows that do not exist are zero).
  for (int e = tid; e < C::ops * BM * (D / 8); e += C::threads) {
    const int o = e / (BM * (D / 8)), r = (e / (D / 8)) % BM, c = e % (D / 8);
    const int t = token_of(PROBE ? 0 : o, r);
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(PROBE && o ? p.r : p.q);
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (t >= 0 && c * 8 < p.d) x = *reinterpret_cast<const uint4*>(src + rowid(t, r) * p.d + c * 8);
    *reinterpret_cast<uint4*>(smem + o * C::op_bytes + (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) * 16)) = x;
  }
  if (tid == 0) {
    for (int s = 0; s < C::stages; ++s) { mbar_init(&bar.full[s], 1); mbar_init(&bar.empty[s], 1); }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar.sfull[s], 1);
      mbar_init(&bar.sfree[s], C::groups * 4);
      mbar_init(&bar.pfull[s][0], C::groups == 1 ? 4 : C::groups * 2);
      mbar_init(&bar.pfull[s][1], C::groups == 1 ? 4 : C::groups * 2);
      mbar_init(&bar.pvdone[s], 1);
      mbar_init(&bar.rowx[s], C::groups * 4);
    }
    mbar_init(&bar.done, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::nsoft + 1) {
    tmem_alloc(&tmem_base_s, C::cols);
    tmem_relinquish();
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = __shfl_sync(0xffffffffu, tmem_base_s, 0);
  volatile int* abort_p = &abort_flag;
  int* const status = p.status;
  constexpr int TO = kStatusTimeout;

  if (warp == C::nsoft + 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (n > 0) {
      const uint64_t xd = smem_desc_sw128(smem_u32(smem), 1024);
      const uint64_t kd = smem_desc_sw128(smem_u32(smem + C::sm_ring), 1024);
      const uint64_t vd = smem_desc_sw128_mn(smem_u32(smem + C::sm_ring), C::half, 1024);
      constexpr uint32_t id_s = idesc_bf16(BM, KT, false, false);
      constexpr uint32_t id_o = idesc_bf16(BM, D, false, true);
      constexpr uint32_t tile16 = C::tile >> 4;
      auto stage = [](int i) { return (uint32_t)(i % C::stages); };
      auto parity = [](int i) { return (uint32_t)((i / C::stages) & 1); };
      auto wait = [&](uint64_t* x, uint32_t par) { return warp_wait(x, par, status, TO, abort_p); };
      // S_o = operand o x K_i^T for operands o .. o + count - 1; the last ones of a tile free its stage
      auto scores = [&](auto o0, auto count, int i) {
        const uint32_t st = stage(2 * i);
        const uint64_t k = kd + (uint64_t)(st * tile16);
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int o = o0; o < o0 + count; ++o) {
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
              mma_ss(tbase + o * KT, xd + (uint64_t)(o * (C::op_bytes >> 4) + (s >> 2) * 1024 + (s & 3) * 2),
                     k + (uint64_t)((s >> 2) * (C::half >> 4) + (s & 3) * 2), id_s, s > 0);
            mma_commit(&bar.sfull[o]);
          }
          if (o0 + count == C::ops) mma_commit(&bar.empty[st]);
        }
        __syncwarp();
      };
      // O_o += P_o V_i over one half of the tile's keys
      auto values = [&](auto o0, auto count, int i, auto half) {
        const uint32_t st = stage(2 * i + 1);
        const uint64_t v = vd + (uint64_t)(st * tile16);
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int o = o0; o < o0 + count; ++o) {
#pragma unroll
            for (int u = 0; u < KT / 32; ++u) {
              const int s = half * (KT / 32) + u;
              mma_ts(tbase + C::t_o + o * D, tbase + C::t_p + o * C::p_stride + s * 8,
                     v + (uint64_t)(s * (2048 >> 4)), id_o, (i > 0 || s > 0) ? 1u : 0u);
            }
            if (half) mma_commit(&bar.pvdone[o]);
          }
          if (half && o0 + count == C::ops) mma_commit(&bar.empty[st]);
        }
        __syncwarp();
      };
      using I0 = std::integral_constant<int, 0>;
      using I1 = std::integral_constant<int, 1>;
      using Per = std::integral_constant<int, PROBE ? 2 : 1>;  // operands of a row block
      // The weights of half a tile at a time: the first product runs while the others are computed.
      auto block = [&](auto h, auto o, int i, bool more) {
        bool ok = wait(&bar.pfull[h][0], i & 1);
        if (ok) values(o, Per{}, i, I0{});
        ok = ok && wait(&bar.pfull[h][1], i & 1);
        if (ok) values(o, Per{}, i, I1{});
        if (ok && C::overlay && more) scores(o, Per{}, i + 1);
        return ok;
      };
      bool ok = wait(&bar.full[0], 0);
      if (ok) scores(I0{}, std::integral_constant<int, C::ops>{}, 0);
      for (int i = 0; i < n && ok; ++i) {
        const bool more = i + 1 < n;
        if (more) ok = wait(&bar.full[stage(2 * i + 2)], parity(2 * i + 2));
        if (!C::overlay && more && ok) {  // one operand with S of its own
          ok = wait(&bar.sfree[0], i & 1);
          if (ok) scores(I0{}, I1{}, i + 1);
        }
        ok = ok && wait(&bar.full[stage(2 * i + 1)], parity(2 * i + 1));
        ok = ok && block(I0{}, I0{}, i, more);
        if (C::blocks == 2) ok = ok && block(I1{}, std::integral_constant<int, C::blocks - 1>{}, i, more);
      }
      if (!ok) *abort_p = 1;
      if (elect_one()) mma_commit(&bar.done);
      __syncwarp();
      volatile int never = 0;
      mbar_wait(&bar.done, 0, status, TO, &never);
    }
    __syncwarp();
  } else if (warp == C::nsoft) {
    // ------------------------------------------------------------------ K/V loader
    const int frag = min(p.page, KT), nfrag = KT / frag;
    if (lane == 0) {
      tma_prefetch_map(&kmap);
      tma_prefetch_map(&vmap);
    }
    int issued = 0;
    for (int i = 0; i < n; ++i) {
      const int j = range.tile(i0 + i) * KT + lane * frag;
      int c2 = p.num_pages * p.Hkv;  // out of range: zeros
      if (lane < nfrag && j < sq.len) {
        const int pg = load_page(p, b, j >> p.page_shift);
        if (pg >= 0) c2 = pg * p.Hkv + hk;
      }
      bool ok = true;
      for (int kv = 0; kv < 2 && ok; ++kv) {
        const int x = 2 * i + kv, st = x % C::stages;
        if (x >= C::stages) ok = warp_wait(&bar.empty[st], ((x / C::stages) - 1) & 1, status, TO, abort_p);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&bar.full[st], C::tile);
        __syncwarp();
        if (lane < nfrag) {
          uint8_t* dst = smem + C::sm_ring + st * C::tile + lane * frag * 128;
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(dst + c * C::half, kv ? &vmap : &kmap, c * 64, j & (p.page - 1), c2, &bar.full[st]);
        }
        issued = x + 1;
      }
      if (!ok) break;
    }
    // Nothing may land in this CTA's shared memory after it exits.
    if (lane == 0) {
      volatile int never = 0;
      for (int x = issued > C::stages ? issued - C::stages : 0; x < issued; ++x)
        mbar_wait(&bar.full[x % C::stages], (x / C::stages) & 1, status, TO, &never);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ softmax + output
    // A group is four warps, one per tensor-memory lane quarter.
    constexpr int NG = C::groups;                  // groups that share a row block
    constexpr int NC = KT / NG;                    // keys of a tile per thread: 64 or 32
    const int r = (warp & 3) * 32 + lane;
    const int h = (warp >> 2) / NG, sub = (warp >> 2) % NG;  // row block, group within it
    const uint32_t lanes = tbase + ((uint32_t)((warp & 3) * 32) << 16);
    const int t = token_of(h, r);
    const int pos = t >= 0 ? p0 + t : p1;          // rows that do not exist are not written
    const int q0 = PROBE ? p0 : min(p0 + h * per, p1), q1 = PROBE ? p1 : min(q0 + per - 1, p1);
    const float c2 = p.inv_h * kLog2e, slack = 8.f / c2;
    float m = -CUDART_INF_F, d1 = 0.f, d2 = 0.f;
    // Exchange among the groups of a row: x[buffer][group][row].
    float* const xm = reinterpret_cast<float*>(smem + C::sm_x);
    auto slot = [&](int buf, int g) -> float& { return xm[((buf * C::blocks + h) * NG + g) * BM + r]; };
    int xphase = 0;  // phases of rowx used so far
    auto exchange = [&]() {
      if (NG == 1) return true;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.rowx[h]);
      return warp_wait(&bar.rowx[h], (xphase++) & 1, status, TO, abort_p);
    };
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      ok = warp_wait(&bar.sfull[h], i & 1, status, TO, abort_p);
      if (PROBE) ok = ok && warp_wait(&bar.sfull[1], i & 1, status, TO, abort_p);
      if (!ok) break;
      tc_fence_after();
      uint32_t s[NC / 32][32], tt[PROBE ? NC / 32 : 1][32];
#pragma unroll
      for (int c = 0; c < NC / 32; ++c) tmem_ld32(lanes + h * KT + sub * NC + c * 32, s[c]);
      if constexpr (PROBE) {
#pragma unroll
        for (int c = 0; c < NC / 32; ++c) tmem_ld32(lanes + KT + sub * NC + c * 32, tt[c]);
      }
      tmem_ld_wait();
      if (!C::overlay) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.sfree[h]);
      }
      const int k0 = range.tile(i0 + i) * KT, kb = k0 + sub * NC;
      if (!all_visible(p, q0, q1, k0, k0 + KT)) {
        // column c is visible when c <= hi and (c > lo or c < first)
        const int hi = pos - kb, lo = pos - p.window - kb, first = p.sinks - kb;
#pragma unroll
        for (int c = 0; c < NC; ++c)
          if (!(c <= hi && (c > lo || c < first))) {
            s[c >> 5][c & 31] = 0xFF800000u;
            if constexpr (PROBE) tt[c >> 5][c & 31] = 0u;  // of a slot that may hold anything
          }
      }
      float t4[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
      for (int c = 0; c < NC; c += 2)
        t4[(c >> 1) & 3] = max3(t4[(c >> 1) & 3], __uint_as_float(s[c >> 5][c & 31]), __uint_as_float(s[c >> 5][(c & 31) + 1]));
      float tm = fmaxf(max3(t4[0], t4[1], t4[2]), t4[3]);
      if (NG > 1) {
        slot(i & 1, sub) = tm;
        if (!(ok = exchange())) break;  // also: every group has read its scores, which P may overwrite
#pragma unroll
        for (int g = 0; g < NG; ++g) tm = fmaxf(tm, slot(i & 1, g));
      }
      // The products that read the previous P and O: where P overwrites S they precede this S in the
      // pipe; otherwise they are waited for before O is rescaled or P written.
      bool drained = C::overlay || i == 0;
      auto drain = [&]() {
        if (drained) return true;
        drained = true;
        const bool d = warp_wait(&bar.pvdone[h], (i - 1) & 1, status, TO, abort_p);
        tc_fence_after();
        return d;
      };
      const bool grow = tm > m + slack || (m == -CUDART_INF_F && tm > m);  // alike in every group
      if (__any_sync(0xffffffffu, grow)) {
        float sc = 1.f;
        if (grow) {
          sc = ex2((m - tm) * c2);  // 0 from -infinity
          m = tm;
          d1 *= sc;
          d2 *= sc;
        }
        if (i > 0) {
          if (!(ok = drain())) break;
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
      if (k0 + KT > sq.len) {
        // the last page's slots past the sequence's end may hold anything: their weight is zero,
        // and so must be the values
        const int x = 2 * i + 1, st = x % C::stages;
        if (!(ok = warp_wait(&bar.full[st], (x / C::stages) & 1, status, TO, abort_p))) break;
        // every warp zeroes every row: its own arrival below is then enough for the products it lets go
        for (int e = lane; e < (k0 + KT - sq.len) * (D / 8); e += 32) {
          const int row = sq.len - k0 + e / (D / 8), c = e % (D / 8);
          *reinterpret_cast<uint4*>(smem + C::sm_ring + st * C::tile + (c >> 3) * C::half + row * 128 + (c & 7) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      const float ref = m == -CUDART_INF_F ? 0.f : m * c2;
      const uint64_t c22 = pair(c2, c2), ref2 = pair(-ref, -ref);
      uint64_t sum[2] = {}, sumt[2] = {};  // pairs of partial sums
#pragma unroll
      for (int c = 0; c < NC / 32; ++c) {
        uint32_t w[16], wt[PROBE ? 16 : 1];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const uint64_t x = fma2(pair(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])), c22, ref2);
          float y0, y1;
          unpair(x, y0, y1);
          y0 = ex2(y0);
          y1 = ex2(y1);
          const uint64_t y = pair(y0, y1);
          sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], y);
          w[e / 2] = pack_bf16(y0, y1);
          if constexpr (PROBE) {
            const uint64_t z = mul2(y, pair(__uint_as_float(tt[c][e]), __uint_as_float(tt[c][e + 1])));
            sumt[(e >> 1) & 1] = add2(sumt[(e >> 1) & 1], z);
            float z0, z1;
            unpair(z, z0, z1);
            wt[e / 2] = pack_bf16(z0, z1);
          }
        }
        if (!(ok = drain())) break;
        tmem_st16(lanes + C::t_p + h * C::p_stride + sub * (NC / 2) + c * 16, w);
        if constexpr (PROBE) tmem_st16(lanes + C::t_p + C::p_stride + sub * (NC / 2) + c * 16, wt);
        // half of the tile's weights are there: with this group's last, or, alone, halfway
        if (c + 1 == NC / 32 || (NG == 1 && c + 1 == NC / 64)) {
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.pfull[h][NG == 1 ? c / (NC / 64) : sub / ((NG + 1) / 2)]);
        }
      }
      if (!ok) break;
      float a0, a1;
      unpair(add2(sum[0], sum[1]), a0, a1);
      d1 += a0 + a1;
      unpair(add2(sumt[0], sumt[1]), a0, a1);
      d2 += a0 + a1;
    }

    if (NG > 1 && ok) {  // the groups' sums
      ok = exchange();  // the last maxima have been read
      if (ok) {
        slot(0, sub) = d1;
        slot(1, sub) = d2;
        ok = exchange();
        d1 = d2 = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          d1 += slot(0, g);
          d2 += slot(1, g);
        }
      }
    }
    if (ok && n > 0) {
      ok = warp_wait(&bar.pvdone[h], (n - 1) & 1, status, TO, abort_p);
      if (PROBE) ok = ok && warp_wait(&bar.pvdone[1], (n - 1) & 1, status, TO, abort_p);
      tc_fence_after();
    }
    if (ok) {
      const float inv = d1 == 0.f ? 0.f : 1.f / d1, f1 = (1.f + d2 * inv) * inv;
      const long long id = t >= 0 ? rowid(t, r) : 0;
      const long long pid = (long long)part * p.tokens * p.Hq + id;
      float bad = 0.f;
      constexpr int NO = D / NG;  // output columns per thread
#pragma unroll 1
      for (int c = sub * NO; c < (sub + 1) * NO; c += 16) {
        uint32_t a[16], e[16];
        if (n > 0) {
          tmem_ld16(lanes + C::t_o + h * D + c, a);
          if (PROBE) tmem_ld16(lanes + C::t_o + D + c, e);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int u = 0; u < 16; ++u) a[u] = e[u] = 0u;
        }
        if (t < 0 || c >= p.dv) continue;
        if (p.split > 1) {
          float* dst = p.part_o + pid * (PROBE ? 2 : 1) * p.dv + c;
#pragma unroll
          for (int u = 0; u < 16; u += 4) {
            *reinterpret_cast<uint4*>(dst + u) = make_uint4(a[u], a[u + 1], a[u + 2], a[u + 3]);
            if (PROBE) *reinterpret_cast<uint4*>(dst + p.dv + u) = make_uint4(e[u], e[u + 1], e[u + 2], e[u + 3]);
          }
          continue;
        }
        uint32_t w[8];
#pragma unroll
        for (int u = 0; u < 16; u += 2) {
          float y0 = __uint_as_float(a[u]) * (PROBE ? f1 : inv);
          float y1 = __uint_as_float(a[u + 1]) * (PROBE ? f1 : inv);
          if (PROBE) {
            y0 = fmaf(-__uint_as_float(e[u]), inv, y0);
            y1 = fmaf(-__uint_as_float(e[u + 1]), inv, y1);
          }
          bad += (y0 + y1) * 0.f;
          w[u / 2] = pack_bf16(y0, y1);
        }
        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + id * p.dv + c);
        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
        dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
      if (t >= 0 && sub == 0) {
        if (p.split > 1) p.part_s[pid] = make_float4(m, d1, d2, 0.f);
        else if (p.lse) p.lse[id] = d1 == 0.f ? -CUDART_INF_F : (m * c2 + log2f(d1)) * kLn2;
      }
      if (p.split == 1) {
        // rows that are not finite, again by themselves: once every group has written its columns,
        // by the first
        if (NG > 1) {
          ok = exchange();  // the sums have been read
          if (ok) slot(0, sub) = bad;
          ok = ok && exchange();
          bad = 0.f;
#pragma unroll
          for (int g = 0; g < NG; ++g) bad += slot(0, g);
        }
        unsigned again = __ballot_sync(0xffffffffu, ok && t >= 0 && !(bad == 0.f) && sub == 0);
        while (again) {
          const int row = (warp & 3) * 32 + __ffs(again) - 1;
          again &= again - 1;
          const int tk = token_of(h, row);
          __syncwarp();
          exact_row<__nv_bfloat16>(p, b, p0 + tk, sq.t0 + tok0 + tk, hk * p.g + row % p.g);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::nsoft + 1) {
    tc_fence_after();
    tmem_dealloc(tbase, C::cols);
  }
}

template <int D, bool PROBE>
cudaError_t launch_tc_t(const Params& p, cudaStream_t s) {
  using C = Cfg<D, PROBE>;
  CUtensorMap kmap, vmap;
  cudaError_t err = encode_page_map(p, p.k, p.d, C::kt, &kmap);
  if (err == cudaSuccess) err = encode_page_map(p, p.v, p.dv, C::kt, &vmap);
  if (err != cudaSuccess) return err;
  const long long blocks = ((long long)p.tokens / (BM / p.g * C::blocks) + p.B) * p.Hkv;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch(attend_tc_kernel<D, PROBE>, dim3((unsigned)blocks, p.split), C::threads, C::bytes, 1, false, s, p,
                kmap, vmap);
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

int tc_tokens(int D, bool probe, int g) { return BM / g * (D == 128 && !probe ? 2 : 1); }

cudaError_t launch_attend_tc(const Params& p, int D, cudaStream_t s) {
  if (p.r) return D == 128 ? launch_tc_t<128, true>(p, s) : launch_tc_t<64, true>(p, s);
  return D == 128 ? launch_tc_t<128, false>(p, s) : launch_tc_t<64, false>(p, s);
}

}  // namespace paged
}  // namespace lla
