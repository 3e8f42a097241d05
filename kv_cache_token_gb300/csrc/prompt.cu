// Causal prompt attention with a sliding window and sink tokens
// (kvevict_attend_prompt), on the fifth-generation tensor cores.
//
// A CTA takes two row tiles of 128 rows.  The rows of a tile are tq = 128 / g
// (rounded down) neighbouring queries of the g heads of one KV head, so one
// copy of a K or V tile serves the whole group, and few queries share a tile's
// mask edges.  Per 128-key tile and row tile h:
//   S_h = Q_h K^T           (operands in shared memory, S_h in tensor memory)
//   P_h = 2^(S_h c - m)     one thread per row reads its 128 logits once, keeps
//                           the running maximum m (moved only when it grows by
//                           more than 2^8) and the sum in fp32, and writes P as
//                           bf16 over S_h
//   O_h += P_h V            (P_h from tensor memory, V from shared memory)
// While the threads of one row tile exponentiate, the tensor cores work for the
// other.  One warp issues the MMAs, one the TMA copies (K and V tiles through
// one ring; Q once).  Tensor memory: S_0, S_1 at columns 0 and 128, O_0 and O_1
// after them.
//
// Tiles no row of the CTA sees are not visited: the list is the sinks' tiles,
// then those from the window's start to the last row.  A tile every row of a
// row tile sees in full is not masked.  In the others hidden logits become
// -inf, and since 0 x inf and 0 x NaN would reach O from a hidden key's value
// row, value elements of such keys that are not finite are set to zero in
// shared memory first, noted, and added at the end to the rows that do see
// them.
//
// Measured (d = 128), ten launches in a row at 2070 MHz and several hundred, where
// the power limit holds the clock near 1930: 16384 tokens, 32 heads, every
// earlier key 1.42 / 1.52 ms, 1550 / 1450 TFLOP/s, 0.78 / 0.83 of the measured
// bf16 rate of a burst / of seconds; 16385 tokens, 64 heads, window 4096 and 4
// sinks 1.57 / 1.62 ms, 1220 / 1190 TFLOP/s, the rest in the three masked tiles of
// every 35 and in starting 4104 CTAs.  No unit is full (8192 tokens: tensor pipe
// active 59% of the time, issue slots 38%): a row tile's chain, S to P to P V and
// the next S, is what a tile takes (tensor memory holds no second S beside two O
// of 128 columns): of 3150 cycles the softmax takes 1400, its own MMAs 1024, and
// the other row tile's MMAs and four hand-overs the rest.  Halving the bytes of K
// and V per tile gains 3%.  Slower were, at d = 128: P handed over in halves (the
// in-order issuer then waits for one row tile with the other ready), an issuing
// warp a row tile (both chains then run in step and share the tensor cores; 7%
// with P in halves, 14% without), the maximum taken alongside the exponentials,
// two threads a row, key tiles of 64 with two S buffers, and part of the
// exponentials by a polynomial.  Heads of 64 take 1.14 ms for the 16384 tokens,
// 970 TFLOP/s.  There too no unit is full (8192 tokens: issue slots 45%,
// exponentials 38%, tensor pipe 37%): two softmax warps a scheduler, each a chain
// of dependent steps.  S of the next tile computed beside P, which d = 64 has room
// for, changed nothing; two threads a row were not tried there.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "kvevict_internal.cuh"
#include "packed_math.cuh"
#include "tcgen05.cuh"

namespace kve {

namespace {

constexpr int kRowTile = 128, kKeyTile = 128;
constexpr int kPromptThreads = 384;      // two softmax warpgroups, one of copies and MMA issue
constexpr int kCopyWarp = 8, kMmaWarp = 9;
constexpr float kPromptGrow = 8.f;       // log2

struct PromptArgs {
  __nv_bfloat16* out;
  float* lse;
  const __nv_bfloat16* v;
  uint32_t* status;
  int n, g, Hq, Hkv, lanes, tq, qtiles, sinks, window;
  float scale2;                          // log2(e) / sqrt(d)
};
struct PromptMaps {
  CUtensorMap q, k, v;
};

template <int D>
struct PromptCfg {
  static constexpr int kHalves = D / 64;                        // 64-element column blocks of a row
  static constexpr int kTile = kHalves * kRowTile * 128;        // bytes of a Q, K or V tile
  static constexpr int kSlots = D == 128 ? 5 : 8;               // K and V tiles in the ring
  static constexpr int kSmem = 2 * kTile + kSlots * kTile + 1024;
  static constexpr uint32_t kIdS = tc::idesc_bf16(kRowTile, kKeyTile, 0);
  static constexpr uint32_t kIdO = tc::idesc_bf16(kRowTile, D, 1);
  static constexpr int kOCol = 256;                             // O_h at kOCol + h * 128
};

struct PromptBars {
  uint64_t q_full, s_full[2], p_full[2], o_full[2], full[8], empty[8];
};

// Which queries a row tile holds and which entries of the CTA's tile list it
// takes: the sinks' tiles, then those from `from` to `to`.  (A tile of hidden
// keys only may be among them; its weights are all zero.)
struct RowTile {
  int a, b;            // first and last query (b < a: none, and no tiles)
  int from, to;
  __device__ __forceinline__ bool active(int t, int sink_tiles) const { return t <= to && (t < sink_tiles || t >= from); }
  __device__ __forceinline__ bool full(int tile, int sinks, int window) const {
    const int k0 = tile * kKeyTile, k1 = k0 + kKeyTile - 1;
    return k1 <= a && (k0 >= b - window + 1 || k1 < sinks);
  }
};

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// true in one thread of the (converged) warp
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
// mbar_wait_bounded with a long suspension a poll (100 us; a completed phase ends
// it at once): a waiting warp that polls often takes issue slots from the other
// row tile's exponentials.  Gives up after 2^14 polls, about a second and a half,
// and returns false.  A prompt has hundreds of waits a CTA, each behind the one
// that failed, so the caller then waits no more: copies and MMAs end, and the
// softmax, whose warps must stay together, runs on without waiting.  Nothing is
// in flight by then: whoever gives up, the others have waited about as long.
__device__ __forceinline__ bool mbar_sleep(uint64_t* bar, uint32_t parity, uint32_t* status) {
  const uint32_t at = smem_u32(bar);
  for (int i = 0; i < (1 << 14); ++i) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(at), "r"(parity), "r"(100000)
        : "memory");
    if (__builtin_expect(ok, 1)) return true;
  }
  set_status(status, ST_TIMEOUT);
  return false;
}
__device__ __forceinline__ void tma_load3(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load4(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}
// MMA and commit by one thread of a converged warp: the predicate is on the
// instruction, so the operands stay in the warp's uniform registers.  (Inside
// a branch taken by one thread every operand is moved there again for every
// instruction, and the issue, 56 cycles an MMA, was what bounded the kernel.)
__device__ __forceinline__ void mma_ss_if(uint32_t who, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, w;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 w, %5, 0;\n"
      " @w tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(who)
      : "memory");
}
__device__ __forceinline__ void mma_ts_if(uint32_t who, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, w;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 w, %5, 0;\n"
      " @w tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(who)
      : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t who, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred w;\n setp.ne.b32 w, %1, 0;\n"
      " @w tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(tc::saddr(bar)),
      "r"(who)
      : "memory");
}
// bits 15 and 31 set where the bf16 halves of w are infinite or NaN
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }

template <int D>
__global__ void __launch_bounds__(kPromptThreads, 1) prompt_kernel(const PromptArgs a,
                                                                   const __grid_constant__ PromptMaps mp) {
  using C = PromptCfg<D>;
  extern __shared__ unsigned char dsm[];
  __shared__ __align__(8) PromptBars bar;
  __shared__ uint32_t sh_taddr;
  __shared__ int sh_bad;
  const int tid = threadIdx.x, warp = tid >> 5, lane_id = tid & 31;
  // longest rows first
  const int qt = a.qtiles - 1 - static_cast<int>(blockIdx.x) / a.lanes, lane = static_cast<int>(blockIdx.x) % a.lanes;
  const int b = lane / a.Hkv, kh = lane % a.Hkv;
  const int i0 = qt * 2 * a.tq;
  RowTile rt[2];
  const int last = min(i0 + 2 * a.tq, a.n) - 1;
  const int near_tile = max(0, i0 - a.window + 1) / kKeyTile;
  const int sink_tiles = min((min(a.sinks, a.n) + kKeyTile - 1) / kKeyTile, near_tile);
  const int tiles = sink_tiles + last / kKeyTile - near_tile + 1;
  auto tile_of = [&](int t) { return t < sink_tiles ? t : near_tile + (t - sink_tiles); };
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    rt[h].a = i0 + h * a.tq;
    rt[h].b = min(rt[h].a + a.tq, a.n) - 1;
    const int from = near_tile * kKeyTile < a.sinks ? near_tile : max(0, rt[h].a - a.window + 1) / kKeyTile;
    rt[h].from = sink_tiles + from - near_tile;
    rt[h].to = rt[h].b < rt[h].a ? -1 : sink_tiles + rt[h].b / kKeyTile - near_tile;
  }

  unsigned char* base = dsm + ((1024u - (smem_u32(dsm) & 1023u)) & 1023u);
  unsigned char* sq = base;
  unsigned char* skv = base + 2 * C::kTile;
  if (warp == kMmaWarp) tc::alloc(&sh_taddr, 512);
  if (tid == 0) {
    sh_bad = 0;
    mbar_init(&bar.q_full, 1);
    for (int h = 0; h < 2; ++h) {
      mbar_init(&bar.s_full[h], 1);
      mbar_init(&bar.p_full[h], 4);
      mbar_init(&bar.o_full[h], 1);
    }
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&bar.full[s], 1);
      mbar_init(&bar.empty[s], 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tm = __reduce_or_sync(0xffffffffu, sh_taddr);

  if (warp >= kCopyWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == kCopyWarp && lane_id == 0) {
      // Q, then K(0), V(0), K(1), V(1), ...
      const int rows = a.g * a.tq;
      uint32_t bytes = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (rt[h].b >= rt[h].a) bytes += static_cast<uint32_t>(C::kHalves * rows * 128);
      mbar_arrive_expect_tx(&bar.q_full, bytes);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (rt[h].b < rt[h].a) continue;
        for (int c = 0; c < C::kHalves; ++c)
          tma_load4(sq + h * C::kTile + c * (kRowTile * 128), &mp.q, c * 64, rt[h].a, kh * a.g, b, &bar.q_full);
      }
      for (int u = 0; u < 2 * tiles; ++u) {
        const int s = u % C::kSlots, use = u / C::kSlots;
        if (use > 0 && !mbar_sleep(&bar.empty[s], (use - 1) & 1, a.status)) break;
        mbar_arrive_expect_tx(&bar.full[s], C::kTile);
        const CUtensorMap* m = (u & 1) ? &mp.v : &mp.k;
        for (int c = 0; c < C::kHalves; ++c)
          tma_load3(skv + s * C::kTile + c * (kKeyTile * 128), m, c * 64, tile_of(u >> 1) * kKeyTile, lane, &bar.full[s]);
      }
    } else if (warp == kMmaWarp) {
      [&] {
        // The whole warp runs the loop (so that descriptors stay in uniform
        // registers) and one thread issues.  Everything a step needs is ready
        // before its waits: bookkeeping between a wait and an issue is time the
        // tensor cores idle.
        const uint32_t leader = elect_one() ? 1u : 0u;
        const uint64_t dq0 = tc::desc_sw128(smem_u32(sq), 16, 1024);
        const uint64_t dk0 = tc::desc_sw128(smem_u32(skv), 16, 1024);
        const uint64_t dv0 = tc::desc_sw128(smem_u32(skv), kKeyTile * 128, 1024);
        if (!mbar_sleep(&bar.q_full, 0, a.status)) return;
        uint32_t done[2] = {0u, 0u};                 // P V products of a row tile so far
        bool now[2], before[2] = {false, false};
        int sk = 0, kphase = 0, sv = 1, vphase = 0;  // ring slots of K(t) and V(t - 1), and their phases
#pragma unroll
        for (int h = 0; h < 2; ++h) now[h] = rt[h].active(0, sink_tiles);
        // step t: O += P V(t - 1), then S(t), a row tile at a time
#pragma unroll 1
        for (int t = 0; t <= tiles; ++t) {
          const uint64_t dv = tc::desc_add(dv0, sv * C::kTile), dk = tc::desc_add(dk0, sk * C::kTile);
          if (t > 0 && !mbar_sleep(&bar.full[sv], vphase, a.status)) return;
          bool k_there = false;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (before[h]) {
              const uint32_t acc = done[h] > 0 ? 1u : 0u;
              if (!mbar_sleep(&bar.p_full[h], done[h] & 1u, a.status)) return;
              tc::fence_after();
#pragma unroll
              for (int ks = 0; ks < kKeyTile / 16; ++ks)
                mma_ts_if(leader, tm + C::kOCol + h * 128, tm + h * 128 + ks * 8, tc::desc_add(dv, ks * 2048), C::kIdO,
                          ks > 0 ? 1u : acc);
              if (t - 1 == rt[h].to) commit_if(leader, &bar.o_full[h]);
              ++done[h];
            }
            if (now[h]) {
              if (!k_there && !mbar_sleep(&bar.full[sk], kphase, a.status)) return;
              k_there = true;
              tc::fence_after();
              const uint64_t dq = tc::desc_add(dq0, h * C::kTile);
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks) {
                const int off = (ks >> 2) * (kKeyTile * 128) + (ks & 3) * 32;
                mma_ss_if(leader, tm + h * 128, tc::desc_add(dq, off), tc::desc_add(dk, off), C::kIdS, ks > 0 ? 1u : 0u);
              }
              commit_if(leader, &bar.s_full[h]);
            }
          }
          if (t < tiles) commit_if(leader, &bar.empty[sk]);
          if (t > 0) commit_if(leader, &bar.empty[sv]);
          sk += 2;
          if (sk >= C::kSlots) { sk -= C::kSlots; kphase ^= 1; }
          if (t > 0) {
            sv += 2;
            if (sv >= C::kSlots) { sv -= C::kSlots; vphase ^= 1; }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            before[h] = now[h];
            now[h] = t + 1 < tiles && rt[h].active(t + 1, sink_tiles);
          }
        }
      }();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int h = warp >> 2;                       // row tile
    const int row = tid & (kRowTile - 1);
    const RowTile my = h ? rt[1] : rt[0];
    const int head = row / a.tq, i = my.a + row - head * a.tq;
    const bool valid = head < a.g && i < a.n;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t aS = tm + lane_off + h * 128, aO = tm + lane_off + C::kOCol + h * 128;
    const float2 sc = make_float2(a.scale2, a.scale2);
    float m_run = -INFINITY, l_run = 0.f;
    int cnt = 0;
    bool alive = true;         // no wait has given up
#pragma unroll 1
    for (int t = 0; t < tiles; ++t) {
      const int tile = tile_of(t);
      if (!my.active(t, sink_tiles)) continue;
      const bool full = my.full(tile, a.sinks, a.window);
      const int k0 = tile * kKeyTile;
      if (alive) alive = mbar_sleep(&bar.s_full[h], cnt & 1, a.status);
      tc::fence_after();
      uint32_t s[8][16];
#pragma unroll
      for (int c = 0; c < 4; ++c) tc::ld16(aS + c * 16, s[c]);
      tc::wait_ld();
#pragma unroll
      for (int c = 0; c < 4; ++c) tc::hold16(s[c]);
#pragma unroll
      for (int c = 4; c < 8; ++c) tc::ld16(aS + c * 16, s[c]);
      if (!full) {
        tc::wait_ld();
#pragma unroll
        for (int c = 4; c < 8; ++c) tc::hold16(s[c]);
        // keys up to the row's own, from its window's start or among the sinks
        const int hi = i - k0, lo = i - a.window + 1 - k0, sk = a.sinks - k0;
#pragma unroll
        for (int c = 0; c < 8; ++c)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int k = c * 16 + e;
            if (!(k <= hi && (k >= lo || k < sk))) s[c][e] = 0xFF800000u;
          }
        // values of keys that some row of the tile does not see (one a thread)
        const int key = k0 + row;
        if (!(key <= my.a && (key >= my.b - a.window + 1 || key < a.sinks))) {
          const int u = 2 * t + 1, sl = u % C::kSlots;
          if (alive) alive = mbar_sleep(&bar.full[sl], (u / C::kSlots) & 1, a.status);
          unsigned char* vr = skv + sl * C::kTile + row * 128;
          bool bad = false;
#pragma unroll 1
          for (int c = 0; c < C::kHalves * 8; ++c) {
            uint4* p = reinterpret_cast<uint4*>(vr + (c >> 3) * (kKeyTile * 128) + (((c & 7) ^ (row & 7)) << 4));
            uint4 x = *p;
            const uint32_t f0 = not_finite(x.x), f1 = not_finite(x.y), f2 = not_finite(x.z), f3 = not_finite(x.w);
            if (f0 | f1 | f2 | f3) {
              // each flagged half to zero
              x.x &= ~((f0 >> 15) * 0xFFFFu);
              x.y &= ~((f1 >> 15) * 0xFFFFu);
              x.z &= ~((f2 >> 15) * 0xFFFFu);
              x.w &= ~((f3 >> 15) * 0xFFFFu);
              *p = x;
              bad = true;
            }
          }
          if (bad) sh_bad = 1;
        }
        fence_proxy_async();
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if (c == 4 && full) {
          tc::wait_ld();
#pragma unroll
          for (int x = 4; x < 8; ++x) tc::hold16(s[x]);
        }
#pragma unroll
        for (int e = 0; e < 16; e += 2)
          mx[(e >> 1) & 3] = fmaxf(mx[(e >> 1) & 3], fmaxf(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])));
      }
      const float tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale2;
      float factor = 1.f;
      if (tmax > m_run + kPromptGrow) {
        factor = m_run == -INFINITY ? 0.f : hw_exp2(m_run - tmax);
        m_run = tmax;
        l_run *= factor;
      }
      const bool grow = __any_sync(0xffffffffu, factor != 1.f);
      const float negm = m_run == -INFINITY ? 0.f : -m_run;
      const float2 nm = make_float2(negm, negm);
      float2 sum0 = make_float2(0.f, 0.f), sum1 = make_float2(0.f, 0.f);
      // exponentials of chunk c in place, then chunk c - 1 rounded and stored:
      // a chunk's stores never wait for exponentials just issued.  (Chunks of 16
      // keys; with 32 the last one's rounding and store, which nothing covers,
      // cost 2% at d = 64.)
#pragma unroll
      for (int c = 0; c < 9; ++c) {
        if (c < 8) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            uint32_t* v = &s[c][2 * e];
            const float2 y = f2_fma(make_float2(__uint_as_float(v[0]), __uint_as_float(v[1])), sc, nm);
            v[0] = __float_as_uint(hw_exp2(y.x));
            v[1] = __float_as_uint(hw_exp2(y.y));
          }
        }
        if (c > 0) {
          uint32_t p[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t* v = &s[c - 1][2 * e];
            const float2 z = make_float2(__uint_as_float(v[0]), __uint_as_float(v[1]));
            if (e & 1) sum1 = f2_add(sum1, z);
            else sum0 = f2_add(sum0, z);
            p[e] = bf16x2(z.x, z.y);
          }
          tc::st8(aS + (c - 1) * 8, p);
        }
      }
      // O is rescaled while nothing adds to it: S(t) was issued after P V of
      // the tile before, and its barrier covers both
      if (cnt > 0 && grow) {
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t o[16];
          tc::ld16(aO + c * 16, o);
          tc::wait_ld();
          tc::hold16(o);
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * factor);
          tc::st16(aO + c * 16, o);
        }
      }
      l_run += (sum0.x + sum0.y) + (sum1.x + sum1.y);
      tc::wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane_id == 0) mbar_arrive(&bar.p_full[h]);
      ++cnt;
    }
    if (cnt > 0) {
      if (alive) (void)mbar_sleep(&bar.o_full[h], 0, a.status);
      tc::fence_after();
    }
    // the other row tile may have zeroed values this one's rows see
    asm volatile("bar.sync 1, 256;" ::: "memory");
    const bool patch = sh_bad != 0;
    const float inv = 1.f / l_run;
    if (cnt > 0) {
      __nv_bfloat16* orow =
          a.out + ((static_cast<size_t>(b) * a.n + (valid ? i : 0)) * a.Hq + static_cast<size_t>(kh) * a.g + (valid ? head : 0)) * D;
#pragma unroll 1
      for (int c = 0; c < D / 16; ++c) {
        uint32_t o[16];
        tc::ld16(aO + c * 16, o);
        tc::wait_ld();
        tc::hold16(o);
        float x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(o[e]);
        if (patch && valid) {
#pragma unroll 1
          for (int t = 0; t < tiles; ++t) {
            const int tile = tile_of(t);
            bool edge = false;
#pragma unroll
            for (int o2 = 0; o2 < 2; ++o2)
              edge |= rt[o2].active(t, sink_tiles) && !rt[o2].full(tile, a.sinks, a.window);
            if (!edge) continue;
            for (int k = tile * kKeyTile; k < min(tile * kKeyTile + kKeyTile, i + 1); ++k) {
              if (!(i - k < a.window || k < a.sinks)) continue;
              const uint32_t* vp =
                  reinterpret_cast<const uint32_t*>(a.v + (static_cast<size_t>(lane) * a.n + k) * D + c * 16);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const uint32_t w = vp[e], f = not_finite(w);
                if (f & 0x8000u) x[2 * e] += __uint_as_float(w << 16);
                if (f & 0x80000000u) x[2 * e + 1] += __uint_as_float(w & 0xFFFF0000u);
              }
            }
          }
        }
        if (valid) {
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = bf16x2(x[2 * e] * inv, x[2 * e + 1] * inv);
          uint4* dst = reinterpret_cast<uint4*>(orow + c * 16);
          dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
          dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
      if (valid && a.lse)
        a.lse[(static_cast<size_t>(b) * a.Hq + static_cast<size_t>(kh) * a.g + head) * a.n + i] =
            (m_run + log2f(l_run)) * 0.6931471805599453f;
    }
    tc::fence_before();
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after();
    tc::dealloc(tm, 512);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

template <int D>
cudaError_t run_prompt(const PromptArgs& a, const PromptMaps& mp, cudaStream_t st) {
  const long long ctas = static_cast<long long>(a.qtiles) * a.lanes;
  if (ctas > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  prompt_kernel<D><<<static_cast<unsigned>(ctas), kPromptThreads, PromptCfg<D>::kSmem, st>>>(a, mp);
  return cudaGetLastError();
}

}  // namespace

cudaError_t prepare_prompt() {
  cudaError_t e = cudaFuncSetAttribute(prompt_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, PromptCfg<128>::kSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(prompt_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, PromptCfg<64>::kSmem);
  return e;
}

cudaError_t launch_attend_prompt(const Ctx& ctx, const void* q, const void* k, const void* v, int n, int sinks,
                                 int window, void* out, float* lse, cudaStream_t st) {
  const Dims& dm = ctx.dims;
  const auto encode = map_encoder();
  if (!encode) return cudaErrorNotSupported;
  PromptArgs a;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.status = ctx.ws.status;
  a.n = n; a.g = dm.g; a.Hq = dm.Hq; a.Hkv = dm.Hkv; a.lanes = dm.lanes;
  a.tq = kRowTile / dm.g;
  a.qtiles = (n - 1) / (2 * a.tq) + 1;
  a.window = window > 0 ? (window < n ? window : n) : n;
  a.sinks = sinks < n ? sinks : n;
  a.scale2 = 1.4426950408889634f / sqrtf(static_cast<float>(dm.d));
  PromptMaps mp;
  const cuuint64_t row = static_cast<cuuint64_t>(dm.d) * 2;
  const cuuint32_t one[4] = {1, 1, 1, 1};
  {
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(dm.d), static_cast<cuuint64_t>(n),
                                static_cast<cuuint64_t>(dm.Hq), static_cast<cuuint64_t>(dm.B)};
    const cuuint64_t strides[3] = {row, row * n, row * n * dm.Hq};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(a.tq), static_cast<cuuint32_t>(dm.g), 1};
    if (encode(&mp.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(q), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  for (int i = 0; i < 2; ++i) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(dm.d), static_cast<cuuint64_t>(n),
                                static_cast<cuuint64_t>(dm.lanes)};
    const cuuint64_t strides[2] = {row, row * n};
    const cuuint32_t box[3] = {64, kKeyTile, 1};
    if (encode(i ? &mp.v : &mp.k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(i ? v : k), dims, strides, box,
               one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  return dm.d == 128 ? run_prompt<128>(a, mp, st) : run_prompt<64>(a, mp, st);
}

}  // namespace kve
