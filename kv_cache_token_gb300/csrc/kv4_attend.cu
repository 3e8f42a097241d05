// Decode attention over the 4-bit cache (kvevict_kv4_attend).
//
// For every lane the g query heads of its group attend the lane's tokens.  A
// page (16 tokens, K and V codes and scales: 2320 bytes at d = 128) is one
// tile of one warp.  A round is two pages for each consumer warp of a CTA; the
// rounds of all lanes, one after the other, are cut into equal runs, one per
// CTA of a grid of one CTA per SM, so every SM streams the same number of
// pages whatever the lanes' lengths.  One more warp of the CTA feeds the
// others: its thread w looks up warp w's page and issues its copy (one
// cp.async.bulk), so the lookups of a round cost one warp's instructions, not
// eleven.  A consumer warp keeps its own running maximum, sum and output; the
// warps of a CTA are joined in shared memory when the CTA leaves a lane.  A
// lane that one CTA holds whole is written at once; parts of a lane go to
// scratch, and the CTA that delivers the last one joins them in order (the
// same result whoever is last).
//
// The codes are never converted.  A nibble n masked in place is the fp16
// subnormal n 2^-22 (bits 2-5 of a half) or n 2^-18 (bits 6-9), which the
// tensor core multiplies exactly: one AND per operand register of two codes
// and one rotation per word of eight.  (Products are aligned by their nominal
// exponents, so a subnormal that far down costs the sum up to 8 bits of 24;
// bits 0-3 would cost 10.)  The factors 2^-22 and 2^-18 belong to fixed
// elements of q (folded into q) or fixed rows of the output (folded in at the
// end), and the codes' offset of 8 is subtracted from the products:
//   S = sum_w ks_w (sum_j n_j q_j - 8 sum_j q_j)       (w: groups of 32)
//   O_w = sum_t (p_t vs_tw) n_t - 8 sum_t p_t vs_tw
// the first through the accumulator's start value, the second by one more MMA
// per group whose left operand is ones.
//
// Weights times value scales are the right operand of O, in fp16 (11 bits).
// Their range is kept by including the value scale's exponent e_t in the
// maximum: u_t = 2^(s_t + e_t - m + 8) with m the running maximum of s + e, so
// that the largest weight-scale product of the lane is between 2^8 and 2^15
// and whatever is below 2^-33 of it is lost; the softmax sum takes u_t 2^-e_t
// in fp32.
//
// Measured: 16 lanes of 131072 tokens, groups of 4 (304 MB): 69 us, 4.4 TB/s,
// 0.65 of the measured copy bandwidth (the copies alone, without the work on
// them, 56 us); 128 lanes of 3276 tokens, groups of 8: 19.8 us, of which the
// stream is 13.  Bound by latency: 289 instructions a page take 0.43 of the issue
// slots and as much of the integer pipe, but a scheduler has three warps (12 a SM
// are all that the accumulators leave room for), each a chain of masks, MMAs and
// exponentials, and a round's copies wait for its slowest warp.  One page a tile
// with 15 warps took 78 us, 15 warps with two pages (spilled registers) 74.
#include "kv4_page.cuh"
#include "kvevict_internal.cuh"
#include "packed_math.cuh"

namespace kve {

namespace {

constexpr int kMaxCtas = 256;          // parts the scratch holds: two a CTA
constexpr int kJoinRounds = 3;         // what joining a lane's parts costs, in rounds
constexpr float kBoost = 8.f;          // log2 of the largest u when m was set
constexpr float kGrow = 6.f;           // m moves when some s + e exceeds it by more
constexpr float kUnscale = 512.f;      // logits: 2^22 of the codes over 2^13 of the query

struct Kv4Attend {
  const unsigned char* pages;
  const int32_t* table;
  const int32_t* lens;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;
  uint32_t* status;
  int32_t* arrived;     // [lanes] parts delivered; zero between calls
  float* parts;         // [2 * CTAs][g][D + 4]: sums, maximum, sum of weights, two unused
  int num_pages, max_pages, lanes, g, Hkv, Hq, sinks, window;
  float scale2;         // log2(e) / sqrt(d)
};

template <int D, int NT>
struct Kv4Cfg {
  static constexpr int kWarps = NT == 1 ? 11 : 7;     // consumer warps: 168 / 255 registers a thread
  static constexpr int kThreads = (kWarps + 1) * 32;
  static constexpr int kPages = 2;                    // pages of a tile
  static constexpr int kStages = 3;                   // tiles in flight per consumer warp
  static constexpr int kHeads = 8 * NT;
  static constexpr int kOStride = D + 4;              // floats; 4 apart: heads land in different banks
  static constexpr int kStageBytes = kPages * Kv4Page<D>::kBytes;
  static constexpr int kQSlots = 4;                   // lanes' queries in flight
  static constexpr int kQBytes = kHeads * D * 2;
  static constexpr int kMergeOff = kWarps * kStages * kStageBytes;
  static constexpr int kQOff = kMergeOff + kWarps * kHeads * kOStride * 4;
  static constexpr int kFragOff = kQOff + kQSlots * kQBytes;
  // a lane's query as MMA fragments: per head tile and group, 16 + 8 bytes a thread; then a factor pair
  static constexpr int kFragBytes = NT * 32 * (Kv4Page<D>::kG * 24 + 8);
  static constexpr int kFixed = kFragOff + kFragBytes;
  static constexpr int smem_for(int lanes) { return kFixed + (2 * lanes + 1) * 4; }
  static_assert(kMergeOff % 16 == 0 && kQOff % 16 == 0 && kFragOff % 16 == 0 && kFixed % 16 == 0, "16-byte pieces");
  // the join of a lane's parts keeps a factor per (part, head) where the merge buffer was
  static_assert(kMaxCtas * kHeads <= kWarps * kHeads * kOStride, "factors fit");
};

// What a lane shows: tokens below `first` and from `near` on, of n.
struct Seen {
  int n, first, near;
  int pa, pb, pages;      // pages [0, pa) and [pb, ...), pages in all
};
__device__ __forceinline__ Seen seen_of(int n, int sinks, int window) {
  Seen s;
  s.n = n;
  const int np = (n + 15) >> 4;
  if (window > 0) {
    s.first = min(sinks, n);
    s.near = max(s.first, n - min(n, window));
    s.pa = (s.first + 15) >> 4;
    s.pb = max(s.pa, s.near >> 4);
    s.pages = s.pa + (np - s.pb);
  } else {
    s.first = n;
    s.near = n;
    s.pa = np;
    s.pb = np;
    s.pages = np;
  }
  return s;
}

__device__ __forceinline__ void mma_f16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1, float c0, float c1, float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t half2_mul(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// The four operand registers of a word: nibbles (i, i + 4), as fp16 n 2^-22 for
// i = 0, 2 and n 2^-18 for i = 1, 3.
__device__ __forceinline__ void code_pairs(uint32_t word, uint32_t (&x)[4]) {
  const uint32_t r = __funnelshift_r(word, word, 8);
  x[0] = word & 0x003C003Cu;
  x[1] = word & 0x03C003C0u;
  x[2] = r & 0x003C003Cu;
  x[3] = r & 0x03C003C0u;
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127

template <int D, int NT>
__global__ void __launch_bounds__(Kv4Cfg<D, NT>::kThreads, 1) kv4_attend_kernel(const Kv4Attend a) {
  using P = Kv4Page<D>;
  using C = Kv4Cfg<D, NT>;
  constexpr int kG = P::kG, kDt = D / 16, W = C::kWarps, S = C::kStages, NP = C::kPages;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint64_t sh_full[W][S], sh_empty[W][S], sh_qfull[C::kQSlots], sh_qempty[C::kQSlots];
  __shared__ float sh_ml[W][C::kHeads][2];
  __shared__ int sh_scan[40];
  __shared__ int sh_most;          // rounds of the longest lane
  const int tid = threadIdx.x, lane_id = tid & 31, warp = tid >> 5;
  if (tid == 0) sh_most = 0;
  float* sh_o = reinterpret_cast<float*>(smem + C::kMergeOff);
  int* sh_prefix = reinterpret_cast<int*>(smem + C::kFixed);     // [lanes + 1] rounds before a lane
  int* sh_len = sh_prefix + a.lanes + 1;                         // [lanes]

  if (lane_id == 0) {
    if (warp < W) {
      for (int s = 0; s < S; ++s) {
        mbar_init(&sh_full[warp][s], NP);
        mbar_init(&sh_empty[warp][s], 1);
      }
    } else {
      for (int s = 0; s < C::kQSlots; ++s) {
        mbar_init(&sh_qfull[s], 1);
        mbar_init(&sh_qempty[s], 1);
      }
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // With a lane to a CTA, which lane it is does not depend on the lengths: its
  // page table comes to L2 while they are read.
  if (warp == C::kWarps && blockIdx.x < a.lanes) {
    const int32_t* row = a.table + static_cast<size_t>(blockIdx.x) * a.max_pages;
    if (lane_id * 32 < a.max_pages) prefetch_l2(row + lane_id * 32);
  }
  // --- rounds of every lane (each CTA computes the same table) ----------------
  {
    const int cap = a.max_pages * 16;
    int carry = 0;
    for (int base = 0; base < a.lanes; base += C::kThreads) {
      const int l = base + tid;
      int rounds = 0;
      if (l < a.lanes) {
        int n = a.lens[l];
        if (n < 0 || n > cap) {
          if (blockIdx.x == 0) set_status(a.status, ST_BAD_INDEX);
          n = n < 0 ? 0 : cap;
        }
        sh_len[l] = n;
        rounds = (seen_of(n, a.sinks, a.window).pages + W * NP - 1) / (W * NP);
        if (rounds == 0 && l % gridDim.x == blockIdx.x) {
          // nothing to attend
          const int b = l / a.Hkv, kh = l % a.Hkv;
          const size_t row = static_cast<size_t>(b) * a.Hq + static_cast<size_t>(kh) * a.g;
          for (int e = 0; e < a.g * D / 8; ++e) reinterpret_cast<uint4*>(a.out + row * D)[e] = make_uint4(0, 0, 0, 0);
          if (a.lse)
            for (int h = 0; h < a.g; ++h) a.lse[row + h] = -INFINITY;
        }
      }
      int tot;
      const int ex = block_excl_scan(rounds, sh_scan, &tot);
      if (l < a.lanes) sh_prefix[l] = carry + ex;
      if (rounds > 0) atomicMax(&sh_most, rounds);
      carry += tot;
    }
    if (tid == 0) sh_prefix[a.lanes] = carry;
  }
  __syncthreads();
  // Equal runs of rounds, or, with a CTA for every lane, a lane each where the
  // longest lane is no longer than a run and the join it spares (128 lanes of
  // 3276 tokens: 19.8 us, against 26.2 in equal runs; 32 lanes of 516: 8.0
  // against 10.6).
  const long long R = sh_prefix[a.lanes], G = min(static_cast<long long>(gridDim.x), R);   // G runs, none empty
  const bool lane_each = a.lanes <= gridDim.x && sh_most <= (R + gridDim.x - 1) / gridDim.x + kJoinRounds;
  int r_begin, r_end;
  if (lane_each) {
    if (blockIdx.x >= a.lanes) return;
    r_begin = sh_prefix[blockIdx.x];
    r_end = sh_prefix[blockIdx.x + 1];
    if (r_begin == r_end) return;
  } else {
    if (blockIdx.x >= G) return;
    r_begin = static_cast<int>(R * blockIdx.x / G);
    r_end = static_cast<int>(R * (blockIdx.x + 1) / G);
  }
  // the lane that holds round r_begin: prefix <= r_begin < next prefix
  int first_lane;
  {
    int lo = lane_each ? blockIdx.x : 0, hi = lane_each ? lo + 1 : a.lanes;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sh_prefix[mid] <= r_begin) lo = mid;
      else hi = mid;
    }
    first_lane = lo;
  }

  if (warp == W) {
    // --- feeding warp: thread 16 p + w copies page p of warp w's tiles ------------
    const int mine = NP == 2 ? lane_id & 15 : lane_id, part = NP == 2 ? lane_id >> 4 : 0;   // W <= 16
    const uint64_t pol = policy_evict_first();
    int l = first_lane - 1, lane_end = r_begin, lane_begin = 0, q_no = 0;
    Seen s = {};
    auto enter = [&](int r) {      // the lane of round r
      ++l;
      while (sh_prefix[l + 1] <= r) ++l;
      lane_begin = sh_prefix[l];
      lane_end = sh_prefix[l + 1];
      s = seen_of(sh_len[l], a.sinks, a.window);
    };
    // Lookups run kAhead rounds before the copies they serve: a page id is a
    // load from DRAM, about as long as a round.
    constexpr int kAhead = 8;
    int ids[kAhead], ls[kAhead], cur_l = -1, sent = 0;    // ls: the round's lane, or ~lane without a tile
    uint32_t have = 0;                                    // bit j: a page of its own in slot j
    auto ahead = [&](int r, int j) {
      ls[j] = ~l;
      have &= ~(1u << j);
      if (r >= r_end) return;
      if (r >= lane_end) enter(r);
      const int k = ((r - lane_begin) * W + mine) * NP;
      ls[j] = ~l;
      if (mine < W && k < s.pages) {
        ls[j] = l;
        if (k + part < s.pages) {
          const int kk = k + part;
          ids[j] = a.table[static_cast<size_t>(l) * a.max_pages + (kk < s.pa ? kk : s.pb + (kk - s.pa))];
          have |= 1u << j;
        }
      }
    };
#pragma unroll
    for (int j = 0; j < kAhead; ++j) ahead(r_begin + j, j);
    for (int r0 = r_begin; r0 < r_end; r0 += kAhead) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (r0 + j >= r_end) break;
        int id = ids[j];
        const bool tile = ls[j] >= 0, page = (have >> j) & 1u;
        const int il = tile ? ls[j] : ~ls[j];
        ahead(r0 + j + kAhead, j);
        if (il != cur_l) {
          cur_l = il;
          if (lane_id == 0) {
            const int slot = q_no % C::kQSlots, use = q_no / C::kQSlots;
            if (use > 0) (void)mbar_wait_bounded(&sh_qempty[slot], (use - 1) & 1, a.status);
            const size_t row = static_cast<size_t>(il / a.Hkv) * a.Hq + static_cast<size_t>(il % a.Hkv) * a.g;
            const uint32_t bytes = static_cast<uint32_t>(a.g) * D * 2;
            fence_proxy_async();
            mbar_arrive_expect_tx(&sh_qfull[slot], bytes);
            bulk_g2s(smem + C::kQOff + slot * C::kQBytes, a.q + row * D, bytes, &sh_qfull[slot]);
          }
          ++q_no;
        }
        if (tile) {
          const int st = sent % S, use = sent / S;
          if (use > 0) (void)mbar_wait_bounded(&sh_empty[mine][st], (use - 1) & 1, a.status);
          if (page) {
            if (id < 0 || id >= a.num_pages) { set_status(a.status, ST_BAD_INDEX); id = 0; }
            fence_proxy_async();
            mbar_arrive_expect_tx(&sh_full[mine][st], P::kUsed);
            bulk_g2s(smem + (mine * S + st) * C::kStageBytes + part * P::kBytes,
                     a.pages + static_cast<size_t>(id) * P::kBytes, P::kUsed, &sh_full[mine][st], pol);
          } else {
            mbar_arrive(&sh_full[mine][st]);
          }
          ++sent;
        }
        __syncwarp();
      }
    }
    // (a consumer that gave up waiting runs ahead of its copies: the CTA ends after they have landed)
    for (int i = max(0, sent - S); i < sent; ++i) (void)mbar_wait_bounded(&sh_full[mine][i % S], (i / S) & 1, a.status);
    return;
  }

  // --- consumer warps -----------------------------------------------------------
  const int gq = lane_id >> 2, cq = lane_id & 3;
  auto sync_consumers = [&]() { asm volatile("bar.sync 1, %0;" ::"n"(W * 32) : "memory"); };
  float o_acc[NT][kDt][4], corr_acc[NT][kG][2], m_run[NT][2], l_run[NT][2];
  uint4* frag_q = reinterpret_cast<uint4*>(smem + C::kFragOff) + lane_id;                        // [nt][w][32]
  float2* frag_s = reinterpret_cast<float2*>(smem + C::kFragOff + NT * kG * 32 * 16) + lane_id;  // [nt][w][32]
  float2* frag_c = frag_s + NT * kG * 32;                                                         // [nt][32]
  auto reset_acc = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int dt = 0; dt < kDt; ++dt) o_acc[nt][dt][0] = o_acc[nt][dt][1] = o_acc[nt][dt][2] = o_acc[nt][dt][3] = 0.f;
#pragma unroll
      for (int w = 0; w < kG; ++w) corr_acc[nt][w][0] = corr_acc[nt][w][1] = 0.f;
      m_run[nt][0] = m_run[nt][1] = -INFINITY;
      l_run[nt][0] = l_run[nt][1] = 0.f;
    }
  };
  // Query fragments in fp16, each head scaled by a power of two so that its
  // largest element is in [2^13, 2^14): exact but for elements below 2^-26 of
  // that one.  Elements that meet codes in bits 6-9 carry another 2^-4.
  // (2^e of a head's largest element, e up to 127, is taken back by frag_c, the
  // 2^9 left of the codes' 2^22 by kUnscale: together they would pass fp32.)
  auto load_q = [&](const unsigned char* qsm) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = nt * 8 + gq;
      uint4 u[kG];
      uint32_t top = 0;
#pragma unroll
      for (int w = 0; w < kG; ++w) {
        u[w] = h < a.g ? *reinterpret_cast<const uint4*>(qsm + (h * D + 32 * w + 8 * cq) * 2) : make_uint4(0, 0, 0, 0);
        const uint32_t x[4] = {u[w].x, u[w].y, u[w].z, u[w].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, max((x[i] << 16) & 0x7FFFFFFFu, x[i] & 0x7FFF0000u));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = max(-100, min(127, static_cast<int>(top >> 23) - 127));
      const float f = pow2(13 - e);
#pragma unroll
      for (int w = 0; w < kG; ++w) {
        const uint32_t x[4] = {u[w].x, u[w].y, u[w].z, u[w].w};
        float v[8], sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] = __uint_as_float(x[i] << 16) * f;
          v[2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u) * f;
        }
        // in the order of the code pairs: nibbles (i, i + 4)
        uint32_t qb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float k = i % 2 ? 0.0625f : 1.f;
          qb[i] = half2_bits(v[i] * k, v[i + 4] * k);
          const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&qb[i]));
          sum = fmaf(y.x + y.y, i % 2 ? 16.f : 1.f, sum);
        }
        frag_q[(nt * kG + w) * 32] = make_uint4(qb[0], qb[1], qb[2], qb[3]);
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sum *= -8.f * 0x1p-22f;
        // to the threads that hold heads 2 cq and 2 cq + 1 of a product
        const float q0 = __shfl_sync(0xffffffffu, sum, 8 * cq), q1 = __shfl_sync(0xffffffffu, sum, 8 * cq + 4);
        frag_s[(nt * kG + w) * 32] = make_float2(q0, q1);
      }
      const float back = pow2(e) * a.scale2;
      const float b0 = __shfl_sync(0xffffffffu, back, 8 * cq), b1 = __shfl_sync(0xffffffffu, back, 8 * cq + 4);
      frag_c[nt * 32] = make_float2(b0, b1);
    }
  };
  auto write_out = [&](size_t row, int d4, float4 acc, float M, float L) {
    const float inv = 1.f / L;
    const __nv_bfloat162 x = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), y = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(a.out + row * D + 4 * d4) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    if (a.lse && d4 == 0) a.lse[row] = (M - kBoost + log2f(L)) * 0.6931471805599453f;
  };
  auto part_of = [&](int c, bool at_start) {
    return a.parts + static_cast<size_t>(2 * c + (at_start ? 0 : 1)) * a.g * (D + 4);
  };
  // Leaving a lane: the warps' sums joined; four elements of a head a thread.
  auto finish = [&](int l, bool whole, bool at_start) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float s = l_run[nt][e];
        s += __shfl_xor_sync(0xffffffffu, s, 4);
        s += __shfl_xor_sync(0xffffffffu, s, 8);
        s += __shfl_xor_sync(0xffffffffu, s, 16);
        const int h = nt * 8 + cq * 2 + e;
        if (gq == 0) {
          sh_ml[warp][h][0] = m_run[nt][e];
          sh_ml[warp][h][1] = s;
        }
        float* po = sh_o + (warp * C::kHeads + h) * C::kOStride;
#pragma unroll
        for (int w = 0; w < kG; ++w) {
          const float off = 8.f * corr_acc[nt][w][e];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int dt = 2 * w + i;
            po[dt * 16 + gq] = fmaf(o_acc[nt][dt][e], 0x1p22f, -off);
            po[dt * 16 + gq + 8] = fmaf(o_acc[nt][dt][2 + e], 0x1p18f, -off);
          }
        }
      }
    }
    sync_consumers();
    const size_t row = static_cast<size_t>(l / a.Hkv) * a.Hq + static_cast<size_t>(l % a.Hkv) * a.g;
    for (int it = tid; it < a.g * (D / 4); it += W * 32) {
      const int h = it / (D / 4), d4 = it % (D / 4);
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < W; ++w) M = fmaxf(M, sh_ml[w][h][0]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float L = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float mw = sh_ml[w][h][0];
        // a warp without a page has zero sums; one of NaN alone has no maximum
        const float f = mw == -INFINITY ? 1.f : hw_exp2(mw - M);
        const float4 v = *reinterpret_cast<const float4*>(sh_o + (w * C::kHeads + h) * C::kOStride + 4 * d4);
        L = fmaf(sh_ml[w][h][1], f, L);
        acc.x = fmaf(v.x, f, acc.x);
        acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z);
        acc.w = fmaf(v.w, f, acc.w);
      }
      if (whole) {
        write_out(row + h, d4, acc, M, L);
      } else {
        float4* ph = reinterpret_cast<float4*>(part_of(blockIdx.x, at_start) + static_cast<size_t>(h) * (D + 4));
        __stcg(ph + d4, acc);
        if (d4 == 0) __stcg(ph + D / 4, make_float4(M, L, 0.f, 0.f));
      }
    }
    sync_consumers();
  };
  auto cta_of = [&](int r) { return static_cast<int>(((static_cast<long long>(r) + 1) * G - 1) / R); };

  // --- the CTA's rounds -------------------------------------------------------------
  int cur = first_lane - 1, lane_begin = 0, lane_end = r_begin, seg_begin = r_begin, used = 0, q_no = 0;
  int part_lane[2] = {-1, -1};       // lanes this CTA has a part of: at its start, at its end
  bool alive = true;
  Seen sn = {};
  auto leave = [&](int r) {
    const bool whole = seg_begin == lane_begin && r == lane_end;
    const bool at_start = seg_begin == r_begin;
    finish(cur, whole, at_start);
    if (!whole) part_lane[at_start ? 0 : 1] = cur;
  };
  for (int r = r_begin; r < r_end; ++r) {
    if (r >= lane_end) {
      if (r > r_begin) leave(r);
      ++cur;
      while (sh_prefix[cur + 1] <= r) ++cur;
      lane_begin = sh_prefix[cur];
      lane_end = sh_prefix[cur + 1];
      seg_begin = r;
      sn = seen_of(sh_len[cur], a.sinks, a.window);
      const int slot = q_no % C::kQSlots;
      if (warp == 0) {
        // (every warp has left the last lane, whose fragments these replace)
        if (alive) alive = mbar_wait_bounded(&sh_qfull[slot], (q_no / C::kQSlots) & 1, a.status);
        load_q(smem + C::kQOff + slot * C::kQBytes);
        __syncwarp();
        if (lane_id == 0) mbar_arrive(&sh_qempty[slot]);
      }
      sync_consumers();
      ++q_no;
      reset_acc();
    }
    const int k = ((r - lane_begin) * W + warp) * NP;
    if (k >= sn.pages) continue;
    int i0[NP];
    bool full = k + NP <= sn.pages;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      // (a page past the last one has tokens past n)
      i0[p] = k + p >= sn.pages ? sn.n : (k + p < sn.pa ? k + p : sn.pb + (k + p - sn.pa)) * 16;
      full = full && i0[p] + 16 <= sn.n && (i0[p] + 16 <= sn.first || i0[p] >= sn.near);
    }
    const int st = used % S;
    if (alive) alive = mbar_wait_bounded(&sh_full[warp][st], (used / S) & 1, a.status);
    ++used;
    const unsigned char* pg0 = smem + (warp * S + st) * C::kStageBytes;

    // S^T = K Q^T, a group of 32 elements of all pages at a time
    float z[NP][NT][4];
    {
      uint32_t ka[NP][kG], kb[NP][kG], sa[NP][kG / 2], sb[NP][kG / 2];
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const unsigned char* pg = pg0 + p * P::kBytes;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) z[p][nt][0] = z[p][nt][1] = z[p][nt][2] = z[p][nt][3] = 0.f;
        const unsigned char* k0 = pg + gq * P::kRow + cq * (4 * kG);
        const unsigned char* s0 = pg + P::kKScale + gq * (2 * kG);
        if constexpr (kG == 4) {
          const uint4 x = *reinterpret_cast<const uint4*>(k0), y = *reinterpret_cast<const uint4*>(k0 + 8 * P::kRow);
          ka[p][0] = x.x; ka[p][1] = x.y; ka[p][2] = x.z; ka[p][3] = x.w;
          kb[p][0] = y.x; kb[p][1] = y.y; kb[p][2] = y.z; kb[p][3] = y.w;
          const uint2 u = *reinterpret_cast<const uint2*>(s0), t = *reinterpret_cast<const uint2*>(s0 + 16 * kG);
          sa[p][0] = u.x; sa[p][1] = u.y;
          sb[p][0] = t.x; sb[p][1] = t.y;
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(k0), y = *reinterpret_cast<const uint2*>(k0 + 8 * P::kRow);
          ka[p][0] = x.x; ka[p][1] = x.y;
          kb[p][0] = y.x; kb[p][1] = y.y;
          sa[p][0] = *reinterpret_cast<const uint32_t*>(s0);
          sb[p][0] = *reinterpret_cast<const uint32_t*>(s0 + 16 * kG);
        }
      }
#pragma unroll
      for (int w = 0; w < kG; ++w) {
        uint4 qf[NT];
        float2 qs[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          qf[nt] = frag_q[(nt * kG + w) * 32];
          qs[nt] = frag_s[(nt * kG + w) * 32];
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const float ks0 = __uint_as_float((w & 1) ? sa[p][w / 2] & 0xFFFF0000u : sa[p][w / 2] << 16);
          const float ks1 = __uint_as_float((w & 1) ? sb[p][w / 2] & 0xFFFF0000u : sb[p][w / 2] << 16);
          uint32_t x[4], y[4];
          code_pairs(ka[p][w], x);
          code_pairs(kb[p][w], y);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float t[4];
            mma_f16(t, x[0], y[0], x[1], y[1], qf[nt].x, qf[nt].y, qs[nt].x, qs[nt].y, qs[nt].x, qs[nt].y);
            mma_f16(t, x[2], y[2], x[3], y[3], qf[nt].z, qf[nt].w, t[0], t[1], t[2], t[3]);
            z[p][nt][0] = fmaf(ks0, t[0], z[p][nt][0]);
            z[p][nt][1] = fmaf(ks0, t[1], z[p][nt][1]);
            z[p][nt][2] = fmaf(ks1, t[2], z[p][nt][2]);
            z[p][nt][3] = fmaf(ks1, t[3], z[p][nt][3]);
          }
        }
      }
    }
    // weights
    float g0[NP], g1[NP];                       // 2^-e of tokens gq and gq + 8
    uint32_t mask[NP][2];                       // tokens 2 cq, 2 cq + 1 and 8 further: what hidden ones hold may be NaN
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int8_t* ep = reinterpret_cast<const int8_t*>(pg0 + p * P::kBytes + P::kVExp);
      int e0 = ep[gq], e1 = ep[gq + 8];
      bool ok0 = true, ok1 = true;
      mask[p][0] = mask[p][1] = 0xFFFFFFFFu;
      if (!full) {
        auto ok = [&](int t) {
          const int i = i0[p] + t;
          return i < sn.n && (i < sn.first || i >= sn.near);
        };
        ok0 = ok(gq);
        ok1 = ok(gq + 8);
        e0 = ok0 ? e0 : 0;
        e1 = ok1 ? e1 : 0;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          mask[p][i] = (ok(2 * cq + 8 * i) ? 0xFFFFu : 0u) | (ok(2 * cq + 1 + 8 * i) ? 0xFFFF0000u : 0u);
      }
      const float f0 = static_cast<float>(e0), f1 = static_cast<float>(e1);
      g0[p] = pow2(-e0);
      g1[p] = pow2(-e1);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float2 ch = frag_c[nt * 32];
#pragma unroll
        for (int e = 0; e < 4; ++e) z[p][nt][e] = fmaf(z[p][nt][e] * kUnscale, e & 1 ? ch.y : ch.x, e < 2 ? f0 : f1);
        if (!full) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!(e < 2 ? ok0 : ok1)) z[p][nt][e] = -INFINITY;
        }
      }
    }
    uint32_t bt[NP][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float top[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        top[e] = fmaxf(z[0][nt][e], z[0][nt][2 + e]);
#pragma unroll
        for (int p = 1; p < NP; ++p) top[e] = fmaxf(top[e], fmaxf(z[p][nt][e], z[p][nt][2 + e]));
      }
      if (__any_sync(0xffffffffu, top[0] > m_run[nt][0] + kGrow || top[1] > m_run[nt][1] + kGrow)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = top[e];
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
          const float mo = m_run[nt][e], mn = fmaxf(mo, t);
          const float c = mo == -INFINITY ? 0.f : hw_exp2(mo - mn);
          m_run[nt][e] = mn;
          l_run[nt][e] *= c;
#pragma unroll
          for (int w = 0; w < kG; ++w) corr_acc[nt][w][e] *= c;
#pragma unroll
          for (int dt = 0; dt < kDt; ++dt) {
            o_acc[nt][dt][e] *= c;
            o_acc[nt][dt][2 + e] *= c;
          }
        }
      }
      const float m0 = m_run[nt][0] - kBoost, m1 = m_run[nt][1] - kBoost;
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        float u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = hw_exp2(z[p][nt][e] - (e & 1 ? m1 : m0));
        l_run[nt][0] = fmaf(u[0], g0[p], fmaf(u[2], g1[p], l_run[nt][0]));
        l_run[nt][1] = fmaf(u[1], g0[p], fmaf(u[3], g1[p], l_run[nt][1]));
        bt[p][nt][0] = transpose8x8(half2_bits(u[0], u[1]));
        bt[p][nt][1] = transpose8x8(half2_bits(u[2], u[3]));
      }
    }
    // O^T += V^T (P vs)^T, a group of 32 elements at a time
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const unsigned char* pg = pg0 + p * P::kBytes;
      uint32_t vw[kDt];
#pragma unroll
      for (int i = 0; i < kDt / 4; ++i) {
        const uint4 x = *reinterpret_cast<const uint4*>(pg + P::kV + i * 512 + lane_id * 16);
        vw[4 * i] = x.x; vw[4 * i + 1] = x.y; vw[4 * i + 2] = x.z; vw[4 * i + 3] = x.w;
      }
      uint2 ratio[kG];
#pragma unroll
      for (int w = 0; w < kG; ++w) ratio[w] = reinterpret_cast<const uint2*>(pg + P::kVRatio + cq * (8 * kG))[w];
      if (!full) {
#pragma unroll
        for (int w = 0; w < kG; ++w) {
          ratio[w].x &= mask[p][0];
          ratio[w].y &= mask[p][1];
        }
      }
      if (p == NP - 1) {
        // the tile has been read: its stage may be filled again
        __syncwarp();
        if (lane_id == 0) mbar_arrive(&sh_empty[warp][st]);
      }
#pragma unroll
      for (int w = 0; w < kG; ++w) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t b0 = half2_mul(bt[p][nt][0], ratio[w].x), b1 = half2_mul(bt[p][nt][1], ratio[w].y);
          // every row of the product is the sum (one accumulator a group: a
          // group of NaN must not reach the others)
          float c[4];
          mma_f16(c, 0x3C003C00u, 0u, 0x3C003C00u, 0u, b0, b1, corr_acc[nt][w][0], corr_acc[nt][w][1], 0.f, 0.f);
          corr_acc[nt][w][0] = c[0];
          corr_acc[nt][w][1] = c[1];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t x[4];
            code_pairs(vw[2 * w + i], x);
            float* o = o_acc[nt][2 * w + i];
            mma_f16(o, x[0], x[1], x[2], x[3], b0, b1, o[0], o[1], o[2], o[3]);
          }
        }
      }
    }
  }
  leave(r_end);

  // --- parts of lanes: the last to arrive joins them ------------------------------
  if (part_lane[0] < 0 && part_lane[1] < 0) return;
  __threadfence();
  sync_consumers();
  if (tid < 2) {
    const int l = part_lane[tid];
    int last = 0;
    if (l >= 0) {
      const int others = cta_of(sh_prefix[l + 1] - 1) - cta_of(sh_prefix[l]);
      last = atomicAdd(a.arrived + l, 1) == others;
      if (last) a.arrived[l] = 0;
      __threadfence();
    }
    sh_scan[tid] = last;
  }
  sync_consumers();
  for (int i = 0; i < 2; ++i) {
    if (!sh_scan[i]) continue;
    const int l = part_lane[i];
    const int c0 = cta_of(sh_prefix[l]), c1 = cta_of(sh_prefix[l + 1] - 1);
    const bool first_at_start = static_cast<int>(R * c0 / G) == sh_prefix[l];
    const size_t row = static_cast<size_t>(l / a.Hkv) * a.Hq + static_cast<size_t>(l % a.Hkv) * a.g;
    // a warp per head: the parts' maximum, their factors and the sum of weights
    for (int h = warp; h < a.g; h += W) {
      float M = -INFINITY, L = 0.f;
      for (int c = c0 + lane_id; c <= c1; c += 32) {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(part_of(c, c > c0 || first_at_start) + h * (D + 4) + D));
        M = fmaxf(M, x.x);
      }
      M = warp_max(M);
      for (int c = c0 + lane_id; c <= c1; c += 32) {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(part_of(c, c > c0 || first_at_start) + h * (D + 4) + D));
        const float f = x.x == -INFINITY ? 1.f : hw_exp2(x.x - M);
        sh_o[(c - c0) * C::kHeads + h] = f;
        L = fmaf(x.y, f, L);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
      if (lane_id == 0) {
        sh_ml[0][h][0] = M;
        sh_ml[0][h][1] = L;
      }
    }
    sync_consumers();
    for (int it = tid; it < a.g * (D / 4); it += W * 32) {
      const int h = it / (D / 4), d4 = it % (D / 4);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
      for (int c = c0; c <= c1; ++c) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(part_of(c, c > c0 || first_at_start) + h * (D + 4)) + d4);
        const float f = sh_o[(c - c0) * C::kHeads + h];
        acc.x = fmaf(v.x, f, acc.x);
        acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z);
        acc.w = fmaf(v.w, f, acc.w);
      }
      write_out(row + h, d4, acc, sh_ml[0][h][0], sh_ml[0][h][1]);
    }
    sync_consumers();
  }
}

template <int D, int NT>
cudaError_t set_smem() {
  return cudaFuncSetAttribute(kv4_attend_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Kv4Cfg<D, NT>::smem_for(1024));
}

}  // namespace

// [lanes] counters, then two parts a CTA of g rows of d sums, a maximum, a sum and two unused
size_t kv4_scratch_bytes(const Dims& dm) {
  const size_t counters = (static_cast<size_t>(dm.lanes) * 4 + 15) / 16 * 16;
  return counters + static_cast<size_t>(2 * kMaxCtas) * dm.g * (dm.d + 4) * 4;
}

cudaError_t prepare_kv4() {
  cudaError_t e = set_smem<128, 1>();
  if (e == cudaSuccess) e = set_smem<128, 2>();
  if (e == cudaSuccess) e = set_smem<64, 1>();
  if (e == cudaSuccess) e = set_smem<64, 2>();
  return e;
}

cudaError_t launch_kv4_attend(const Ctx& ctx, const kvevict_kv4& c, const int32_t* lens, const void* q, int sinks,
                              int window, void* out, float* lse, cudaStream_t st) {
  const Dims& dm = ctx.dims;
  Kv4Attend a;
  a.pages = static_cast<const unsigned char*>(c.pages);
  a.table = c.table; a.num_pages = c.num_pages; a.max_pages = c.max_pages;
  a.lens = lens;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse; a.status = ctx.ws.status;
  a.arrived = static_cast<int32_t*>(c.scratch);
  a.parts = reinterpret_cast<float*>(static_cast<char*>(c.scratch) + (static_cast<size_t>(dm.lanes) * 4 + 15) / 16 * 16);
  a.lanes = dm.lanes; a.g = dm.g; a.Hkv = dm.Hkv; a.Hq = dm.Hq; a.sinks = sinks; a.window = window;
  a.scale2 = 1.4426950408889634f / sqrtf(static_cast<float>(dm.d));
  const int grid = ctx.sm_count < kMaxCtas ? ctx.sm_count : kMaxCtas;
  const bool two = dm.g > 8;
  if (dm.d == 128) {
    if (two) return launch_k(kv4_attend_kernel<128, 2>, dim3(grid), dim3(Kv4Cfg<128, 2>::kThreads),
                              Kv4Cfg<128, 2>::smem_for(dm.lanes), st, false, a);
    return launch_k(kv4_attend_kernel<128, 1>, dim3(grid), dim3(Kv4Cfg<128, 1>::kThreads),
                              Kv4Cfg<128, 1>::smem_for(dm.lanes), st, false, a);
  }
  if (two) return launch_k(kv4_attend_kernel<64, 2>, dim3(grid), dim3(Kv4Cfg<64, 2>::kThreads),
                              Kv4Cfg<64, 2>::smem_for(dm.lanes), st, false, a);
  return launch_k(kv4_attend_kernel<64, 1>, dim3(grid), dim3(Kv4Cfg<64, 1>::kThreads),
                              Kv4Cfg<64, 1>::smem_for(dm.lanes), st, false, a);
}

}  // namespace kve
