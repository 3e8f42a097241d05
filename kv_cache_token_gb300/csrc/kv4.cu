// The 4-bit cache of kept tokens: storing rows (kvevict_kv4_write,
// kvevict_kv4_pack) and reading their values back (kvevict_kv4_read).
//
// A page belongs to one CTA: the tokens of one call that fall into a page are
// coded together, because a word of V codes holds nibbles of four tokens and
// has to be merged by a single owner.  A thread codes eight elements (one
// 16-byte load, one word of codes); the four threads of a group and the d / 8
// threads of a row are neighbours in a warp, so the group's largest magnitude
// and the row's largest scale are shuffles.
//
// Storing is bound by instructions (about 160 for eight elements of a warp, 75%
// of the issue slots; the four threads of a group each work out its scale,
// reciprocal and ratio): 32768 tokens of 8 lanes, d = 128, 172 MB, in 47 us, 3.7
// TB/s; 3276 kept tokens of 128 lanes packed, 274 MB, in 80 us.  Reading back is
// bound by memory: the same tokens in 32 us, 5.4 TB/s, and 48 us, 5.7 TB/s.
#include "kv4_page.cuh"
#include "kvevict_internal.cuh"
#include "packed_math.cuh"

namespace kve {

namespace {

constexpr int kKv4Threads = 256;

struct Kv4Store {
  unsigned char* pages;
  const int32_t* table;
  int num_pages, max_pages;
  // source: rows [lanes][n][d], or a layer's pools through its tables
  const __nv_bfloat16* k; const __nv_bfloat16* v;
  const int32_t* starts;      // null: 0
  const int32_t* slot;        // pack: the layer's slots [lanes][cap] and counts
  const int32_t* count;
  int cap, pool_rows;
  int n;
  uint32_t* status;
};

// x / scale from a reciprocal within an ulp: Markstein's correction of the
// product by its exact residual.  A quotient that is a number of fp32 comes out
// exactly (the correction's own error is far below half an ulp), and any other
// within two ulps, so rounding it to an integer rounds x / scale: of bf16 numbers
// the quotient is a tie of two integers exactly or off it by more than 2^-10.
__device__ __forceinline__ float div_rn(float x, float scale, float rcp) {
  const float q = x * rcp;
  return fmaf(fmaf(-q, scale, x), rcp, q);
}

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); }
__device__ __forceinline__ __nv_bfloat162 max_abs(__nv_bfloat162 a, __nv_bfloat162 b) { return __hmax2_nan(a, b); }

// grid (groups of `per` pages a lane can touch, lanes).  The rows of the next
// page are loaded while one is coded.
// (Five CTAs a SM: 48 registers.  Left to itself the compiler took 55 for the
// pack in one arrangement, four CTAs: 133 us for 3276 tokens x 128 lanes packed
// and read, against 127; with six, 128.)
template <int D, bool kPack>
__global__ void __launch_bounds__(kKv4Threads, 5) kv4_store_kernel(Kv4Store a, int per) {
  using P = Kv4Page<D>;
  constexpr int kChunks = D / 8;                          // 16-byte pieces of a row
  constexpr int kItems = 2 * 16 * kChunks / kKv4Threads;  // pieces a thread codes of a page
  constexpr int kVStride = D + 16;
  static_assert(kItems <= 2, "K pieces, then V pieces");
  const int l = blockIdx.y, tid = threadIdx.x;
  int start = 0, n = a.n;
  if (kPack) {
    n = a.count[l];
    if (n < 0 || n > a.cap) {
      if (tid == 0) set_status(a.status, ST_BAD_INDEX);
      return;
    }
  } else if (a.starts) {
    start = a.starts[l];
  }
  if (start < 0 || static_cast<long long>(start) + n > static_cast<long long>(a.max_pages) * 16) {
    if (tid == 0) set_status(a.status, ST_CAPACITY);
    return;
  }
  const int end = start + n;
  const int p_begin = start / 16 + blockIdx.x * per;
  const int p_end = min(p_begin + per, (end + 15) / 16);
  if (p_begin >= p_end) return;
  __shared__ __align__(16) uint8_t sh_v[2][16 * kVStride];       // V codes by token
  // piece i of this thread: K pieces of the page first, then V pieces
  auto load = [&](int pi, uint4 (&u)[kItems]) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const bool isv = kItems == 2 ? i == 1 : tid >= 16 * kChunks;
      const int rem = tid % (16 * kChunks);
      const int t = pi * 16 + rem / kChunks;
      u[i] = make_uint4(0, 0, 0, 0);
      if (t >= start && t < end) {
        size_t row;
        bool there = true;
        if (kPack) {
          const int s = a.slot[static_cast<size_t>(l) * a.cap + t];
          there = s >= 0 && s < a.pool_rows;
          row = s;
        } else {
          row = static_cast<size_t>(l) * a.n + (t - start);
        }
        if (there) {
          u[i] = *reinterpret_cast<const uint4*>((isv ? a.v : a.k) + row * D + (rem % kChunks) * 8);
        } else {      // no such row: the token holds NaN, not another's values
          set_status(a.status, ST_BAD_INDEX);
          u[i] = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
        }
      }
    }
  };
  uint4 next[kItems];
  const int32_t* table = a.table + static_cast<size_t>(l) * a.max_pages;
  int next_id = table[p_begin];
  load(p_begin, next);
  for (int pi = p_begin; pi < p_end; ++pi) {
    uint4 u[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) u[i] = next[i];
    const int id = next_id;
    if (pi + 1 < p_end) {
      next_id = table[pi + 1];
      load(pi + 1, next);
    }
    if (id < 0 || id >= a.num_pages) {
      if (tid == 0) set_status(a.status, ST_BAD_INDEX);
      __syncthreads();      // the page after this one takes the buffer of the one before
      continue;
    }
    unsigned char* page = a.pages + static_cast<size_t>(id) * P::kBytes;
    const int lo = max(start - pi * 16, 0), hi = min(end - pi * 16, 16);   // this call's tokens of the page
    uint8_t* codes = sh_v[pi & 1];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const bool isv = kItems == 2 ? i == 1 : tid >= 16 * kChunks;
      const int rem = tid % (16 * kChunks);
      const int t = rem / kChunks, ch = rem % kChunks;
      const bool mine = t >= lo && t < hi;
      const uint32_t uw[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
      // the largest magnitude of the group, NaN if there is one
      __nv_bfloat162 top2 = max_abs(max_abs(as_bf162(uw[0] & 0x7FFF7FFFu), as_bf162(uw[1] & 0x7FFF7FFFu)),
                                    max_abs(as_bf162(uw[2] & 0x7FFF7FFFu), as_bf162(uw[3] & 0x7FFF7FFFu)));
      top2 = max_abs(top2, __shfl_xor_sync(0xffffffffu, top2, 1));
      top2 = max_abs(top2, __shfl_xor_sync(0xffffffffu, top2, 2));
      const float top = __bfloat162float(__hmax_nan(__low2bfloat16(top2), __high2bfloat16(top2)));
      const bool far = !(top >= 0x1p-64f && top < 0x1p64f);      // zero, tiny, or not to be held
      const __nv_bfloat16 sb = __float2bfloat16_rn(far ? top / 7.0f : div_rn(top, 7.0f, 1.0f / 7.0f));
      float scale = __bfloat162float(sb);
      const bool bad = !(scale < 0x1p63f);
      const int w = ch >> 2, c = ch & 3;
      bool slow = far;
      if (!isv) {
        if (mine && c == 0) {
          reinterpret_cast<__nv_bfloat16*>(page + P::kKScale)[t * P::kG + w] =
              bad ? __float2bfloat16_rn(__int_as_float(0x7FC00000)) : sb;
        }
      } else {
        // one exponent per token: that of its largest scale
        float m = bad ? 0.f : scale;
#pragma unroll
        for (int o = 4; o < kChunks; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        int e = static_cast<int>(__float_as_uint(m) >> 23) - 127;
        e = max(P::kExpMin, min(P::kExpMax, e));
        const float up = __int_as_float((e + 127) << 23), down = __int_as_float((127 - e) << 23);   // 2^e, 2^-e
        const __half r = bad ? __float2half_rn(__int_as_float(0x7FC00000)) : __float2half_rn(scale * down);
        slow = slow || !(scale * down >= 0x1p-14f);              // the ratio may have been rounded
        scale = __half2float(r) * up;
        if (mine && c == 0) reinterpret_cast<__half*>(page + P::kVRatio)[P::v_ratio(t, w)] = r;
        if (mine && ch == 0) reinterpret_cast<int8_t*>(page + P::kVExp)[t] = static_cast<int8_t>(e);
      }
      // Codes: x / scale to the nearest integer (ties to even) by adding
      // 1.5 2^23 + 8, which leaves code + 8 in the low bits.
      // |x / scale| is at most 7 / (1 - 2^-8) < 7.5 here, so no clamp.
      uint32_t code[8];
      if (!slow) {
        float rcp;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rcp) : "f"(scale));
        const float2 rc = make_float2(rcp, rcp), ns = make_float2(-scale, -scale), magic = make_float2(12582920.f, 12582920.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = make_float2(__uint_as_float(uw[j] << 16), __uint_as_float(uw[j] & 0xFFFF0000u));
          const float2 q = f2_mul(x, rc);
          const float2 y = f2_add(f2_fma(f2_fma(q, ns, x), rc, q), magic);
          code[2 * j] = __float_as_uint(y.x);
          code[2 * j + 1] = __float_as_uint(y.y);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float x = __uint_as_float(j & 1 ? uw[j / 2] & 0xFFFF0000u : uw[j / 2] << 16);
          float f = !bad && scale > 0.f ? rintf(__fdiv_rn(x, scale)) : 0.f;
          f = fminf(7.f, fmaxf(-7.f, f));
          code[j] = __float_as_uint(f + 12582920.f);
        }
      }
      // the words of low nibbles and of low bytes (what the nibbles' upper
      // neighbours add is a constant, taken off again)
      constexpr uint32_t kHigh = 0x4B400000u;
      uint32_t word = 0;
#pragma unroll
      for (int j = 7; j >= 0; --j) word = word * 16u + code[j];
      word -= kHigh * 0x11111111u;
      const uint32_t vlo = __byte_perm(__byte_perm(code[0], code[1], 0x0040), __byte_perm(code[2], code[3], 0x0040), 0x5410);
      const uint32_t vhi = __byte_perm(__byte_perm(code[4], code[5], 0x0040), __byte_perm(code[6], code[7], 0x0040), 0x5410);
      if (!isv) {
        if (mine) reinterpret_cast<uint32_t*>(page)[t * (P::kRow / 4) + c * P::kG + w] = P::pack(word);
      } else {
        *reinterpret_cast<uint2*>(codes + t * kVStride + ch * 8) = make_uint2(vlo, vhi);
      }
    }
    __syncthreads();
    // V words: the nibbles of this call's tokens replaced.  One warp does a
    // page's, the warps in turn.  (The next page's codes go to the other
    // buffer, so one barrier a page is enough.)  Thread (dt, cq) has elements
    // 16 dt .. + 15 of tokens 2 cq, 2 cq + 8, 2 cq + 1, 2 cq + 9: byte k of the
    // word of gq is the pair of codes (gq, gq + 8) of the k-th of them.
    const int lane = tid & 31, dt = lane >> 2, cq = lane & 3;
    if ((tid >> 5) == (pi & (kKv4Threads / 32 - 1)) && dt < D / 16) {
      uint32_t pair[4][2], mask = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int t = 2 * cq + (k >> 1) + (k & 1) * 8;
        const uint4 x = *reinterpret_cast<const uint4*>(codes + t * kVStride + dt * 16);
        pair[k][0] = x.x | x.z << 4;
        pair[k][1] = x.y | x.w << 4;
        if (t >= lo && t < hi) mask |= 0xFFu << (8 * k);
      }
      uint32_t* vw = reinterpret_cast<uint32_t*>(page + P::kV);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        // a 4 x 4 transpose of bytes
        const uint32_t a0 = __byte_perm(pair[0][x], pair[1][x], 0x5140), a1 = __byte_perm(pair[0][x], pair[1][x], 0x7362);
        const uint32_t b0 = __byte_perm(pair[2][x], pair[3][x], 0x5140), b1 = __byte_perm(pair[2][x], pair[3][x], 0x7362);
        const uint32_t word[4] = {__byte_perm(a0, b0, 0x5410), __byte_perm(a0, b0, 0x7632), __byte_perm(a1, b1, 0x5410),
                                  __byte_perm(a1, b1, 0x7632)};
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t* p = vw + P::v_word(dt, (4 * x + g) * 4 + cq);
          *p = P::pack(mask == 0xFFFFFFFFu ? word[g] : (P::unpack(*p) & ~mask) | (word[g] & mask));
        }
      }
    }
  }
}

struct Kv4Load {
  const unsigned char* pages;
  const int32_t* table;
  int num_pages, max_pages;
  const int32_t* starts; const int32_t* lens;
  int n;
  __nv_bfloat16* k; __nv_bfloat16* v;
  uint32_t* status;
};

// A code pair (nibbles of the halves' low bits) as bf16 numbers times two
// scales: 128 + n and 136 are exact in bf16, as is the difference, and the
// product is rounded once.
__device__ __forceinline__ uint32_t pair_values(uint32_t nibbles, __nv_bfloat162 scale) {
  const __nv_bfloat162 n = as_bf162((nibbles & 0x000F000Fu) | 0x43004300u);
  const __nv_bfloat162 v = __hmul2(__hsub2(n, __float2bfloat162_rn(136.f)), scale);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// grid (groups of warps' pages, lanes): a warp reads out a page through its own
// part of shared memory, so warps wait for nobody.
template <int D>
__global__ void __launch_bounds__(kKv4Threads) kv4_load_kernel(Kv4Load a) {
  using P = Kv4Page<D>;
  constexpr int kChunks = D / 8, kWarps = kKv4Threads / 32;
  constexpr int kPieces = P::kUsed / 16;
  const int l = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int start = a.starts ? a.starts[l] : 0;
  if (start < 0) {
    if (threadIdx.x == 0) set_status(a.status, ST_BAD_INDEX);
    return;
  }
  const long long all = static_cast<long long>(a.max_pages) * 16;
  long long end = min(all, static_cast<long long>(start) + a.n);
  if (a.lens) end = min(end, max(0ll, static_cast<long long>(a.lens[l])));
  const long long pi = start / 16 + static_cast<long long>(blockIdx.x) * kWarps + warp;
  // (bounded before the cast: a start near 2^31 puts pi * 16 past it, and the difference below -2^31)
  const int lo = static_cast<int>(max(start - pi * 16, 0ll));
  const int hi = static_cast<int>(max(0ll, min(end - pi * 16, 16ll)));
  if (lo >= hi) return;
  const int id = a.table[static_cast<size_t>(l) * a.max_pages + pi];
  if (id < 0 || id >= a.num_pages) {
    if (lane == 0) set_status(a.status, ST_BAD_INDEX);
    return;
  }
  __shared__ __align__(16) uint4 sh_page[kWarps][kPieces];
  const uint4* src = reinterpret_cast<const uint4*>(a.pages + static_cast<size_t>(id) * P::kBytes);
#pragma unroll
  for (int i = 0; i < (kPieces + 31) / 32; ++i)
    if (lane + 32 * i < kPieces) sh_page[warp][lane + 32 * i] = src[lane + 32 * i];
  __syncwarp();
  const unsigned char* page = reinterpret_cast<const unsigned char*>(sh_page[warp]);
  const long long row0 = static_cast<long long>(l) * a.n + (pi * 16 - start);      // output row of the page's first token
  // K: eight elements at a time, two rows a pass
#pragma unroll
  for (int i = 0; i < 16 * kChunks / 32; ++i) {
    const int it = lane + 32 * i, t = it / kChunks, ch = it % kChunks, w = ch >> 2, c = ch & 3;
    if (t < lo || t >= hi) continue;
    const uint32_t word = P::unpack(reinterpret_cast<const uint32_t*>(page)[t * (P::kRow / 4) + c * P::kG + w]);
    const __nv_bfloat162 sc = __bfloat162bfloat162(reinterpret_cast<const __nv_bfloat16*>(page + P::kKScale)[t * P::kG + w]);
    uint32_t v[4];      // elements (j, j + 4)
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = pair_values(word >> (4 * j), sc);
    *reinterpret_cast<uint4*>(a.k + (row0 + t) * D + ch * 8) =
        make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410), __byte_perm(v[0], v[1], 0x7632),
                   __byte_perm(v[2], v[3], 0x7632));
  }
  // V: a thread takes the words of tile dt and quad cq, 16 elements of tokens
  // 2 cq, 2 cq + 1 and 8 further
  const int dt = lane >> 2, cq = lane & 3, w = dt >> 1;
  if (dt < D / 16) {
    const uint2 ratio = *reinterpret_cast<const uint2*>(page + P::kVRatio + (cq * P::kG + w) * 8);
    const int8_t* ex = reinterpret_cast<const int8_t*>(page + P::kVExp);
    auto scales = [&](uint32_t r, int t) {      // of tokens t, t + 1: ratio * 2^e has at most 8 bits
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r));
      return __floats2bfloat162_rn(ldexpf(f.x, ex[t]), ldexpf(f.y, ex[t + 1]));
    };
    const __nv_bfloat162 s0 = scales(ratio.x, 2 * cq), s1 = scales(ratio.y, 2 * cq + 8);
    const uint32_t* vw = reinterpret_cast<const uint32_t*>(page + P::kV);
#pragma unroll
    for (int half = 0; half < 2; ++half) {      // elements 16 dt .. + 7, then + 8 .. + 15
      uint32_t x0[8], x1[8];                    // tokens (2 cq, 2 cq + 1), and 8 further, of element gq
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        const uint32_t word = P::unpack(vw[P::v_word(dt, g * 4 + cq)]);
        x0[g] = pair_values(word >> (4 * half), s0);
        x1[g] = pair_values(word >> (4 * half + 8), s1);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int t = 2 * cq + (k & 1) + (k >> 1) * 8;
        if (t < lo || t >= hi) continue;
        const uint32_t* x = k < 2 ? x0 : x1;
        const uint32_t sel = k & 1 ? 0x7632 : 0x5410;
        *reinterpret_cast<uint4*>(a.v + (row0 + t) * D + dt * 16 + half * 8) =
            make_uint4(__byte_perm(x[0], x[1], sel), __byte_perm(x[2], x[3], sel), __byte_perm(x[4], x[5], sel),
                       __byte_perm(x[6], x[7], sel));
      }
    }
  }
}

// Pages of a CTA: enough that the loads of one hide behind the work on the one
// before, as long as the grid still fills the GPU several times over (stored and
// read back, 32768 tokens x 8 lanes: 78 us with four, 95 with one; 1024 tokens x
// 8 lanes: 8.7 us with four, 7.5 with one).
int pages_per_cta(const Ctx& ctx, long long pages) {
  return pages >= 32ll * ctx.sm_count ? 4 : 1;
}

}  // namespace

size_t kv4_page_bytes(int d) { return d == 128 ? Kv4Page<128>::kBytes : Kv4Page<64>::kBytes; }

cudaError_t launch_kv4_write(const Ctx& ctx, const kvevict_kv4& c, const int32_t* starts, int n, const void* k,
                             const void* v, cudaStream_t st) {
  const Dims& dm = ctx.dims;
  Kv4Store a = {};
  a.pages = static_cast<unsigned char*>(c.pages);
  a.table = c.table; a.num_pages = c.num_pages; a.max_pages = c.max_pages;
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.starts = starts; a.n = n; a.status = ctx.ws.status;
  const int most = static_cast<int>((static_cast<long long>(n) + 30) / 16);      // pages that n tokens can touch
  const int per = pages_per_cta(ctx, static_cast<long long>(most) * dm.lanes);
  const dim3 grid((most + per - 1) / per, dm.lanes);
  if (dm.d == 128) kv4_store_kernel<128, false><<<grid, kKv4Threads, 0, st>>>(a, per);
  else kv4_store_kernel<64, false><<<grid, kKv4Threads, 0, st>>>(a, per);
  return cudaGetLastError();
}

cudaError_t launch_kv4_pack(const Ctx& ctx, int layer, const kvevict_kv4& c, cudaStream_t st) {
  const Dims& dm = ctx.dims;
  const LayerState ls = layer_state(ctx, layer);
  Kv4Store a = {};
  a.pages = static_cast<unsigned char*>(c.pages);
  a.table = c.table; a.num_pages = c.num_pages; a.max_pages = c.max_pages;
  a.k = static_cast<const __nv_bfloat16*>(ls.k_pool);
  a.v = static_cast<const __nv_bfloat16*>(ls.v_pool);
  a.slot = ls.slot; a.count = ls.count; a.cap = dm.cap; a.pool_rows = dm.P * kBlock;
  a.status = ctx.ws.status;
  const int table = (dm.cap + 15) / 16, most = table < c.max_pages ? table : c.max_pages;
  const int per = pages_per_cta(ctx, static_cast<long long>(most) * dm.lanes);
  const dim3 grid((most + per - 1) / per, dm.lanes);
  if (dm.d == 128) kv4_store_kernel<128, true><<<grid, kKv4Threads, 0, st>>>(a, per);
  else kv4_store_kernel<64, true><<<grid, kKv4Threads, 0, st>>>(a, per);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Ctx& ctx, const kvevict_kv4& c, const int32_t* starts, const int32_t* lens, int n,
                            void* k, void* v, cudaStream_t st) {
  const Dims& dm = ctx.dims;
  Kv4Load a = {};
  a.pages = static_cast<const unsigned char*>(c.pages);
  a.table = c.table; a.num_pages = c.num_pages; a.max_pages = c.max_pages;
  a.starts = starts; a.lens = lens; a.n = n;
  a.k = static_cast<__nv_bfloat16*>(k);
  a.v = static_cast<__nv_bfloat16*>(v);
  a.status = ctx.ws.status;
  const int most = static_cast<int>((static_cast<long long>(n) + 30) / 16);
  constexpr int kWarps = kKv4Threads / 32;
  const dim3 grid((most + kWarps - 1) / kWarps, dm.lanes);
  if (dm.d == 128) kv4_load_kernel<128><<<grid, kKv4Threads, 0, st>>>(a);
  else kv4_load_kernel<64><<<grid, kKv4Threads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace kve
