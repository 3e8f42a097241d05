// Per-head norm and rotation of a projection row, written in the engine's
// layouts (kvevict_norm_rope).
//
// d / 8 threads hold a head row, two quads of four elements each: thread c has
// quads c and c + r/8 of the rotated part, so half-split pairs (i, i + r/2)
// and neighbouring pairs (2i, 2i + 1) both meet within a thread and only the
// mean of squares crosses threads.  (With one 16-byte chunk a thread and the
// partner fetched by eight shuffles, the shuffles took longer than the memory:
// 269 us where this takes 137.)  The arithmetic is packed, two elements an
// instruction.
//
// Bound by memory: 32768 tokens of 48 heads of 128 (bf16) are read and written
// once, 805 MB, in 137 us: 5.9 TB/s, 0.87 of the measured copy bandwidth.
//
// Angle of pair i at position p: turns = p * f_i mod 1 with
// f_i = base^(-2i/r) / 2 pi held as a 64-bit fraction of a turn, so the low 64
// bits of the product are its remainder (an fp32 product p * w loses 1e-2 rad at
// p = 10^5; what f_i itself is off by is in rope_turns.h).  The remainder's
// distance from the nearest quarter turn, 32 bits of it rounded to fp32, gives
// the angle to 2^-28 turn whatever the position (the whole remainder would keep
// 2^-26).  Sines and cosines are taken once per token and shared by all its heads
// through shared memory.
#include <cstring>

#include "kvevict_internal.cuh"
#include "packed_math.cuh"
#include "rope_turns.h"

namespace kve {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kUnroll = 3;

struct RopeArgs {
  const unsigned char* qkv;
  long long batch_stride, row_stride;   // bytes
  const void* wq; const void* wk;
  const int32_t* pos;
  unsigned char* q; unsigned char* k; unsigned char* v;
  float eps;
  int n, pos0, r, interleaved, Hq, Hkv;
  int tok;             // tokens of a CTA
  uint64_t freq[kRopePairs];   // fractions of a turn per position
};

// Four elements: 8 bytes of bf16, 16 of fp32.
template <typename T>
struct Quad;
template <>
struct Quad<__nv_bfloat16> {
  using V = uint2;
  static __device__ __forceinline__ void unpack(const V& u, float2* x) {
    x[0] = make_float2(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u));
    x[1] = make_float2(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
  }
  static __device__ __forceinline__ V pack(const float2* x) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0].x, x[0].y), b = __floats2bfloat162_rn(x[1].x, x[1].y);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
};
template <>
struct Quad<float> {
  using V = float4;
  static __device__ __forceinline__ void unpack(const V& u, float2* x) {
    x[0] = make_float2(u.x, u.y);
    x[1] = make_float2(u.z, u.w);
  }
  static __device__ __forceinline__ V pack(const float2* x) { return make_float4(x[0].x, x[0].y, x[1].x, x[1].y); }
};

// grid (token groups, head groups, B)
template <typename T, int D, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  using Q = Quad<T>;
  using V = typename Q::V;
  constexpr int kRow = D / 8;                       // threads of a head row
  constexpr int kRows = kRopeThreads / kRow;        // rows in flight
  extern __shared__ __align__(16) float sh_rope[];  // weights of q and k [2][D], cosines and sines [tok][2][r / 2]
  float* sh_cs = sh_rope + 2 * D;
  const int tid = threadIdx.x, b = blockIdx.z;
  const int t0 = blockIdx.x * a.tok;
  const int nt = min(a.tok, a.n - t0);
  const int pairs = a.r / 2;
  for (int e = tid; e < nt * pairs; e += kRopeThreads) {
    const int t = e / pairs, i = e - t * pairs;
    const long long p = a.pos ? a.pos[t0 + t] : static_cast<long long>(a.pos0) + t0 + t;
    const unsigned long long turn = a.freq[i] * static_cast<unsigned long long>(p);
    // the nearest quarter turn, and what is left of it: the signed top half, at
    // most 2^29 (an eighth of a turn), in units of half a turn
    const unsigned quarter = static_cast<unsigned>((turn + (1ull << 61)) >> 62);
    const int rest = static_cast<int>((turn - (static_cast<unsigned long long>(quarter) << 62)) >> 32);
    float s, c;
    sincospif(static_cast<float>(rest) * 0x1p-31f, &s, &c);
    const float cc = quarter & 1 ? s : c, ss = quarter & 1 ? c : s;      // up to sign
    sh_cs[t * a.r + i] = quarter == 1 || quarter == 2 ? -cc : cc;
    sh_cs[t * a.r + pairs + i] = quarter >= 2 ? -ss : ss;
  }
  for (int i = tid; i < D; i += kRopeThreads) {
    if (a.wq) sh_rope[i] = static_cast<float>(static_cast<const T*>(a.wq)[i]);
    if (a.wk) sh_rope[D + i] = static_cast<float>(static_cast<const T*>(a.wk)[i]);
  }
  __syncthreads();
  const int c = tid % kRow;
  const bool turns = c < a.r / 8;
  // this thread's quads
  const int qa = turns ? c : a.r / 8 + c, qb = turns ? c + a.r / 8 : qa + (D - a.r) / 8;
  // its angles: of the pairs (i, i + r/2) of elements 4 c .. 4 c + 3, or of the two pairs of each quad
  const int at0 = kInterleaved ? 2 * qa : 4 * c, at1 = kInterleaved ? 2 * qb : 4 * c + 2;
  const int heads = a.Hq + 2 * a.Hkv, turning = a.Hq + a.Hkv;
  // the threads of a row agree on its head; rows of a warp may differ
  const unsigned who = ((1u << kRow) - 1u) << (tid & 31 & ~(kRow - 1));
  const int step = kRows * gridDim.y;
  for (int h0 = blockIdx.y * kRows + tid / kRow; h0 < heads; h0 += kUnroll * step) {
    // kUnroll heads a thread, token after token; the next token's rows are
    // loaded before this one's are worked on
    const unsigned char* src = a.qkv + b * a.batch_stride + t0 * a.row_stride + static_cast<size_t>(h0) * D * sizeof(T);
    V* dst[kUnroll];
    const float* w[kUnroll];
    V ua[kUnroll], ub[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const int h = h0 + j * step;
      w[j] = nullptr;
      if (h < heads) {
        const V* row = reinterpret_cast<const V*>(src + static_cast<size_t>(j) * step * D * sizeof(T));
        ua[j] = row[qa];
        ub[j] = row[qb];
        const bool is_q = h < a.Hq, is_k = !is_q && h < turning;
        const long long orow = is_q ? static_cast<long long>(b) * a.Hq + h
                                    : static_cast<long long>(b) * a.Hkv + (h - (is_k ? a.Hq : turning));
        unsigned char* base = is_q ? a.q : is_k ? a.k : a.v;
        dst[j] = reinterpret_cast<V*>(base + ((orow * a.n + t0) * D) * static_cast<long long>(sizeof(T)));
        if (is_q && a.wq) w[j] = sh_rope;
        if (is_k && a.wk) w[j] = sh_rope + D;
      }
    }
    for (int t = 0; t < nt; ++t) {
      V xa[kUnroll], xb[kUnroll];
      src += a.row_stride;
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        xa[j] = ua[j];
        xb[j] = ub[j];
        if (t + 1 < nt && h0 + j * step < heads) {
          const V* row = reinterpret_cast<const V*>(src + static_cast<size_t>(j) * step * D * sizeof(T));
          ua[j] = row[qa];
          ub[j] = row[qb];
        }
      }
      float2 c0 = make_float2(1.f, 1.f), c1 = c0, s0 = make_float2(0.f, 0.f), s1 = s0;
      if (turns) {
        const float* at = sh_cs + t * a.r;
        c0 = *reinterpret_cast<const float2*>(at + at0);
        c1 = *reinterpret_cast<const float2*>(at + at1);
        s0 = *reinterpret_cast<const float2*>(at + pairs + at0);
        s1 = *reinterpret_cast<const float2*>(at + pairs + at1);
      }
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int h = h0 + j * step;
        if (h >= heads) break;
        if (h < turning) {
          float2 x[4];
          Q::unpack(xa[j], x);
          Q::unpack(xb[j], x + 2);
          if (w[j]) {
            float2 sq = f2_mul(x[0], x[0]);
            sq = f2_fma(x[1], x[1], sq);
            sq = f2_fma(x[2], x[2], sq);
            sq = f2_fma(x[3], x[3], sq);
            float ss = sq.x + sq.y;
#pragma unroll
            for (int m = kRow / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(who, ss, m);
            // (within 2 ulp; 1 / sqrtf gave fp32 rows no smaller an error, 6.4e-8 against 6.2e-8, and took 5.6 -> 6.0 us)
            const float inv = rsqrtf(ss * (1.f / D) + a.eps);
            const float4 wa = reinterpret_cast<const float4*>(w[j])[qa], wb = reinterpret_cast<const float4*>(w[j])[qb];
            const float2 iv = make_float2(inv, inv);
            x[0] = f2_mul(f2_mul(x[0], iv), make_float2(wa.x, wa.y));
            x[1] = f2_mul(f2_mul(x[1], iv), make_float2(wa.z, wa.w));
            x[2] = f2_mul(f2_mul(x[2], iv), make_float2(wb.x, wb.y));
            x[3] = f2_mul(f2_mul(x[3], iv), make_float2(wb.z, wb.w));
          }
          if (turns) {
            if (kInterleaved) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float cc = i == 0 ? c0.x : i == 1 ? c0.y : i == 2 ? c1.x : c1.y;
                const float ss = i == 0 ? s0.x : i == 1 ? s0.y : i == 2 ? s1.x : s1.y;
                x[i] = f2_fma(x[i], make_float2(cc, cc), f2_mul(make_float2(x[i].y, x[i].x), make_float2(-ss, ss)));
              }
            } else {
              const float2 n0 = make_float2(-s0.x, -s0.y), n1 = make_float2(-s1.x, -s1.y);
              const float2 y0 = f2_fma(x[0], c0, f2_mul(x[2], n0)), y1 = f2_fma(x[1], c1, f2_mul(x[3], n1));
              x[2] = f2_fma(x[2], c0, f2_mul(x[0], s0));
              x[3] = f2_fma(x[3], c1, f2_mul(x[1], s1));
              x[0] = y0;
              x[1] = y1;
            }
          }
          xa[j] = Q::pack(x);
          xb[j] = Q::pack(x + 2);
        }
        dst[j][qa] = xa[j];
        dst[j][qb] = xb[j];
        dst[j] += D / 4;
      }
    }
  }
}

}  // namespace

cudaError_t launch_norm_rope(const Ctx& ctx, const void* qkv, long long batch_stride, long long row_stride, int n,
                             const void* wq, const void* wk, float eps, const int32_t* pos, int pos0, int r,
                             double base, int interleaved, void* q, void* k, void* v, cudaStream_t st) {
  const Dims& dm = ctx.dims;
  const int es = dm.dtype == KVEVICT_BF16 ? 2 : 4;
  RopeArgs a;
  a.qkv = static_cast<const unsigned char*>(qkv);
  a.batch_stride = batch_stride * es;
  a.row_stride = row_stride * es;
  a.wq = wq; a.wk = wk; a.pos = pos;
  a.q = static_cast<unsigned char*>(q);
  a.k = static_cast<unsigned char*>(k);
  a.v = static_cast<unsigned char*>(v);
  a.eps = eps; a.n = n; a.pos0 = pos0; a.r = r; a.interleaved = interleaved;
  a.Hq = dm.Hq; a.Hkv = dm.Hkv;
  memcpy(a.freq, turn_table(base, r), sizeof(a.freq));
  // A CTA takes up to eight tokens, which share its start (angles, norm
  // weights) and overlap loads with work, as long as there are CTAs for two
  // on every SM (32768 tokens: 137 us, against 228 with a token a CTA; 2331
  // tokens in fp32: 5.5 against 12.3).  Few tokens spread their heads over CTAs
  // instead (4 tokens: 2.8 us, against 3.4 with all heads in one CTA).
  const int rows = kRopeThreads / (dm.d / 8), groups = (dm.Hq + 2 * dm.Hkv + rows - 1) / rows;
  const long long tokens = static_cast<long long>(n) * dm.B, fill = 2ll * ctx.sm_count;
  a.tok = tokens >= 8 * fill ? 8 : static_cast<int>((tokens + fill - 1) / fill);
  const int split = tokens >= ctx.sm_count ? 1 : groups;
  const dim3 grid((n + a.tok - 1) / a.tok, split, dm.B);
  const size_t sm = (2 * static_cast<size_t>(dm.d) + static_cast<size_t>(a.tok) * r) * sizeof(float);
  const bool inter = interleaved != 0;
#define KVE_ROPE(T, D)                                                                  \
  (inter ? norm_rope_kernel<T, D, true><<<grid, kRopeThreads, sm, st>>>(a)              \
         : norm_rope_kernel<T, D, false><<<grid, kRopeThreads, sm, st>>>(a))
  if (dm.dtype == KVEVICT_BF16) {
    if (dm.d == 128) KVE_ROPE(__nv_bfloat16, 128);
    else KVE_ROPE(__nv_bfloat16, 64);
  } else {
    if (dm.d == 128) KVE_ROPE(float, 128);
    else KVE_ROPE(float, 64);
  }
#undef KVE_ROPE
  return cudaGetLastError();
}

}  // namespace kve
