// gemm_int8.cu -- linear layers in 8-bit integers for sm_100a: activations quantized with a scale for
// each row (token), weights with a scale for each row (output channel), products summed exactly in
// int32 on the tensor cores (tcgen05 kind::i8):
//   s[m]    = amax_k |x[m, k]| / 127 (1 for a row of zeros),  c[m, k] = rint(127 x[m, k] / amax)
//   y[m, n] = (sum_k c[m, k] w8[n, k]) * s[m] * s_w[n] (+ bias[n])
//
//   k_quant_int8_rows  the per-row quantize, one read of x (a row stays in registers)
//   k_gemm_int8_one    one or two tokens: dp4a on streamed weights, with the quantize inside
//   k_gemm_int8_few    up to 64 tokens: weight rows are the MMA's M, tokens its N, K is split over a cluster
//                      whose partial sums meet in shared memory
//   k_gemm_int8_pair   otherwise: 256 x BN output tiles on pairs of SMs (cta_group::2)
// The sums are exact, so every path gives the same bits.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "device_once.h"
#include "launch.h"
#include "quant_math.cuh"
#include "sm100_ptx.cuh"
#include "tensor_map.h"

namespace qattn {

template <bool FP16>
__device__ __forceinline__ uint16_t to16(float v) {
  if (FP16) return __half_as_ushort(__float2half_rn(v));
  return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
// Two at once: one conversion instruction for both, on another unit than the single one's.
template <bool FP16>
__device__ __forceinline__ uint32_t to16x2(float lo, float hi) {
  if (FP16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
template <bool FP16>
__device__ __forceinline__ float from16(uint32_t bits) {
  if (FP16) return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
  return __uint_as_float(bits << 16);
}

// -------------------------------------------------------------------------------------------
// Per-row quantize.  T threads hold a row of up to T * 8 * NV elements in registers between the
// maximum and the codes, so x crosses memory once; longer rows are read a second time (from L2).
// 127 x is exact in FP32 (at most 18 bits) and its quotient by amax is correctly rounded.  A
// quotient of two such numbers is a half integer exactly or is further from one than FP32
// rounding moves it (by 2^-20 of its value or more), so the code is the exact quotient's
// nearest integer, ties to even.  Adding 1.5 * 2^23 rounds to that integer in the low byte.
// A row with a non-finite element gets scale NaN and codes 0 (its outputs become NaN, the other
// rows are unaffected) and records DEV_ERR_NONFINITE.
// -------------------------------------------------------------------------------------------
// Power of two that brings a row's maximum to where 127 x cannot overflow and the quotient's residual
// stays normal (bf16 reaches 2^127 and 2^-133); scaling by it is exact wherever the code is not 0.
__device__ __forceinline__ float scale_pow2(float amax) {
  return amax > 0x1p+100f ? 0x1p-60f : amax < 0x1p-60f ? 0x1p+80f : 1.0f;
}

// How a row's codes are formed: p a power of two (scale_pow2), c = (127 p, 127 p), and for the quotient by
// p * amax its rounded reciprocal and its negative, packed.
struct RowCode {
  f32x2 c, r, na;
};

// Codes of eight elements, two to an instruction until they are packed.
template <bool FP16>
__device__ __forceinline__ uint2 codes8(const uint32_t (&w)[4], const RowCode& k) {
  const f32x2 magic = pack_f32x2(12582912.0f, 12582912.0f);
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2 x = FP16 ? pack_f32x2(from16<true>(w[i] & 0xFFFFu), from16<true>(w[i] >> 16))
                         : pack_f32x2(bf16_lo(w[i]), bf16_hi(w[i]));
    float lo, hi;
    unpack_f32x2(add_f32x2(div_f32x2(mul_f32x2(x, k.c), k.r, k.na), magic), lo, hi);
    h[i] = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x0040);   // low bytes
  }
  return make_uint2(__byte_perm(h[0], h[1], 0x5410), __byte_perm(h[2], h[3], 0x5410));
}

// Scale of a row whose largest magnitude has the bit pattern mx, and how its codes are formed.
struct RowScale {
  float scale;
  bool finite;
  RowCode code;
};
template <bool FP16>
__device__ __forceinline__ RowScale row_scale_of(uint32_t mx) {
  RowScale s;
  s.finite = mx < (FP16 ? 0x7C00u : 0x7F80u);
  float amax = from16<FP16>(mx);
  s.scale = !s.finite ? __int_as_float(0x7FFFFFFF) : mx == 0 ? 1.0f : __fdiv_rn(amax, 127.0f);
  if (mx == 0) amax = 1.0f;
  const float p2 = scale_pow2(amax), c127 = 127.0f * p2;
  amax *= p2;
  const float r = __frcp_rn(amax);
  s.code = {pack_f32x2(c127, c127), pack_f32x2(r, r), pack_f32x2(-amax, -amax)};
  return s;
}

// Eight elements of a row from `at` (a multiple of 8); those past K read as zero.
template <bool VEC>
__device__ __forceinline__ uint4 load8(const uint16_t* row, int at, int K) {
  if (VEC && at + 8 <= K) return __ldg(reinterpret_cast<const uint4*>(row + at));
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (at + j < K) w[j >> 1] |= static_cast<uint32_t>(__ldg(row + at + j)) << (16 * (j & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int T, int NV, bool FP16, bool VEC>
__global__ void __launch_bounds__(256) k_quant_int8_rows(const uint16_t* __restrict__ x, int64_t ldx,
                                                         int M, int K, int8_t* __restrict__ out,
                                                         int64_t ldo, float* __restrict__ scale,
                                                         int* __restrict__ err) {
  constexpr int ROWS = 256 / T, WARPS = T / 32;
  grid_launch_dependents();
  const int sub = threadIdx.x / T, tid = threadIdx.x % T;
  const int m = blockIdx.x * ROWS + sub;
  const uint16_t* row = x + static_cast<int64_t>(m) * ldx;
  uint4 v[NV];
  uint32_t m2 = 0;
  if (m < M) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = (i * T + tid) * 8;
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (at < K) v[i] = load8<VEC>(row, at, K);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      m2 = __vmaxu2(m2, v[i].x & 0x7FFF7FFFu);
      m2 = __vmaxu2(m2, v[i].y & 0x7FFF7FFFu);
      m2 = __vmaxu2(m2, v[i].z & 0x7FFF7FFFu);
      m2 = __vmaxu2(m2, v[i].w & 0x7FFF7FFFu);
    }
    for (int at = (NV * T + tid) * 8; at < K; at += T * 8) {
      const uint4 u = load8<VEC>(row, at, K);
      m2 = __vmaxu2(m2, u.x & 0x7FFF7FFFu);
      m2 = __vmaxu2(m2, u.y & 0x7FFF7FFFu);
      m2 = __vmaxu2(m2, u.z & 0x7FFF7FFFu);
      m2 = __vmaxu2(m2, u.w & 0x7FFF7FFFu);
    }
  }
  uint32_t mx = __reduce_max_sync(0xFFFFFFFFu, max(m2 & 0xFFFFu, m2 >> 16));
  if (WARPS > 1) {
    __shared__ uint32_t part[8];
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = mx;
    __syncthreads();
    mx = part[sub * WARPS];
#pragma unroll
    for (int i = 1; i < WARPS; ++i) mx = max(mx, part[sub * WARPS + i]);
  }
  if (m >= M) return;
  const RowScale rs = row_scale_of<FP16>(mx);
  if (tid == 0) {
    if (!rs.finite) atomicExch(err, DEV_ERR_NONFINITE);
    scale[m] = rs.scale;
  }
  int8_t* orow = out + static_cast<int64_t>(m) * ldo;
  auto put = [&](const uint4& u, int at) {
    if (!QATTN_IN_BOUNDS(err, at >= 0 && at < K)) return;
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint2 c = make_uint2(0u, 0u);
    if (rs.finite) c = codes8<FP16>(w, rs.code);
    if (at + 8 <= K) {
      *reinterpret_cast<uint2*>(orow + at) = c;
    } else {
      for (int j = 0; at + j < K; ++j)
        orow[at + j] = static_cast<int8_t>((j < 4 ? c.x >> (8 * j) : c.y >> (8 * (j - 4))) & 0xFFu);
    }
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = (i * T + tid) * 8;
    if (at < K) put(v[i], at);
  }
  for (int at = (NV * T + tid) * 8; at < K; at += T * 8) put(load8<VEC>(row, at, K), at);
}

template <int T, int NV>
static void launch_rows(const void* x, int64_t ldx, bool fp16, bool vec, int M, int K, int8_t* out,
                        int64_t ldo, float* scale, int* err, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(M) + 256 / T - 1) / (256 / T));
  const uint16_t* p = static_cast<const uint16_t*>(x);
  if (fp16 && vec) k_quant_int8_rows<T, NV, true, true><<<grid, 256, 0, stream>>>(p, ldx, M, K, out, ldo, scale, err);
  else if (fp16) k_quant_int8_rows<T, NV, true, false><<<grid, 256, 0, stream>>>(p, ldx, M, K, out, ldo, scale, err);
  else if (vec) k_quant_int8_rows<T, NV, false, true><<<grid, 256, 0, stream>>>(p, ldx, M, K, out, ldo, scale, err);
  else k_quant_int8_rows<T, NV, false, false><<<grid, 256, 0, stream>>>(p, ldx, M, K, out, ldo, scale, err);
}

// Threads and registers by the row's length: what holds a row with the fewest idle registers (12288 elements on
// 256 x 6 against 256 x 8 vectors: 4608 rows 28.0 / 30.2 us); with few rows, more threads for each (64 rows of 4096:
// 2.0 us on 256 threads, 2.5 on 128; 8704 rows 21.3 / 20.6).
cudaError_t launch_quant_int8_rows(const void* x, int64_t ldx, int fp16, int M, int K, int8_t* out,
                                   int64_t ldo, float* scale, int* err, cudaStream_t stream) {
  const bool vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && ldx % 8 == 0;
  if (K <= 1024) launch_rows<32, 4>(x, ldx, fp16, vec, M, K, out, ldo, scale, err, stream);
  else if (K <= 4096 && M <= 512) launch_rows<256, 2>(x, ldx, fp16, vec, M, K, out, ldo, scale, err, stream);
  else if (K <= 4096) launch_rows<128, 4>(x, ldx, fp16, vec, M, K, out, ldo, scale, err, stream);
  else if (K <= 8192) launch_rows<256, 4>(x, ldx, fp16, vec, M, K, out, ldo, scale, err, stream);
  else if (K <= 12288) launch_rows<256, 6>(x, ldx, fp16, vec, M, K, out, ldo, scale, err, stream);
  else launch_rows<256, 8>(x, ldx, fp16, vec, M, K, out, ldo, scale, err, stream);
  return cudaGetLastError();
}

// -------------------------------------------------------------------------------------------
// Single tokens (one or two): the weights are read once with plain 16-byte loads and multiplied with dp4a, which asks
// for the first weights sooner than a copy engine, tensor memory and a cluster that have to be set up first.  A warp takes
// ROWS weight rows at a time over all of K, eight chunks of 512 bytes in flight; the tokens' codes
// lie in shared memory.  One row where every row then has its warp (N <= 32 for each SM), else two, which halves the
// reads of the codes: N x K = 4096 x 11008 10.7 / 11.9 us, 4096 x 4096 5.7 / 6.0, 6144 x 4096 7.9 / 7.3, 18944 x 4096
// 14.3 / 14.1.  (More tokens are faster with the cluster kernel: four at 6144 x 4096 10.5 against 13.3.)
// QUANT: every block quantizes the tokens itself (a few KB, from L2) while its first weights are on their way, and
// block 0 also writes the codes and scales out, so that a linear layer is one launch.
// Bound by the weights' stream and what it takes to start it: 18944 x 4096 runs at 5.5 TB/s, 6144 x 4096 at 3.7 of 6.55.
// -------------------------------------------------------------------------------------------
namespace one {
constexpr int THREADS = 512, WARPS = THREADS / 32, BLOCKS = 2;   // per SM
constexpr int MOST_TOKENS = 2;
constexpr int MOST_BYTES = 96 * 1024;              // of codes in shared memory
}  // namespace one

__device__ __forceinline__ uint4 load_stream16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// 16 codes of a row from byte `at`, those past K zero.
__device__ __forceinline__ uint4 load_codes16(const int8_t* row, int at, int K) {
  if (at + 16 <= K) return load_stream16(row + at);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (at + j < K) w[j >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(row[at + j])) << (8 * (j & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

struct OneArgs {
  const uint16_t* x;                               // QUANT: the tokens, and where their codes and scales go
  int64_t ldx;
  int8_t* x8;                                      // else the codes
  int64_t ldx8;
  float* s_x;
  const int8_t* w;
  int64_t ldw;
};

template <int TOK, int ROWS, bool FP16, bool QUANT, bool VEC>
__global__ void __launch_bounds__(one::THREADS, one::BLOCKS)
    k_gemm_int8_one(const __grid_constant__ OneArgs o, const __grid_constant__ GemmInt8Args args) {
  using namespace one;
  constexpr int CHUNKS = 8 / ROWS;
  extern __shared__ __align__(16) uint8_t one_codes[];   // [TOK][kpad]
  __shared__ uint32_t part[WARPS][TOK];
  __shared__ float scales[TOK];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int K = args.K, kpad = (K + 15) / 16 * 16, steps = (kpad + 511) / 512;
  int n = (static_cast<int>(blockIdx.x) * WARPS + warp) * ROWS;

  uint4 w[ROWS][CHUNKS];
  auto load = [&](int first) {                     // chunks first .. first + CHUNKS - 1 of rows n ..
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const int at = ((first + c) * 32 + lane) * 16;
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        w[r][c] = make_uint4(0u, 0u, 0u, 0u);
        if (at < K && n + r < args.N) w[r][c] = load_codes16(o.w + (n + r) * o.ldw, at, K);
      }
    }
  };
  load(0);

  if (QUANT) {
    uint32_t mx[TOK];
#pragma unroll
    for (int m = 0; m < TOK; ++m) {
      uint32_t m2 = 0;
      if (m < args.M) {
        const uint16_t* row = o.x + m * o.ldx;
        for (int at = threadIdx.x * 8; at < K; at += THREADS * 8) {
          const uint4 v = load8<VEC>(row, at, K);
          m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                     __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
        }
      }
      mx[m] = __reduce_max_sync(0xFFFFFFFFu, max(m2 & 0xFFFFu, m2 >> 16));
      if (lane == 0) part[warp][m] = mx[m];
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < TOK; ++m) {
      uint32_t top = part[0][m];
#pragma unroll
      for (int i = 1; i < WARPS; ++i) top = max(top, part[i][m]);
      const RowScale rs = row_scale_of<FP16>(top);
      if (threadIdx.x == 0) {
        scales[m] = rs.scale;
        if (blockIdx.x == 0 && m < args.M) {
          o.s_x[m] = rs.scale;
          if (!rs.finite) atomicExch(args.err, DEV_ERR_NONFINITE);
        }
      }
      const uint16_t* row = o.x + m * o.ldx;
      for (int at = threadIdx.x * 8; at < kpad; at += THREADS * 8) {
        uint2 c = make_uint2(0u, 0u);
        if (m < args.M && at < K && rs.finite) {
          const uint4 v = load8<VEC>(row, at, K);
          const uint32_t e[4] = {v.x, v.y, v.z, v.w};
          c = codes8<FP16>(e, rs.code);
        }
        *reinterpret_cast<uint2*>(one_codes + m * kpad + at) = c;
        if (blockIdx.x == 0 && m < args.M) {
          int8_t* to = o.x8 + m * o.ldx8 + at;
          if (at + 8 <= K) {
            *reinterpret_cast<uint2*>(to) = c;
          } else {
            for (int j = 0; at + j < K; ++j)
              to[j] = static_cast<int8_t>((j < 4 ? c.x >> (8 * j) : c.y >> (8 * (j - 4))) & 0xFFu);
          }
        }
      }
    }
  } else {
#pragma unroll
    for (int m = 0; m < TOK; ++m) {
      if (threadIdx.x == 0) scales[m] = m < args.M ? args.s_a[m] : 0.0f;
      for (int at = threadIdx.x * 16; at < kpad; at += THREADS * 16)
        *reinterpret_cast<uint4*>(one_codes + m * kpad + at) =
            m < args.M ? load_codes16(o.x8 + m * o.ldx8, at, K) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  __syncthreads();

  for (; n < args.N; n += static_cast<int>(gridDim.x) * WARPS * ROWS) {
    int acc[ROWS][TOK];
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int m = 0; m < TOK; ++m) acc[r][m] = 0;
    for (int first = 0; first < steps; first += CHUNKS) {
      if (first > 0 || n >= static_cast<int>(gridDim.x) * WARPS * ROWS) load(first);   // the first is here already
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c) {
        const int at = ((first + c) * 32 + lane) * 16;
        if (at < kpad) {
#pragma unroll
          for (int m = 0; m < TOK; ++m) {
            const uint4 x = *reinterpret_cast<const uint4*>(one_codes + m * kpad + at);
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
              int a = acc[r][m];
              a = __dp4a(static_cast<int>(w[r][c].x), static_cast<int>(x.x), a);
              a = __dp4a(static_cast<int>(w[r][c].y), static_cast<int>(x.y), a);
              a = __dp4a(static_cast<int>(w[r][c].z), static_cast<int>(x.z), a);
              acc[r][m] = __dp4a(static_cast<int>(w[r][c].w), static_cast<int>(x.w), a);
            }
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
#pragma unroll
      for (int m = 0; m < TOK; ++m) {
        const int a = __reduce_add_sync(0xFFFFFFFFu, acc[r][m]);
        if (lane == r * TOK + m && n + r < args.N && m < args.M && QATTN_IN_BOUNDS(args.err, n + r < args.N)) {
          const float b = args.bias ? __ldg(args.bias + n + r) : 0.0f;
          static_cast<uint16_t*>(args.y)[m * args.ldy + n + r] =
              to16<FP16>(fmaf(static_cast<float>(a) * scales[m], __ldg(args.s_b + n + r), b));
        }
      }
    }
  }
}

// -------------------------------------------------------------------------------------------
// Few tokens: bound by streaming the weights once.  One CTA takes 128 weight rows (the
// MMA's M = 128, the TMEM lanes) against all tokens (N = TOK, 16 to 64) over a range of K; the
// CTAs of a cluster share the 128 rows and cut K, so that a narrow layer still keeps every SM
// loading.  int32 partial sums meet in distributed shared memory: exact, so neither the cut nor
// the order changes a result, and no workspace or atomics are needed.  Groups of four tokens go round the CTAs; every
// CTA sends its sums of a group to the owner with asynchronous stores that count on the owner's barrier, so that
// nobody waits for the whole cluster at the end (two cluster barriers and the loads between them took 2 us).
//   warp 0      TMA producer of the weights: it sets the barriers up and starts without waiting for the other
//               warps or for the preceding grid (the quantize writes only the activations)
//   warp 10     TMA producer of the tokens' codes (one thread issues a copy in about 100 clocks; two producers
//               halve the time of a K block)
//   warp 1      MMA issuer and TMEM owner
//   warps 2-9   epilogue: lane = output channel, column = token; two warps for each TMEM lane quarter,
//               each with every other group of eight tokens
// The producer and the issuer are picked with elect.sync: under `lane == 0` the compiler moves every operand of a
// copy or MMA through a vote, and a K block took 600 clocks instead of 370 whatever its size.
// Bound by latency: a call takes 4 us before any stream (16 x 512 x 1024), 24 x 4096 x 11008 13.4 us with the quantize,
// 45 MB of weights of which are 6.9.  (Up to 64 tokens: 64 x 4096 x 11008 12.8 us here and 19.4 on pairs of SMs, 64 x 9216
// x 4096 12.1 / 16.3.)
// -------------------------------------------------------------------------------------------
namespace few {
constexpr int BN = 128;                  // weight rows per CTA
constexpr int BK = 128;
constexpr int THREADS = 352;
constexpr int TILE_W = BN * BK;
constexpr int MOST_STAGES = 10;
template <int TOK>
struct Smem {
  static constexpr int TILE_X = TOK * BK;
  static constexpr int STAGE = TILE_W + TILE_X;
  // full, empty, accumulator, drain, partial sums
  static constexpr int NBARS = 2 * MOST_STAGES + 3;
  static constexpr int OFF_BAR = 0;
  static constexpr int OFF_TMEM = OFF_BAR + 8 * NBARS;
  static constexpr int OFF_ABORT = OFF_TMEM + 4;
  static constexpr int OFF_SA = (OFF_ABORT + 4 + 15) / 16 * 16;   // the tile's token scales
  static constexpr int OFF_RED = OFF_SA + 4 * TOK;                // partial sums: [peer][group][channel] of 16 bytes
  // a CTA owns up to ceil(TOK / 4 / split) groups from split peers, 2 KB each
  static constexpr int RED = (TOK / 4 + 8) * 2048;
  static constexpr int OFF_STAGES = (OFF_RED + RED + 1023) / 1024 * 1024;
  static constexpr int bytes(int stages) { return OFF_STAGES + stages * STAGE + 1024; }
  // one CTA an SM with all it can hold in flight, or two
  static constexpr int ALONE = (226 * 1024 - OFF_STAGES - 1024) / STAGE < MOST_STAGES
                                   ? (226 * 1024 - OFF_STAGES - 1024) / STAGE : MOST_STAGES;
  static constexpr int SHARED = (112 * 1024 - OFF_STAGES - 1024) / STAGE;
  static_assert(TILE_X % 1024 == 0 && SHARED >= 2 && NBARS <= 32, "alignment, stages, a lane for each barrier");
};
}  // namespace few

// s_a may come from the preceding grid, still running when this one starts: no load that the compiler may
// move in front of the wait for it or that may be served from the read-only path.
__device__ __forceinline__ float row_scale(const GemmInt8Args& a, int m) {
  return *const_cast<const volatile float*>(a.s_a + m);
}

template <int TOK, bool FP16>
__global__ void __launch_bounds__(few::THREADS, 2)
    k_gemm_int8_few(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                    const __grid_constant__ GemmInt8Args args) {
  using namespace few;
  using S = Smem<TOK>;
  const int stages = args.stages;
  constexpr uint32_t TMEM_COLS = TOK < 32 ? 32 : TOK;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = smem_u32(smem_raw);
  const uint32_t base_u32 = (raw_u32 + 1023u) & ~1023u;   // the same offset in every CTA
  uint8_t* base = smem_raw + (base_u32 - raw_u32);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int split = args.split;                           // CTAs of the cluster
  const int rank = static_cast<int>(cluster_ctarank());
  const int n0 = static_cast<int>(cluster_id()) * BN;
  // K blocks: each CTA kb_each, the first kb_more one more (no division here: with them, and the barriers set up by one
  // thread, the first copy left 1 us later)
  const int kb0 = rank * args.kb_each + (rank < args.kb_more ? rank : args.kb_more);
  const int nkb = args.kb_each + (rank < args.kb_more ? 1 : 0);             // >= 1

  const uint32_t bar0 = base_u32 + S::OFF_BAR;
  auto BAR = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
  constexpr int B_FULL = 0, B_EMPTY = MOST_STAGES, B_ACC = 2 * MOST_STAGES, B_DRAIN = B_ACC + 1, B_RED = B_ACC + 2;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(base + S::OFF_ABORT);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + S::OFF_TMEM);
  float* s_tok = reinterpret_cast<float*>(base + S::OFF_SA);
  auto by_split = [&](int g) { return (g * args.split_inv) >> 16; };        // g / split for small g
  const int tokens = args.M, groups = (tokens + 3) / 4, per = by_split(groups - 1) + 1;   // an owner's, at most
  const int mine = by_split(groups - rank + split - 1);                     // this CTA's: rank, rank + split, ..
  const uint32_t stage0 = base_u32 + S::OFF_STAGES;
  const uint64_t tlim = args.timeout_ns;
  if (warp == 0) {
    if (lane < S::NBARS) mbar_init(BAR(lane), 1);
    if (lane == 0) *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
      if (split > 1 && mine > 0) mbar_arrive_expect_tx(BAR(B_RED), static_cast<uint32_t>(mine * split) * 2048u);
      (void)QATTN_IN_BOUNDS(args.err, n0 < args.N && nkb >= 1 && (kb0 + nkb - 1) * BK < args.K);
    }
    __syncwarp();
    asm volatile("bar.arrive 2, 352;" ::: "memory");   // the barriers are ready; nothing else is needed here
  } else {
    if (warp == 1) {
      tmem_alloc(base_u32 + S::OFF_TMEM, TMEM_COLS);
      tmem_relinquish();
    }
    tc_fence_before();
    asm volatile("bar.sync 2, 352;" ::: "memory");
    tc_fence_after();
  }
  if (split > 1) cluster_arrive();                 // this CTA's barriers are ready for its peers' sums
  const uint32_t tmem = warp == 0 ? 0u : *tmem_slot;

  bool got = false;                                // epilogue threads: the accumulator is complete
  if (warp == 0) {
    // ======================= TMA producer: weights =======================
    if (elect_one()) {
      int s = 0;
      uint32_t phase = 1;                          // of the stage's use before; the first round passes at once
      int u = 0;
      for (; u < nkb; ++u) {
        if (!mbar_wait(BAR(B_EMPTY + s), phase, tlim, abort_flag, args.err)) break;
        mbar_arrive_expect_tx(BAR(B_FULL + s), S::STAGE);
        tma_load_2d(stage0 + s * S::STAGE, &tm_w, BAR(B_FULL + s), (kb0 + u) * BK, n0);
        if (++s == stages) { s = 0; phase ^= 1u; }
      }
      // every copy has landed before the CTA may exit (instant when healthy)
      for (int j = u - 1; j >= 0 && j >= u - stages; --j)
        mbar_drain(BAR(B_FULL + j % stages), (j / stages) & 1, tlim);
    }
  } else if (warp == 10) {
    // ======================= TMA producer: tokens =======================
    if (elect_one()) {
      grid_wait_prior();
      int s = 0;
      uint32_t phase = 1;
      int u = 0;
      for (; u < nkb; ++u) {
        if (!mbar_wait(BAR(B_EMPTY + s), phase, tlim, abort_flag, args.err)) break;
        tma_load_2d(stage0 + s * S::STAGE + TILE_W, &tm_x, BAR(B_FULL + s), (kb0 + u) * BK, 0);
        if (++s == stages) { s = 0; phase ^= 1u; }
      }
      // every copy has landed before the CTA may exit (instant when healthy)
      for (int j = u - 1; j >= 0 && j >= u - stages; --j)
        mbar_drain(BAR(B_FULL + j % stages), (j / stages) & 1, tlim);
    }
  } else if (warp == 1) {
    // ======================= MMA issuer =======================
    if (elect_one()) {
      constexpr uint32_t IDESC = idesc_s8_s32(BN, TOK);
      bool ok = true;
      int s = 0;
      uint32_t phase = 0;
      for (int u = 0; u < nkb; ++u) {
        ok = mbar_wait(BAR(B_FULL + s), phase, tlim, abort_flag, args.err);
        if (!ok) break;
        tc_fence_after();
        const uint32_t w_s = stage0 + s * S::STAGE, x_s = stage0 + s * S::STAGE + TILE_W;
#pragma unroll
        for (int kk = 0; kk < BK / 32; ++kk)
          mma_i8_ss(tmem, smem_desc(w_s + kk * 32, 16, 1024, 2u), smem_desc(x_s + kk * 32, 16, 1024, 2u),
                    IDESC, (u > 0 || kk > 0) ? 1u : 0u);
        mma_commit(BAR(B_EMPTY + s));
        if (++s == stages) { s = 0; phase ^= 1u; }
      }
      if (ok) mma_commit(BAR(B_ACC));
      mma_commit(BAR(B_DRAIN));
      mbar_drain(BAR(B_DRAIN), 0, tlim);
    }
  } else {
    // ======================= epilogue: lane = output channel, column = token =======================
    const int quarter = warp & 3, half = (warp - 2) >> 2, r = quarter * 32 + lane, n = n0 + r;
    float s_n = 0.0f, b_n = 0.0f;
    if (n < args.N) {
      s_n = __ldg(args.s_b + n);
      if (args.bias) b_n = __ldg(args.bias + n);
    }
    // The token scales may come from the preceding grid, still running when this one starts: no load
    // in front of the wait for it.  They pass through shared memory; read for each column from
    // global memory they cost a round trip a column in a row.
    grid_wait_prior();
    for (int i = static_cast<int>(threadIdx.x) - 64; i < TOK; i += 256)
      s_tok[i] = i < tokens ? row_scale(args, i) : 0.0f;
    asm volatile("bar.sync 1, 256;" ::: "memory");
    got = __all_sync(0xFFFFFFFFu, mbar_wait(BAR(B_ACC), 0, tlim, abort_flag, args.err));
    uint16_t* y = static_cast<uint16_t*>(args.y) + n;
    // four tokens from column c on (their scales on 16 bytes)
    auto put4 = [&](const int (&a)[4], int c) {
      const float4 st = *reinterpret_cast<const float4*>(s_tok + c);
      const float s4[4] = {st.x, st.y, st.z, st.w};
      uint16_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = to16<FP16>(fmaf(static_cast<float>(a[e]) * s4[e], s_n, b_n));
      if (n < args.N) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < tokens && QATTN_IN_BOUNDS(args.err, c + e < args.M)) y[(c + e) * args.ldy] = o[e];
      }
    };
    if (split > 1) cluster_wait();                 // the peers' barriers are ready
    if (got) {
      tc_fence_after();
      const uint32_t acc = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll 1
      for (int c = half * 8; c < tokens; c += 16) {
        uint32_t v[8];
        tmem_ld8(acc + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int g = c / 4 + j;
          const int a[4] = {static_cast<int>(v[4 * j]), static_cast<int>(v[4 * j + 1]), static_cast<int>(v[4 * j + 2]),
                            static_cast<int>(v[4 * j + 3])};
          if (split == 1) {
            put4(a, c + 4 * j);
          } else if (g < groups) {
            const int i = by_split(g), owner = g - i * split;
            st_async_v4(mapa_shared(base_u32 + S::OFF_RED + static_cast<uint32_t>(((rank * per + i) * 128 + r) * 16),
                                    static_cast<uint32_t>(owner)),
                        a, mapa_shared(BAR(B_RED), static_cast<uint32_t>(owner)));
          }
        }
      }
      if (split > 1 && mine > 0) {
        got = __all_sync(0xFFFFFFFFu, mbar_wait<true>(BAR(B_RED), 0, tlim, abort_flag, args.err));   // the peers' stores
        for (int i = half; got && i < mine; i += 2) {
          int a[4] = {0, 0, 0, 0};
          for (int p = 0; p < split; ++p) {
            const int4 v = *reinterpret_cast<const int4*>(base + S::OFF_RED + ((p * per + i) * 128 + r) * 16);
            a[0] += v.x;
            a[1] += v.y;
            a[2] += v.z;
            a[3] += v.w;
          }
          put4(a, 4 * (i * split + rank));
        }
      }
    }
  }

  if (split > 1 && (warp < 2 || warp == 10)) cluster_wait();
  tc_fence_before();
  __syncthreads();
  // A CTA that has given up keeps its shared memory until its peers have exited or given up too: their sums may
  // still be on their way here.  (The flag is the same for every thread: its writers are past the barrier.)
  if (split > 1 && *abort_flag) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// -------------------------------------------------------------------------------------------
// Pair kernel: two SMs (a cluster of two CTAs) on one 256 x BN output tile, the roles of the FP8
// pair GEMM (gemm_fp8.cu) with kind::i8:
//   warp 0 (both CTAs)  TMA producer of its 128 rows of A and BN / 2 rows of B, into a ring whose
//                       `full` barriers live in the leading CTA
//   warp 1              TMEM owner; in the leading CTA the MMA issuer (two accumulators)
//   warps 2-9 (both)    epilogue of the CTA's 128 rows, overlapping the next tile's MMAs; two warps for
//                       each TMEM lane quarter, each with half of the columns
// (The producer and the issuer are picked with elect.sync, see above: 470 clocks a K block instead of 684.)
// Tiles are visited m-fastest.  Every wait is bounded and both CTAs reach both cluster barriers.
// Bound by the MMA: a 256 x 256 x 128 block takes 520 clocks of the pair (512 at the nominal rate), 8704 x 12288 x 4096
// 265 to 300 us by the card's power limit (2920 to 3300 TOP/s); one wave (512 x 9216 x 4096, 17.7 us) adds 1.2 us until
// the first block, 2.3 of epilogue and 1 at the end.  Two producers, as above, changed nothing here (18.0 against 18.2,
// and 1 to 4 % slower at 4608 x 4096 x 12288).
// -------------------------------------------------------------------------------------------
namespace pair8 {
constexpr int BM = 256;
constexpr int BK = 128;
constexpr int THREADS = 320;
constexpr int EPI_WARPS = 8;
constexpr int TILE_A = (BM / 2) * BK;
template <int BN>
struct Smem {
  static constexpr int TILE_B = (BN / 2) * BK;
  static constexpr int STAGES = (192 * 1024) / (TILE_A + TILE_B);
  static constexpr int OFF_A = 0, OFF_B = STAGES * TILE_A;
  static constexpr int OFF_BAR = OFF_B + STAGES * TILE_B;
  static constexpr int NBARS = 2 * STAGES + 4 + 1;
  static constexpr int OFF_TMEM = OFF_BAR + 8 * NBARS;
  static constexpr int OFF_ABORT = OFF_TMEM + 4;
  static constexpr int OFF_T = (OFF_ABORT + 4 + 15) / 16 * 16; // per epilogue warp: 32 x 32 16-bit outputs,
  static constexpr int COLS0 = (BN / 2 + 31) / 32 * 32;        // columns of the first epilogue warps; the others': the rest
  static constexpr int WARP_T = 32 * 64 + 2 * COLS0 * 4;        // and its columns' scales and biases
  static constexpr int ALLOC = OFF_T + EPI_WARPS * WARP_T + 1024;
  static constexpr uint32_t TMEM_COLS = BN <= 64 ? 128 : BN <= 128 ? 256 : 512;
  static constexpr uint32_t STAGE_TX = 2u * (TILE_A + TILE_B);
  static_assert(TILE_B % 1024 == 0 && NBARS <= 32, "alignment, a lane for each barrier");
  static_assert(ALLOC <= 227 * 1024, "shared memory per CTA");
};
}  // namespace pair8

// 32 x 32 outputs of a warp (lane = row m of the accumulator, columns n ..): y = acc * s_a * s_b + bias, through
// shared memory so that a store instruction writes whole rows: 8 rows of 64 bytes where rows start on 16 bytes, else
// one row's 32 neighbours.  Stored by the lanes as they hold the rows, an instruction touches 32 lines: a tile's
// epilogue took 11000 clocks on four warps, 4400 now on eight.  sb, bias: the 32 columns' values in shared memory.
template <bool FP16>
__device__ __forceinline__ void epilogue_int8(const GemmInt8Args& a, const uint32_t (&v)[32], float s_m, int m_warp,
                                              int n, bool vec, const float* sb, const float* bias, uint8_t* tile) {
  if (!QATTN_IN_BOUNDS(a.err, n < a.N)) return;
  const int lane = threadIdx.x & 31;
  const int rows = min(32, a.M - m_warp);          // may be <= 0
  const f32x2 s2 = pack_f32x2(s_m, s_m);
  // 16-byte piece j of row r lies at piece j ^ (r / 2 % 4): no bank conflict either way
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const ulonglong2 s0 = *reinterpret_cast<const ulonglong2*>(sb + 8 * j), s1 = *reinterpret_cast<const ulonglong2*>(sb + 8 * j + 4);
    const ulonglong2 b0 = *reinterpret_cast<const ulonglong2*>(bias + 8 * j), b1 = *reinterpret_cast<const ulonglong2*>(bias + 8 * j + 4);
    const f32x2 sv[4] = {s0.x, s0.y, s1.x, s1.y}, bv[4] = {b0.x, b0.y, b1.x, b1.y};
    uint32_t p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 8 * j + 2 * e;
      const f32x2 acc = pack_f32x2(static_cast<float>(static_cast<int>(v[i])), static_cast<float>(static_cast<int>(v[i + 1])));
      float lo, hi;
      unpack_f32x2(fma_f32x2(mul_f32x2(acc, s2), sv[e], bv[e]), lo, hi);
      p[e] = to16x2<FP16>(lo, hi);
    }
    *reinterpret_cast<uint4*>(tile + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) = make_uint4(p[0], p[1], p[2], p[3]);
  }
  __syncwarp();
  uint16_t* y = static_cast<uint16_t*>(a.y) + m_warp * a.ldy + n;
  if (vec && n + 32 <= a.N) {
    const int j = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2);
      if (r < rows)
        *reinterpret_cast<uint4*>(y + r * a.ldy + 8 * j) =
            *reinterpret_cast<const uint4*>(tile + r * 64 + ((j ^ ((r >> 1) & 3)) << 4));
    }
  } else if (n + lane < a.N) {
#pragma unroll 8
    for (int r = 0; r < rows; ++r)
      y[r * a.ldy + lane] = *reinterpret_cast<const uint16_t*>(tile + r * 64 + (((lane >> 3) ^ ((r >> 1) & 3)) << 4) + (lane & 7) * 2);
  }
  __syncwarp();
}

template <int BN, bool FP16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(pair8::THREADS, 1)
    k_gemm_int8_pair(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                     const __grid_constant__ GemmInt8Args args) {
  using namespace pair8;
  using S = Smem<BN>;
  constexpr int STAGES = S::STAGES;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = smem_u32(smem_raw);
  const uint32_t base_u32 = (raw_u32 + 1023u) & ~1023u;   // the same offset in both CTAs
  uint8_t* base = smem_raw + (base_u32 - raw_u32);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();                  // 0 leads the pair
  const bool leader = rank == 0;
  const int pair = static_cast<int>(blockIdx.x >> 1), npairs = static_cast<int>(gridDim.x >> 1);

  const int tiles_m = (args.M + BM - 1) / BM;
  const int tiles = tiles_m * ((args.N + BN - 1) / BN);   // the host launches <= tiles pairs
  const int kblocks = (args.K + BK - 1) / BK;

  const uint32_t bar0 = base_u32 + S::OFF_BAR;
  auto BAR = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
  constexpr int B_FULL = 0, B_EMPTY = STAGES, B_ACCF = 2 * STAGES, B_ACCE = B_ACCF + 2;
  constexpr int B_DRAIN = B_ACCE + 2;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(base + S::OFF_ABORT);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + S::OFF_TMEM);
  if (warp == 0) {                     // a lane for each barrier
    if (lane < S::NBARS) mbar_init(BAR(lane), lane >= B_ACCE && lane < B_ACCE + 2 ? 2 * EPI_WARPS : 1);
    if (lane == 0) *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(base_u32 + S::OFF_TMEM, S::TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();                      // barriers of both CTAs initialised, TMEM allocated
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint64_t tlim = args.timeout_ns;

  if (warp == 0) {
    // ======================= TMA producer (both CTAs) =======================
    if (elect_one()) {
      tma_prefetch_desc(&tm_a);
      tma_prefetch_desc(&tm_b);
      grid_wait_prior();
      int u = 0;
      bool ok = true;
      for (int t = pair; ok && t < tiles; t += npairs) {
        const int m0 = (t % tiles_m) * BM + static_cast<int>(rank) * (BM / 2);
        const int n0 = (t / tiles_m) * BN + static_cast<int>(rank) * (BN / 2);
        (void)QATTN_IN_BOUNDS(args.err, (t % tiles_m) * BM < args.M && (t / tiles_m) * BN < args.N);
        for (int kb = 0; kb < kblocks; ++kb, ++u) {
          const int s = u % STAGES;
          if (u >= STAGES &&
              !mbar_wait(BAR(B_EMPTY + s), ((u / STAGES) - 1) & 1, tlim, abort_flag, args.err)) {
            ok = false;
            break;
          }
          if (leader) mbar_arrive_expect_tx(BAR(B_FULL + s), S::STAGE_TX);
          const uint32_t full_lead = mapa_shared(BAR(B_FULL + s), 0);
          tma_load_2d_pair(base_u32 + S::OFF_A + s * TILE_A, &tm_a, full_lead, kb * BK, m0);
          tma_load_2d_pair(base_u32 + S::OFF_B + s * S::TILE_B, &tm_b, full_lead, kb * BK, n0);
        }
      }
      // the MMAs have released every stage this CTA filled
      for (int j = u - 1; j >= 0 && j >= u - STAGES; --j)
        mbar_drain(BAR(B_EMPTY + j % STAGES), (j / STAGES) & 1, tlim);
    }
  } else if (warp == 1) {
    // ======================= MMA issuer (leading CTA) =======================
    if (leader && elect_one()) {
      constexpr uint32_t IDESC = idesc_s8_s32(BM, BN);
      int u = 0, i = 0;
      bool ok = true;
      for (int t = pair; ok && t < tiles; t += npairs, ++i) {
        const int ab = i & 1;
        // both CTAs' epilogues have read out the tile that used this accumulator two tiles ago
        if (i >= 2)
          ok = mbar_wait(BAR(B_ACCE + ab), ((i >> 1) - 1) & 1, tlim, abort_flag, args.err);
        if (!ok) break;
        tc_fence_after();
        const uint32_t acc = tmem + static_cast<uint32_t>(ab * BN);
        for (int kb = 0; kb < kblocks; ++kb, ++u) {
          const int s = u % STAGES;
          ok = mbar_wait(BAR(B_FULL + s), (u / STAGES) & 1, tlim, abort_flag, args.err);
          if (!ok) break;
          tc_fence_after();
          const uint32_t a_s = base_u32 + S::OFF_A + s * TILE_A;
          const uint32_t b_s = base_u32 + S::OFF_B + s * S::TILE_B;
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk)
            mma_i8_ss_pair(acc, smem_desc(a_s + kk * 32, 16, 1024, 2u), smem_desc(b_s + kk * 32, 16, 1024, 2u),
                           IDESC, (kb > 0 || kk > 0) ? 1u : 0u);
          mma_commit_pair_both(BAR(B_EMPTY + s));                 // stage free in both CTAs
        }
        if (ok) mma_commit_pair_both(BAR(B_ACCF + ab));           // accumulator complete
      }
      mma_commit_pair(BAR(B_DRAIN));
      mbar_drain(BAR(B_DRAIN), 0, tlim);
    }
  } else {
    // ======================= epilogue warps (both CTAs) =======================
    grid_wait_prior();                             // s_a comes from the preceding grid
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const int cols = half == 0 ? S::COLS0 : BN - S::COLS0;     // of this warp
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    uint8_t* stage = base + S::OFF_T + (warp - 2) * S::WARP_T;
    float* sb = reinterpret_cast<float*>(stage + 32 * 64);
    float* bias = sb + S::COLS0;
    const bool vec = (reinterpret_cast<uintptr_t>(args.y) & 15) == 0 && args.ldy % 8 == 0;
    int i = 0;
    for (int t = pair; t < tiles; t += npairs, ++i) {
      const int ab = i & 1;
      const int m_warp = (t % tiles_m) * BM + static_cast<int>(rank) * (BM / 2) + quarter * 32, m = m_warp + lane;
      const int n0 = (t / tiles_m) * BN + half * S::COLS0;
      const float s_m = m < args.M ? row_scale(args, m) : 0.0f;
      for (int e = lane; e < cols; e += 32) {
        sb[e] = n0 + e < args.N ? __ldg(args.s_b + n0 + e) : 0.0f;
        bias[e] = args.bias && n0 + e < args.N ? __ldg(args.bias + n0 + e) : 0.0f;
      }
      __syncwarp();
      const bool ok = mbar_wait(BAR(B_ACCF + ab), (i >> 1) & 1, tlim, abort_flag, args.err);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      tc_fence_after();
      const uint32_t acc = tmem + lane_off + static_cast<uint32_t>(ab * BN + half * S::COLS0);
      uint32_t v[2][32];
      tmem_ld32(acc, v[0]);
      tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < S::COLS0; c += 32) {
        if (c >= cols || n0 + c >= args.N) break;  // uniform
        // the next 32 columns are read while these are converted and stored
        if (c + 32 < cols) tmem_ld32(acc + c + 32, v[(c / 32 + 1) & 1]);
        epilogue_int8<FP16>(args, v[(c / 32) & 1], s_m, m_warp, n0 + c, vec, sb + c, bias + c, stage);
        tmem_wait_ld();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(BAR(B_ACCE + ab), 0));   // read out
    }
  }

  tc_fence_before();
  cluster_sync();                      // no MMA, load or arrival of either CTA is outstanding
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, S::TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------------------------

// [rows, K] int8, K contiguous, `ld` bytes between rows (a multiple of 16); box of `box_rows` rows x
// 128 bytes, 128-byte swizzle; reads past the last row or past K return zeros, which add nothing.
static bool make_map_rows(CUtensorMap* map, const void* ptr, int rows, int K, int64_t ld, int box_rows) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
  cuuint32_t box[2] = {128u, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1u, 1u};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class K>
static cudaError_t launch_ex(K kernel, DeviceOnce& once, dim3 grid, unsigned cluster, int threads, int most_smem,
                             int smem, bool early, cudaStream_t stream, const CUtensorMap& a, const CUtensorMap& b,
                             const GemmInt8Args& args) {
  const void* fn = reinterpret_cast<const void*>(kernel);
  if (once.get([fn, most_smem] {
        return static_cast<int>(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, most_smem));
      }) != static_cast<int>(cudaSuccess))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  unsigned n = 0;
  if (cluster > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = cluster;
    at[n].val.clusterDim.y = 1;
    at[n++].val.clusterDim.z = 1;
  }
  if (early) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = at;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, a, b, args);
}

// Clusters of `split` CTAs that are resident at once at one CTA an SM.  They do not cross the SMs' groups, so there may be
// fewer than SMs / split: 48 clusters of three take two rounds on 148 SMs.
template <int TOK, bool FP16>
static int few_resident(int split, int num_sms) {
  constexpr int SMEM = few::Smem<TOK>::bytes(few::Smem<TOK>::ALONE);
  cudaFuncSetAttribute(k_gemm_int8_few<TOK, FP16>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(num_sms / split * split));
  cfg.blockDim = dim3(few::THREADS);
  cfg.dynamicSmemBytes = SMEM;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = static_cast<unsigned>(split);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, k_gemm_int8_few<TOK, FP16>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

// CTAs that share 128 weight rows: as many as keep all tiles resident at one CTA an SM, with at least two K blocks
// each.  16 tokens, K = 4096, splits 1 / 2 / 3 / 4 / 8: N = 4096 9.3 / 8.3 / 7.9 / 7.4 / 7.9 us, 6144 9.7 / 9.2 / 14.0 /
// 9.5 / 10.9, 1024 7.8 / 6.7 / 6.1 / 5.4 / 4.5, 12288 12.4 / 13.7 / 16.0 / 15.0 / 17.1; 64 x 1024 x 1024 with four blocks
// each 6.0, two 5.1.
template <int TOK, bool FP16>
static int few_split(int64_t tiles, int kblocks, int num_sms) {
  static DeviceOnce resident[9];
  for (int split = 8; split > 1; --split) {
    if (split > kblocks / 2 || tiles * split > num_sms) continue;
    if (tiles <= resident[split].get([split, num_sms] { return few_resident<TOK, FP16>(split, num_sms); })) return split;
  }
  return 1;
}

template <int TOK, bool FP16>
static cudaError_t launch_few(const int8_t* x, int64_t ldx, const int8_t* w, int64_t ldw, const GemmInt8Args& a,
                              int num_sms, bool early, cudaStream_t stream) {
  static DeviceOnce once;
  using S = few::Smem<TOK>;
  CUtensorMap mw, mx;
  if (!make_map_rows(&mw, w, a.N, a.K, ldw, few::BN) || !make_map_rows(&mx, x, a.M, a.K, ldx, TOK))
    return cudaErrorInvalidValue;
  const int64_t tiles = (static_cast<int64_t>(a.N) + few::BN - 1) / few::BN;
  const int kblocks = (a.K + few::BK - 1) / few::BK;
  GemmInt8Args b = a;
  b.split = few_split<TOK, FP16>(tiles, kblocks, num_sms);
  b.split_inv = 65536 / b.split + 1;
  b.kb_each = kblocks / b.split;
  b.kb_more = kblocks % b.split;
  b.stages = tiles * b.split <= num_sms ? S::ALONE : S::SHARED;
  return launch_ex(k_gemm_int8_few<TOK, FP16>, once, dim3(static_cast<unsigned>(tiles * b.split)),
                   static_cast<unsigned>(b.split), few::THREADS, S::bytes(S::ALONE), S::bytes(b.stages), early, stream,
                   mw, mx, b);
}

template <int BN, bool FP16>
static cudaError_t launch_pair(const int8_t* x, int64_t ldx, const int8_t* w, int64_t ldw, const GemmInt8Args& a,
                               int num_sms, bool early, cudaStream_t stream) {
  static DeviceOnce once, resident;
  CUtensorMap ma, mb;
  if (!make_map_rows(&ma, x, a.M, a.K, ldx, pair8::BM / 2) || !make_map_rows(&mb, w, a.N, a.K, ldw, BN / 2))
    return cudaErrorInvalidValue;
  const int most = resident.get([num_sms] {
    cudaFuncSetAttribute(k_gemm_int8_pair<BN, FP16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                         pair8::Smem<BN>::ALLOC);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(num_sms & ~1));
    cfg.blockDim = dim3(pair8::THREADS);
    cfg.dynamicSmemBytes = pair8::Smem<BN>::ALLOC;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, k_gemm_int8_pair<BN, FP16>, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = num_sms / 2;
    }
    return n;
  });
  const int64_t tiles = (static_cast<int64_t>(a.M) + pair8::BM - 1) / pair8::BM * ((a.N + BN - 1) / BN);
  const int pairs = tiles < most ? static_cast<int>(tiles) : most;
  return launch_ex(k_gemm_int8_pair<BN, FP16>, once, dim3(static_cast<unsigned>(2 * pairs)), 0, pair8::THREADS,
                   pair8::Smem<BN>::ALLOC, pair8::Smem<BN>::ALLOC, early, stream, ma, mb, a);
}

template <int TOK, int ROWS, bool FP16, bool QUANT, bool VEC>
static cudaError_t launch_one_rows(const OneArgs& o, const GemmInt8Args& a, int num_sms, cudaStream_t stream) {
  static DeviceOnce once;
  const void* fn = reinterpret_cast<const void*>(k_gemm_int8_one<TOK, ROWS, FP16, QUANT, VEC>);
  if (once.get([fn] {
        return static_cast<int>(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, one::MOST_BYTES));
      }) != static_cast<int>(cudaSuccess))
    return cudaErrorInvalidValue;
  const int per_block = one::WARPS * ROWS;
  const int64_t blocks = (static_cast<int64_t>(a.N) + per_block - 1) / per_block, most = static_cast<int64_t>(num_sms) * one::BLOCKS;
  k_gemm_int8_one<TOK, ROWS, FP16, QUANT, VEC><<<static_cast<unsigned>(blocks < most ? blocks : most), one::THREADS,
                                           TOK * ((a.K + 15) / 16 * 16), stream>>>(o, a);
  return cudaGetLastError();
}

template <int TOK, bool FP16, bool QUANT, bool VEC>
static cudaError_t launch_one_as(const OneArgs& o, const GemmInt8Args& a, int num_sms, cudaStream_t stream) {
  if (a.N <= num_sms * one::BLOCKS * one::WARPS) return launch_one_rows<TOK, 1, FP16, QUANT, VEC>(o, a, num_sms, stream);
  return launch_one_rows<TOK, 2, FP16, QUANT, VEC>(o, a, num_sms, stream);
}

template <int TOK, bool QUANT>
static cudaError_t launch_one(const OneArgs& o, const GemmInt8Args& a, int fp16, int num_sms, cudaStream_t stream) {
  const bool vec = !QUANT || ((reinterpret_cast<uintptr_t>(o.x) & 15) == 0 && o.ldx % 8 == 0);
  if (fp16 && vec) return launch_one_as<TOK, true, QUANT, true>(o, a, num_sms, stream);
  if (vec) return launch_one_as<TOK, false, QUANT, true>(o, a, num_sms, stream);
  if constexpr (QUANT) {
    if (fp16) return launch_one_as<TOK, true, QUANT, false>(o, a, num_sms, stream);
    return launch_one_as<TOK, false, QUANT, false>(o, a, num_sms, stream);
  }
  return cudaErrorInvalidValue;
}

// One or two tokens whose codes fit shared memory.
static bool one_fits(int M, int K) {
  return M <= one::MOST_TOKENS && static_cast<int64_t>(M) * ((K + 15) / 16 * 16) <= one::MOST_BYTES;
}

template <bool QUANT>
static cudaError_t launch_one_m(const OneArgs& o, const GemmInt8Args& a, int fp16, int num_sms, cudaStream_t stream) {
  if (a.M == 1) return launch_one<1, QUANT>(o, a, fp16, num_sms, stream);
  return launch_one<2, QUANT>(o, a, fp16, num_sms, stream);
}

// Columns of a pair tile: the pairs run waves of tiles, and the width that fills its last wave best wins.  A wave takes,
// in us for a K block of 128, 0.175 with 64 columns (bound by the copies: 53 of 64 bytes a clock into an SM) to 0.30 with
// 256 (bound by the MMA: 0.265 at the full clock, more at the one that the card's power leaves), and the epilogue that
// nothing overlaps up to 1.6 more than with 64.  The numbers are a fit to whole calls and not a rate for each width: over 51
// sizes (130 to 8704 tokens, widths 512 to 16384, all six timed in turn) the pick is 0.2 % slower than the best on average
// and 3 % at most; with 224 columns at 224 / 256 of 0.30, 0.4 % and 7.7 %.
// Measured on 74 pairs (64 / 128 / 160 / 192 / 224 / 256 columns): 333 x 5120 x 5120 25.7 / 20.0 / 14.5 / 16.2 / 17.1 /
// 18.6 us, 1500 x 2048 x 8192 37.4 / 28.0 / 29.6 / 21.3 / 22.9 / 25.3, 512 x 4096 x 4096 16.3 / 12.0 / 12.8 / 14.2 / 15.1 / 16.3,
// 1024 x 9216 x 4096 50.0 / 32.2 / 32.7 / 30.9 / 32.3 / 28.6, 2048 x 12288 x 4096 122 / 80.0 / 72.0 / 71.3 / 69.2 / 78.8.
static int pair_columns(int M, int N, int K, int pairs) {
  const int cols[6] = {64, 128, 160, 192, 224, 256};
  const double block[6] = {0.175, 0.195, 0.216, 0.232, 0.25, 0.30}, tail[6] = {0.0, 0.5, 0.8, 1.0, 1.3, 1.6};
  const double kblocks = (K + pair8::BK - 1) / pair8::BK;
  int best = 256;
  double least = 1e30;
  for (int i = 5; i >= 0; --i) {
    const int64_t tiles = (static_cast<int64_t>(M) + pair8::BM - 1) / pair8::BM * ((N + cols[i] - 1) / cols[i]);
    const double t = static_cast<double>((tiles + pairs - 1) / pairs) * kblocks * block[i] + tail[i];
    if (t < least) {
      least = t;
      best = cols[i];
    }
  }
  return best;
}

template <bool FP16>
static cudaError_t launch_any(const int8_t* x, int64_t ldx, const int8_t* w, int64_t ldw, const GemmInt8Args& a,
                              int num_sms, bool early, cudaStream_t stream) {
  if (a.M <= 16) return launch_few<16, FP16>(x, ldx, w, ldw, a, num_sms, early, stream);
  if (a.M <= 32) return launch_few<32, FP16>(x, ldx, w, ldw, a, num_sms, early, stream);
  if (a.M <= 64) return launch_few<64, FP16>(x, ldx, w, ldw, a, num_sms, early, stream);
  switch (pair_columns(a.M, a.N, a.K, num_sms / 2)) {
    case 64: return launch_pair<64, FP16>(x, ldx, w, ldw, a, num_sms, early, stream);
    case 128: return launch_pair<128, FP16>(x, ldx, w, ldw, a, num_sms, early, stream);
    case 160: return launch_pair<160, FP16>(x, ldx, w, ldw, a, num_sms, early, stream);
    case 192: return launch_pair<192, FP16>(x, ldx, w, ldw, a, num_sms, early, stream);
    case 224: return launch_pair<224, FP16>(x, ldx, w, ldw, a, num_sms, early, stream);
    default: return launch_pair<256, FP16>(x, ldx, w, ldw, a, num_sms, early, stream);
  }
}

static cudaError_t launch_codes(const int8_t* a8, int64_t lda, const int8_t* b8, int64_t ldb, const GemmInt8Args& a,
                                int fp16, int num_sms, bool early, cudaStream_t stream) {
  return fp16 ? launch_any<true>(a8, lda, b8, ldb, a, num_sms, early, stream)
              : launch_any<false>(a8, lda, b8, ldb, a, num_sms, early, stream);
}

cudaError_t launch_gemm_int8(const int8_t* a8, int64_t lda, const int8_t* b8, int64_t ldb, const GemmInt8Args& a,
                             int fp16, int num_sms, cudaStream_t stream) {
  if (one_fits(a.M, a.K))
    return launch_one_m<false>({nullptr, 0, const_cast<int8_t*>(a8), lda, nullptr, b8, ldb}, a, fp16, num_sms, stream);
  return launch_codes(a8, lda, b8, ldb, a, fp16, num_sms, false, stream);
}

cudaError_t launch_linear_int8(const void* x, int64_t ldx, int8_t* x8, int64_t ldx8, float* s_x, const int8_t* w8,
                               int64_t ldw, const GemmInt8Args& a, int fp16, int num_sms, cudaStream_t stream) {
  if (one_fits(a.M, a.K))
    return launch_one_m<true>({static_cast<const uint16_t*>(x), ldx, x8, ldx8, s_x, w8, ldw}, a, fp16, num_sms, stream);
  const cudaError_t e = launch_quant_int8_rows(x, ldx, fp16, a.M, a.K, x8, ldx8, s_x, a.err, stream);
  if (e != cudaSuccess) return e;
  return launch_codes(x8, ldx8, w8, ldw, a, fp16, num_sms, true, stream);
}

}  // namespace qattn
