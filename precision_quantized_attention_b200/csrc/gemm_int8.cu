// gemm_int8.cu -- linear layers in 8-bit integers for sm_100a: activations quantized with a scale for
// each row (token), weights with a scale for each row (output channel), products summed exactly in
// int32 on the tensor cores (tcgen05 kind::i8):
//   s[m]    = amax_k |x[m, k]| / 127 (1 for a row of zeros),  c[m, k] = rint(127 x[m, k] / amax)
//   y[m, n] = (sum_k c[m, k] w8[n, k]) * s[m] * s_w[n] (+ bias[n])
//
//   k_quant_int8_rows  the per-row quantize, one read of x (a row stays in registers)
//   k_gemm_int8_few    few tokens (one tile of them): weight rows are the MMA's M, tokens its N, K is
//                      split over a cluster whose partial sums meet in shared memory
//   k_gemm_int8_pair   otherwise: 256 x BN output tiles on pairs of SMs (cta_group::2)
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
// c127 = 127 * p and amax = p * (the row's), p a power of two (see scale_pow2); r = RN(1 / amax).
__device__ __forceinline__ uint32_t code_int8(float x, float c127, float amax, float r) {
  const float q = div_rn_by(c127 * x, amax, r);
  return static_cast<uint32_t>(__float_as_int(q + 12582912.0f)) & 0xFFu;
}

// Power of two that brings a row's maximum to where 127 x cannot overflow and the quotient's residual
// stays normal (bf16 reaches 2^127 and 2^-133); scaling by it is exact wherever the code is not 0.
__device__ __forceinline__ float scale_pow2(float amax) {
  return amax > 0x1p+100f ? 0x1p-60f : amax < 0x1p-60f ? 0x1p+80f : 1.0f;
}

template <bool FP16>
__device__ __forceinline__ uint2 codes8(const uint32_t (&w)[4], float c127, float amax, float r) {
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[2 * i] = code_int8(from16<FP16>(w[i] & 0xFFFFu), c127, amax, r);
    c[2 * i + 1] = code_int8(from16<FP16>(w[i] >> 16), c127, amax, r);
  }
  return make_uint2(c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24),
                    c[4] | (c[5] << 8) | (c[6] << 16) | (c[7] << 24));
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
  if (m >= M || !QATTN_IN_BOUNDS(err, m >= 0)) return;
  const bool finite = mx < (FP16 ? 0x7C00u : 0x7F80u);
  float amax = from16<FP16>(mx);
  if (tid == 0) {
    if (!finite) atomicExch(err, DEV_ERR_NONFINITE);
    scale[m] = !finite ? __int_as_float(0x7FFFFFFF) : mx == 0 ? 1.0f : __fdiv_rn(amax, 127.0f);
  }
  if (mx == 0) amax = 1.0f;
  const float p2 = scale_pow2(amax), c127 = 127.0f * p2;
  amax *= p2;
  const float r = __frcp_rn(amax);
  int8_t* orow = out + static_cast<int64_t>(m) * ldo;
  auto put = [&](const uint4& u, int at) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint2 c = make_uint2(0u, 0u);
    if (finite) c = codes8<FP16>(w, c127, amax, r);
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

// A warp for rows of up to 1024 elements, 128 threads up to 4096, a block beyond (in registers up
// to 16384).
cudaError_t launch_quant_int8_rows(const void* x, int64_t ldx, int fp16, int M, int K, int8_t* out,
                                   int64_t ldo, float* scale, int* err, cudaStream_t stream) {
  const bool vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && ldx % 8 == 0;
  if (K <= 1024) launch_rows<32, 4>(x, ldx, fp16, vec, M, K, out, ldo, scale, err, stream);
  else if (K <= 4096) launch_rows<128, 4>(x, ldx, fp16, vec, M, K, out, ldo, scale, err, stream);
  else if (K <= 8192) launch_rows<256, 4>(x, ldx, fp16, vec, M, K, out, ldo, scale, err, stream);
  else launch_rows<256, 8>(x, ldx, fp16, vec, M, K, out, ldo, scale, err, stream);
  return cudaGetLastError();
}

// -------------------------------------------------------------------------------------------
// Few tokens (M <= 128): bound by streaming the weights once.  One CTA takes 128 weight rows (the
// MMA's M = 128, the TMEM lanes) against all tokens (N = TOK, 16 to 128) over a range of K; the
// CTAs of a cluster share the 128 rows and cut K, so that a narrow layer still keeps every SM
// loading.  int32 partial sums meet through distributed shared memory: exact, so neither the cut nor
// the order changes a result, and no workspace or atomics are needed.
//   warp 0      TMA producer; the weights of the first stages are requested before the wait for the
//               preceding grid (the quantize writes only the activations)
//   warp 1      MMA issuer and TMEM owner
//   warps 2-5   epilogue: lane = output channel, column = token
// -------------------------------------------------------------------------------------------
namespace few {
constexpr int BN = 128;                  // weight rows per CTA
constexpr int BK = 128;
constexpr int THREADS = 192;
constexpr int TILE_W = BN * BK;
template <int TOK>
struct Smem {
  static constexpr int TILE_X = TOK * BK;
  static constexpr int STAGE = TILE_W + TILE_X;
  static constexpr int STAGES = (104 * 1024) / STAGE;          // two CTAs fit an SM
  static constexpr int OFF_W = 0, OFF_X = STAGES * TILE_W;
  static constexpr int OFF_BAR = OFF_X + STAGES * TILE_X;
  static constexpr int NBARS = 2 * STAGES + 2;                 // full, empty, accumulator, drain
  static constexpr int OFF_TMEM = OFF_BAR + 8 * NBARS;
  static constexpr int OFF_ABORT = OFF_TMEM + 4;
  static constexpr int ALLOC = OFF_ABORT + 4 + 1024;
  static_assert(TOK * 128 * 4 <= STAGES * STAGE, "partial sums reuse the stages");
  static_assert(TILE_X % 1024 == 0, "alignment");
};
}  // namespace few

template <int TOK, bool FP16>
__global__ void __launch_bounds__(few::THREADS, 2)
    k_gemm_int8_few(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                    const __grid_constant__ GemmInt8Args args) {
  using namespace few;
  using S = Smem<TOK>;
  constexpr int STAGES = S::STAGES;
  constexpr uint32_t TMEM_COLS = TOK < 32 ? 32 : TOK;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = smem_u32(smem_raw);
  const uint32_t base_u32 = (raw_u32 + 1023u) & ~1023u;   // the same offset in every CTA
  uint8_t* base = smem_raw + (base_u32 - raw_u32);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int split = args.split;                           // CTAs of the cluster
  const int rank = static_cast<int>(cluster_ctarank());
  const int n0 = static_cast<int>(blockIdx.x) / split * BN;
  const int kblocks = (args.K + BK - 1) / BK;
  const int kb0 = static_cast<int>(static_cast<int64_t>(kblocks) * rank / split);
  const int nkb = static_cast<int>(static_cast<int64_t>(kblocks) * (rank + 1) / split) - kb0;   // >= 1

  const uint32_t bar0 = base_u32 + S::OFF_BAR;
  auto BAR = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
  constexpr int B_FULL = 0, B_EMPTY = STAGES, B_ACC = 2 * STAGES, B_DRAIN = B_ACC + 1;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(base + S::OFF_ABORT);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + S::OFF_TMEM);
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) { mbar_init(BAR(B_FULL + i), 1); mbar_init(BAR(B_EMPTY + i), 1); }
    mbar_init(BAR(B_ACC), 1);
    mbar_init(BAR(B_DRAIN), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(base_u32 + S::OFF_TMEM, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint64_t tlim = args.timeout_ns;

  bool got = false;                                // epilogue threads: the accumulator is complete
  if (warp == 0) {
    // ======================= TMA producer =======================
    if (lane == 0) {
      (void)QATTN_IN_BOUNDS(args.err, n0 < args.N && nkb >= 1 && kb0 + nkb <= kblocks);
      const int pre = nkb < STAGES ? nkb : STAGES;
      for (int u = 0; u < pre; ++u) {
        mbar_arrive_expect_tx(BAR(B_FULL + u), S::STAGE);
        tma_load_2d(base_u32 + S::OFF_W + u * TILE_W, &tm_w, BAR(B_FULL + u), (kb0 + u) * BK, n0);
      }
      grid_wait_prior();
      for (int u = 0; u < pre; ++u)
        tma_load_2d(base_u32 + S::OFF_X + u * S::TILE_X, &tm_x, BAR(B_FULL + u), (kb0 + u) * BK, 0);
      int u = pre;
      for (; u < nkb; ++u) {
        const int s = u % STAGES;
        if (!mbar_wait(BAR(B_EMPTY + s), ((u / STAGES) - 1) & 1, tlim, abort_flag, args.err)) break;
        mbar_arrive_expect_tx(BAR(B_FULL + s), S::STAGE);
        tma_load_2d(base_u32 + S::OFF_W + s * TILE_W, &tm_w, BAR(B_FULL + s), (kb0 + u) * BK, n0);
        tma_load_2d(base_u32 + S::OFF_X + s * S::TILE_X, &tm_x, BAR(B_FULL + s), (kb0 + u) * BK, 0);
      }
      for (int j = u - 1; j >= 0 && j >= u - STAGES; --j)
        mbar_drain(BAR(B_FULL + j % STAGES), (j / STAGES) & 1, tlim);
    }
  } else if (warp == 1) {
    // ======================= MMA issuer =======================
    if (lane == 0) {
      constexpr uint32_t IDESC = idesc_s8_s32(BN, TOK);
      bool ok = true;
      for (int u = 0; u < nkb; ++u) {
        const int s = u % STAGES;
        ok = mbar_wait(BAR(B_FULL + s), (u / STAGES) & 1, tlim, abort_flag, args.err);
        if (!ok) break;
        tc_fence_after();
        const uint32_t w_s = base_u32 + S::OFF_W + s * TILE_W, x_s = base_u32 + S::OFF_X + s * S::TILE_X;
#pragma unroll
        for (int kk = 0; kk < BK / 32; ++kk)
          mma_i8_ss(tmem, smem_desc(w_s + kk * 32, 16, 1024, 2u), smem_desc(x_s + kk * 32, 16, 1024, 2u),
                    IDESC, (u > 0 || kk > 0) ? 1u : 0u);
        mma_commit(BAR(B_EMPTY + s));
      }
      if (ok) mma_commit(BAR(B_ACC));
      mma_commit(BAR(B_DRAIN));
      mbar_drain(BAR(B_DRAIN), 0, tlim);
    }
  } else {
    // ======================= accumulator =======================
    got = __all_sync(0xFFFFFFFFu, mbar_wait(BAR(B_ACC), 0, tlim, abort_flag, args.err));
    grid_wait_prior();                             // s_a comes from the preceding grid
    if (got) {
      tc_fence_after();
      const int quarter = warp & 3, r = quarter * 32 + lane;
      const uint32_t acc = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
      const int n = n0 + r;
      float s_n = 0.0f, b_n = 0.0f;
      if (split == 1 && n < args.N) {
        s_n = __ldg(args.s_b + n);
        if (args.bias) b_n = __ldg(args.bias + n);
      }
#pragma unroll 1
      for (int c = 0; c < TOK; c += 16) {
        if (c >= args.M) break;                    // uniform: columns past the last token
        uint32_t v[2][8];
        tmem_ld8(acc + c, v[0]);
        tmem_ld8(acc + c + 8, v[1]);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int a = static_cast<int>(v[e >> 3][e & 7]);
          if (split > 1) {                         // the stages are free: every MMA has completed
            *reinterpret_cast<int*>(base + ((c + e) * 128 + r) * 4) = a;
          } else if (n < args.N && c + e < args.M) {
            const float y = fmaf(static_cast<float>(a) * __ldg(args.s_a + c + e), s_n, b_n);
            static_cast<uint16_t*>(args.y)[(c + e) * args.ldy + n] = to16<FP16>(y);
          }
        }
      }
    }
  }

  tc_fence_before();
  if (split > 1) {
    cluster_sync();                                // partial sums of every CTA are in shared memory
    if (warp >= 2 && got) {
      const int r = static_cast<int>(threadIdx.x) - 64, n = n0 + r;
      if (n < args.N) {
        const float s_n = __ldg(args.s_b + n), b_n = args.bias ? __ldg(args.bias + n) : 0.0f;
        for (int m = rank; m < args.M; m += split) {       // tokens of this CTA
          const uint32_t at = base_u32 + static_cast<uint32_t>((m * 128 + r) * 4);
          int a = 0;
          for (int p = 0; p < split; ++p) a += ld_cluster_s32(mapa_shared(at, static_cast<uint32_t>(p)));
          const float y = fmaf(static_cast<float>(a) * __ldg(args.s_a + m), s_n, b_n);
          if (QATTN_IN_BOUNDS(args.err, m < args.M && n < args.N))
            static_cast<uint16_t*>(args.y)[m * args.ldy + n] = to16<FP16>(y);
        }
      }
    }
    cluster_sync();                                // the peers have read this CTA's sums
  } else {
    __syncthreads();
  }
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
//   warps 2-5 (both)    epilogue of the CTA's 128 rows, overlapping the next tile's MMAs
// Tiles are visited m-fastest.  Every wait is bounded and both CTAs reach both cluster barriers.
// -------------------------------------------------------------------------------------------
namespace pair8 {
constexpr int BM = 256;
constexpr int BK = 128;
constexpr int THREADS = 192;
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
  static constexpr int ALLOC = OFF_ABORT + 4 + 1024;
  static constexpr uint32_t TMEM_COLS = 2 * BN;
  static constexpr uint32_t STAGE_TX = 2u * (TILE_A + TILE_B);
  static_assert(TILE_B % 1024 == 0, "alignment");
  static_assert(ALLOC <= 227 * 1024, "shared memory per CTA");
};
}  // namespace pair8

// 32 columns of one output row: y = acc * s_a * s_b + bias, 16-byte stores where the row is
// aligned and the chunk lies inside the output.
template <bool FP16>
__device__ __forceinline__ void epilogue_int8(const GemmInt8Args& a, const uint32_t (&v)[32], float s_m,
                                              int m, int n, bool vec) {
  if (!QATTN_IN_BOUNDS(a.err, m < a.M && n < a.N)) return;
  uint16_t* y = static_cast<uint16_t*>(a.y) + m * a.ldy + n;
  if (vec && n + 32 <= a.N) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      uint32_t p[4];
      const float4* sp = reinterpret_cast<const float4*>(a.s_b + n + 8 * g);
      const float4 s0 = __ldg(sp), s1 = __ldg(sp + 1);
      float4 b0 = make_float4(0.f, 0.f, 0.f, 0.f), b1 = b0;
      if (a.bias) {
        const float4* bp = reinterpret_cast<const float4*>(a.bias + n + 8 * g);
        b0 = __ldg(bp);
        b1 = __ldg(bp + 1);
      }
      const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
      const float b[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 8 * g + 2 * e;
        const float lo = fmaf(static_cast<float>(static_cast<int>(v[i])) * s_m, s[2 * e], b[2 * e]);
        const float hi = fmaf(static_cast<float>(static_cast<int>(v[i + 1])) * s_m, s[2 * e + 1], b[2 * e + 1]);
        p[e] = static_cast<uint32_t>(to16<FP16>(lo)) | (static_cast<uint32_t>(to16<FP16>(hi)) << 16);
      }
      reinterpret_cast<uint4*>(y)[g] = make_uint4(p[0], p[1], p[2], p[3]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      if (n + e < a.N) {
        const float b = a.bias ? __ldg(a.bias + n + e) : 0.0f;
        y[e] = to16<FP16>(fmaf(static_cast<float>(static_cast<int>(v[e])) * s_m, __ldg(a.s_b + n + e), b));
      }
    }
  }
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
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) { mbar_init(BAR(B_FULL + i), 1); mbar_init(BAR(B_EMPTY + i), 1); }
    for (int b = 0; b < 2; ++b) { mbar_init(BAR(B_ACCF + b), 1); mbar_init(BAR(B_ACCE + b), 8); }
    mbar_init(BAR(B_DRAIN), 1);
    *abort_flag = 0;
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
    if (lane == 0) {
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
    if (leader && lane == 0) {
      constexpr uint32_t IDESC = idesc_s8_s32(BM, BN);
      const uint32_t peer = rank ^ 1u;
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
          mma_commit_pair(BAR(B_EMPTY + s));                      // stage free in both CTAs
          mma_commit_pair(mapa_shared(BAR(B_EMPTY + s), peer));
        }
        if (ok) {
          mma_commit_pair(BAR(B_ACCF + ab));                      // accumulator complete
          mma_commit_pair(mapa_shared(BAR(B_ACCF + ab), peer));
        }
      }
      mma_commit_pair(BAR(B_DRAIN));
      mbar_drain(BAR(B_DRAIN), 0, tlim);
    }
  } else {
    // ======================= epilogue warps (both CTAs) =======================
    grid_wait_prior();                             // s_a comes from the preceding grid
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const bool vec = ((reinterpret_cast<uintptr_t>(args.y) | reinterpret_cast<uintptr_t>(args.s_b) |
                       reinterpret_cast<uintptr_t>(args.bias)) & 15) == 0 && args.ldy % 8 == 0;
    int i = 0;
    for (int t = pair; t < tiles; t += npairs, ++i) {
      const int ab = i & 1;
      const bool ok = mbar_wait(BAR(B_ACCF + ab), (i >> 1) & 1, tlim, abort_flag, args.err);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      tc_fence_after();
      const int m = (t % tiles_m) * BM + static_cast<int>(rank) * (BM / 2) + r;
      const int n0 = (t / tiles_m) * BN;
      const float s_m = m < args.M ? __ldg(args.s_a + m) : 0.0f;
      const uint32_t acc = tmem + lane_off + static_cast<uint32_t>(ab * BN);
#pragma unroll 1
      for (int c = 0; c < BN / 32; ++c) {
        uint32_t v[32];
        tmem_ld32(acc + c * 32, v);
        tmem_wait_ld();
        if (m < args.M && n0 + c * 32 < args.N) epilogue_int8<FP16>(args, v, s_m, m, n0 + c * 32, vec);
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
static cudaError_t launch_ex(K kernel, DeviceOnce& once, dim3 grid, unsigned cluster, int threads, int smem,
                             bool early, cudaStream_t stream, const CUtensorMap& a, const CUtensorMap& b,
                             const GemmInt8Args& args) {
  const void* fn = reinterpret_cast<const void*>(kernel);
  if (once.get([fn, smem] {
        return static_cast<int>(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
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

// How many CTAs share 128 weight rows: enough to give every SM a CTA, with at least four K blocks
// each.
static int few_split(int N, int K, int num_sms) {
  const int tiles = (N + few::BN - 1) / few::BN, kblocks = (K + few::BK - 1) / few::BK;
  int split = num_sms / tiles;
  if (split > kblocks / 4) split = kblocks / 4;
  return split < 1 ? 1 : split > 8 ? 8 : split;
}

template <int TOK, bool FP16>
static cudaError_t launch_few(const int8_t* x, int64_t ldx, const int8_t* w, int64_t ldw, const GemmInt8Args& a,
                              int num_sms, bool early, cudaStream_t stream) {
  static DeviceOnce once;
  CUtensorMap mw, mx;
  if (!make_map_rows(&mw, w, a.N, a.K, ldw, few::BN) || !make_map_rows(&mx, x, a.M, a.K, ldx, TOK))
    return cudaErrorInvalidValue;
  GemmInt8Args b = a;
  b.split = few_split(a.N, a.K, num_sms);
  const dim3 grid(static_cast<unsigned>((a.N + few::BN - 1) / few::BN * b.split));
  return launch_ex(k_gemm_int8_few<TOK, FP16>, once, grid, static_cast<unsigned>(b.split), few::THREADS,
                   few::Smem<TOK>::ALLOC, early, stream, mw, mx, b);
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
                   pair8::Smem<BN>::ALLOC, early, stream, ma, mb, a);
}

template <bool FP16>
static cudaError_t launch_any(const int8_t* x, int64_t ldx, const int8_t* w, int64_t ldw, const GemmInt8Args& a,
                              int num_sms, bool early, cudaStream_t stream) {
  if (a.M <= 16) return launch_few<16, FP16>(x, ldx, w, ldw, a, num_sms, early, stream);
  if (a.M <= 32) return launch_few<32, FP16>(x, ldx, w, ldw, a, num_sms, early, stream);
  if (a.M <= 64) return launch_few<64, FP16>(x, ldx, w, ldw, a, num_sms, early, stream);
  if (a.M <= 128) return launch_few<128, FP16>(x, ldx, w, ldw, a, num_sms, early, stream);
  return launch_pair<256, FP16>(x, ldx, w, ldw, a, num_sms, early, stream);
}

cudaError_t launch_gemm_int8(const int8_t* a8, int64_t lda, const int8_t* b8, int64_t ldb,
                             const GemmInt8Args& a, int fp16, int num_sms, bool early,
                             cudaStream_t stream) {
  return fp16 ? launch_any<true>(a8, lda, b8, ldb, a, num_sms, early, stream)
              : launch_any<false>(a8, lda, b8, ldb, a, num_sms, early, stream);
}

}  // namespace qattn
