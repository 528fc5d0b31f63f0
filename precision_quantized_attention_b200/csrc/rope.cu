// rope.cu -- rotary positions with several axes, and the per-head RMS norm of queries and keys with
// the rotation, the layout change to [B, H, L, D] and (optionally) the per-tensor FP8 quantize in
// one pass, for the stretch between the QKV projection and the quantized attention.
//
//   k_rope_table   table[t, p] = (cos a, sin a), a = pos[t, axis(p)] * freq(p)
//   k_norm_rope    y = rot(x * rsqrt(mean x^2 + eps) * w), per head row of D channels, then 16-bit
//                  or E4M3 under a given amax (the arithmetic of qattn_quantize_fp8)
//
// Both are bound by memory: each element is read once and written once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "launch.h"
#include "quant_math.cuh"
#include "sm100_ptx.cuh"

namespace qattn {

// -------------------------------------------------------------------------------------------
// Rotary table.  The angle of a far position needs more than 32 bits before it is reduced, so the
// position times the frequency (in turns) is formed in 64 bits and reduced there to a quarter
// turn and a rest of at most an eighth; cos and sin of the rest are taken in 32 bits, where
// rounding the rest moves the angle by at most 2^-24 of pi / 4.
// A thread keeps one pair (its frequency stays in registers) and steps over tokens; a block's
// stores are contiguous.
// -------------------------------------------------------------------------------------------
template <class P>
__global__ void __launch_bounds__(256) k_rope_table(const P* __restrict__ pos, int64_t pos_stride,
                                                    int tokens, int pairs,
                                                    const __grid_constant__ RopeFreqs f,
                                                    float2* __restrict__ table) {
  const int p = threadIdx.x % pairs, per_block = blockDim.x / pairs;
  const double turns4 = 4.0 * f.turns[p];
  const P* mine = pos + f.axis[p];
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * per_block + threadIdx.x / pairs; t < tokens;
       t += static_cast<int64_t>(gridDim.x) * per_block) {
    const double a = static_cast<double>(__ldg(mine + t * pos_stride)) * turns4;   // quarter turns
    double quarter;
    int q;
    if (fabs(a) < 0x1p+51) {
      // adding 1.5 * 2^52 rounds to an integer whose low bits stand in the low word
      const double m = a + 6755399441055744.0;
      quarter = m - 6755399441055744.0;
      q = __double2loint(m);
    } else {
      quarter = rint(a);                           // past 2^51 every double is a multiple of 1/2
      q = static_cast<int>(quarter - 4.0 * floor(quarter * 0.25));
    }
    // Taylor sums of sin(pi x / 2) / x and cos(pi x / 2) in x^2 for the rest x, |x| <= 1/2: coefficients
    // (pi / 2)^k / k!, the first ones left out below 2^-28
    const float x = static_cast<float>(a - quarter), z = x * x;
    const float s =
        x * fmaf(z, fmaf(z, fmaf(z, fmaf(z, 0.0001604411848f, -0.004681754135f), 0.07969262625f), -0.6459640975f), 1.570796327f);
    const float c =
        fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -2.520204237e-05f, 0.0009192602748f), -0.02086348076f), 0.2536695079f), -1.23370055f), 1.0f);
    const float c1 = (q & 1) ? -s : c, s1 = (q & 1) ? c : s;
    table[t * pairs + p] = (q & 2) ? make_float2(-c1, -s1) : make_float2(c1, s1);
  }
}

cudaError_t launch_rope_table(const void* pos, int pos_is_float, int64_t pos_stride, int tokens,
                              int pairs, const RopeFreqs& f, float* table, int num_sms,
                              cudaStream_t stream) {
  const int per_block = 256 / pairs;
  const int64_t blocks = (static_cast<int64_t>(tokens) + per_block - 1) / per_block;
  const int64_t most = static_cast<int64_t>(num_sms) * 8;
  const unsigned grid = static_cast<unsigned>(blocks < most ? blocks : most);
  const int threads = per_block * pairs;
  if (pos_is_float)
    k_rope_table<float><<<grid, threads, 0, stream>>>(static_cast<const float*>(pos), pos_stride, tokens,
                                                      pairs, f, reinterpret_cast<float2*>(table));
  else
    k_rope_table<int><<<grid, threads, 0, stream>>>(static_cast<const int*>(pos), pos_stride, tokens,
                                                    pairs, f, reinterpret_cast<float2*>(table));
  return cudaGetLastError();
}

// -------------------------------------------------------------------------------------------
// Norm + rotation.  A head row of D channels is held by a group of G lanes, eight channels (one
// 16-byte load) a lane, so a warp works on 32 / G heads at once and the sum of squares is a
// shuffle over the group.  A warp takes one token and a run of its heads: the token's cos and sin
// times the norm's weights are formed once as two coefficients a channel,
//   y_j = r * (a_j x_j + b_j x_partner(j)),   a = w cos,   b = -/+ w_partner sin,
// and reused for every head.  Statistics, coefficients and products are 32-bit; y is rounded to
// the tensor's 16-bit type, and E4M3 codes are those of that rounded value, so that the codes are the
// ones qattn_quantize_fp8 would write from the 16-bit output.
//
// The arithmetic runs on packed pairs of floats (two elements an instruction): the scalar form spent
// 22 instructions an element with E4M3 output and was bound by issue slots, not by memory.
// With adjacent channels as partners (PAIRS) a packed pair holds the first channels of two partner
// pairs, another their second channels, so that no half has to be swapped.
// -------------------------------------------------------------------------------------------
template <bool FP16>
__device__ __forceinline__ void unpack2(uint32_t w, float& lo, float& hi) {
  if (FP16) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    lo = f.x;
    hi = f.y;
  } else {
    lo = bf16_lo(w);
    hi = bf16_hi(w);
  }
}

template <bool FP16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (FP16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Scale of E4M3 codes: s, r = RN(1 / s), and both packed for the fast quotient.
struct CodeDiv {
  float s, r;
  f32x2 rr, ns;
};

// E4M3 codes of four 16-bit values.  FAST: the quotient of div_rn_by, whose zeros have lost their
// sign; the codes get the values' signs back (the others have them already).
template <bool FP16, bool FAST>
__device__ __forceinline__ uint32_t codes4(uint32_t w0, uint32_t w1, const CodeDiv& d) {
  float v[4];
  unpack2<FP16>(w0, v[0], v[1]);
  unpack2<FP16>(w1, v[2], v[3]);
  if constexpr (FAST) {
    unpack_f32x2(div_f32x2(pack_f32x2(v[0], v[1]), d.rr, d.ns), v[0], v[1]);
    unpack_f32x2(div_f32x2(pack_f32x2(v[2], v[3]), d.rr, d.ns), v[2], v[3]);
    return cvt_e4m3x2(v[0], v[1]) | (cvt_e4m3x2(v[2], v[3]) << 16) |
           (__byte_perm(w0, w1, 0x7531) & 0x80808080u);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __fdiv_rn(v[i], d.s);
    return cvt_e4m3x2(v[0], v[1]) | (cvt_e4m3x2(v[2], v[3]) << 16);
  }
}

constexpr int ROPE_WARPS = 8;
constexpr int ROPE_UNROLL = 4;          // head steps whose loads are in flight together

// Eight floats (two 16-byte loads).
__device__ __forceinline__ void load_f8(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

template <int G, bool PAIRS, bool FP16>
__global__ void __launch_bounds__(32 * ROPE_WARPS)
    k_norm_rope(const __grid_constant__ NormRopeArgs args) {
  constexpr int HEADS = 32 / G;         // heads a warp holds at once
  constexpr uint32_t INF16 = FP16 ? 0x7C00u : 0x7F80u;
  int si = 0;
  while (si + 1 < args.n && blockIdx.x >= args.seg[si + 1].first_block) ++si;
  const NormRopeSeg& sg = args.seg[si];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gl = lane % G, hsub = lane / G;
  const uint32_t item = (blockIdx.x - sg.first_block) * ROPE_WARPS + warp;
  uint32_t m2 = 0;                      // largest |y| bit patterns (two 16-bit halves)
  bool bad = false;
  if (item < sg.items) {                // warp-uniform
    // token fastest, so that the warps of a block write neighbouring rows of the same heads
    const uint32_t rest = item / static_cast<uint32_t>(sg.L);
    const int t = static_cast<int>(item - rest * static_cast<uint32_t>(sg.L));
    const int b = static_cast<int>(rest / static_cast<uint32_t>(sg.chunks));
    const int chunk = static_cast<int>(rest) - b * sg.chunks;
    const int c0 = gl * 8;
    const bool live = c0 < args.D;      // lanes past D in a group idle (D not a power of two)
    const bool norm = sg.weight != nullptr;
    const bool plain = !norm && sg.table == nullptr;

    // Packed coefficients.  PAIRS: pair i holds the first channels of partner pairs 2i and 2i + 1 (a, b)
    // and pair i + 2 their second channels; else pair i holds channels 2i and 2i + 1.
    f32x2 ca[4], cb[4];
    int partner = lane;
    if (!plain) {
      float w[8], a[8], bb[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = 1.0f;
      if (norm && live) load_f8(sg.weight + c0, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) { a[j] = w[j]; bb[j] = 0.0f; }
      if (sg.table != nullptr && c0 < args.R) {          // R is a multiple of 16: a lane is in or out
        const float* row = sg.table + b * sg.table_b + static_cast<int64_t>(t) * args.R;   // R/2 (cos, sin)
        if (PAIRS) {
          float cs[8];
          load_f8(row + c0, cs);
#pragma unroll
          for (int p = 0; p < 8; p += 2) {
            a[p] = w[p] * cs[p];
            bb[p] = -w[p + 1] * cs[p + 1];
            a[p + 1] = w[p + 1] * cs[p];
            bb[p + 1] = w[p] * cs[p + 1];
          }
        } else {
          const int half = args.R / 2;
          const bool upper = c0 >= half;
          const int other = upper ? c0 - half : c0 + half;
          partner = upper ? lane - half / 8 : lane + half / 8;
          float wq[8], cs[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) wq[j] = 1.0f;
          if (norm) load_f8(sg.weight + other, wq);
          row += 2 * (upper ? other : c0);
#pragma unroll
          for (int g = 0; g < 8; g += 4) {
            load_f8(row + 2 * g, cs);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              a[g + p] = w[g + p] * cs[2 * p];
              bb[g + p] = (upper ? wq[g + p] : -wq[g + p]) * cs[2 * p + 1];
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j0 = PAIRS ? (i < 2 ? 4 * i : 4 * (i - 2) + 1) : 2 * i, j1 = PAIRS ? j0 + 2 : j0 + 1;
        ca[i] = pack_f32x2(a[j0], a[j1]);
        cb[i] = pack_f32x2(bb[j0], bb[j1]);
      }
    }

    // E4M3: scale of the given amax (a non-finite amax writes no code)
    CodeDiv cd{1.0f, 1.0f, 0, 0};
    bool fast = true, write = true;
    if (sg.e4m3) {
      const float amax = __ldg(sg.amax);
      write = amax <= 3.402823466e38f;            // false for inf and NaN
      bad = !write;
      cd.s = amax == 0.0f ? 1.0f : __fdiv_rn(amax, 448.0f);
      cd.r = __frcp_rn(cd.s);
      cd.rr = pack_f32x2(cd.r, cd.r);
      cd.ns = pack_f32x2(-cd.s, -cd.s);
      fast = markstein_ok(cd.s);
      if (write && item == 0 && lane == 0) *sg.scale_out = cd.s;
    }

    const int h_first = chunk * sg.steps * HEADS;
    const int h_end = min(sg.H, h_first + sg.steps * HEADS);
    const uint16_t* x = static_cast<const uint16_t*>(sg.x) + b * sg.x_b + t * sg.x_t + c0;
    const int64_t out0 = b * sg.o_b + t * sg.o_t + c0;
    for (int h0 = h_first; h0 < h_end; h0 += ROPE_UNROLL * HEADS) {
      uint4 v[ROPE_UNROLL];
#pragma unroll
      for (int u = 0; u < ROPE_UNROLL; ++u) {
        const int h = h0 + u * HEADS + hsub;
        v[u] = make_uint4(0u, 0u, 0u, 0u);
        if (live && h < h_end) v[u] = __ldcs(reinterpret_cast<const uint4*>(x + h * sg.x_h));
      }
#pragma unroll
      for (int u = 0; u < ROPE_UNROLL; ++u) {
        if (h0 + u * HEADS >= h_end) break;       // uniform
        const int h = h0 + u * HEADS + hsub;
        uint32_t w4[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
        if (!plain) {
          f32x2 f[4], y[4];
          float e[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) unpack2<FP16>(w4[i], e[2 * i], e[2 * i + 1]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j0 = PAIRS ? (i < 2 ? 4 * i : 4 * (i - 2) + 1) : 2 * i, j1 = PAIRS ? j0 + 2 : j0 + 1;
            f[i] = pack_f32x2(e[j0], e[j1]);
          }
          if (PAIRS) {
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = fma_f32x2(cb[i], f[i ^ 2], mul_f32x2(ca[i], f[i]));
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float p0, p1;
              unpack2<FP16>(__shfl_sync(0xFFFFFFFFu, w4[i], partner), p0, p1);
              y[i] = fma_f32x2(cb[i], pack_f32x2(p0, p1), mul_f32x2(ca[i], f[i]));
            }
          }
          if (norm) {
            f32x2 s2 = mul_f32x2(f[0], f[0]);
#pragma unroll
            for (int i = 1; i < 4; ++i) s2 = fma_f32x2(f[i], f[i], s2);
            float ss, s1;
            unpack_f32x2(s2, ss, s1);
            ss += s1;
#pragma unroll
            for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
            bad |= !(ss <= 3.402823466e38f);      // a non-finite element, or squares past FP32
            const float r = rsqrtf(fmaf(ss, args.inv_d, args.eps));
            const f32x2 r2 = pack_f32x2(r, r);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = mul_f32x2(y[i], r2);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j0 = PAIRS ? (i < 2 ? 4 * i : 4 * (i - 2) + 1) : 2 * i, j1 = PAIRS ? j0 + 2 : j0 + 1;
            unpack_f32x2(y[i], e[j0], e[j1]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) w4[i] = pack2<FP16>(e[2 * i], e[2 * i + 1]);
        }
        if (!live || h >= h_end) continue;
        uint32_t mv = w4[0] & 0x7FFF7FFFu;
#pragma unroll
        for (int i = 1; i < 4; ++i) mv = __vmaxu2(mv, w4[i] & 0x7FFF7FFFu);
        m2 = __vmaxu2(m2, mv);
        const int64_t off = out0 + h * sg.o_h;
        if (sg.e4m3) {
          if (!write) continue;
          uint2 c;
          // the fast quotient of an infinity is NaN; the division saturates it
          if (fast && max(mv & 0xFFFFu, mv >> 16) < INF16) {
            c.x = codes4<FP16, true>(w4[0], w4[1], cd);
            c.y = codes4<FP16, true>(w4[2], w4[3], cd);
          } else {
            c.x = codes4<FP16, false>(w4[0], w4[1], cd);
            c.y = codes4<FP16, false>(w4[2], w4[3], cd);
          }
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(sg.out) + off) = c;
        } else {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(sg.out) + off) =
              make_uint4(w4[0], w4[1], w4[2], w4[3]);
        }
      }
    }
  }
  const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, max(m2 & 0xFFFFu, m2 >> 16));
  bad |= m >= INF16;
  if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) atomicExch(args.err, DEV_ERR_NONFINITE);
  if (!sg.e4m3 && sg.amax != nullptr) {           // running amax: its order cannot change the result
    __shared__ uint32_t block_max;
    if (threadIdx.x == 0) block_max = 0;
    __syncthreads();
    if (lane == 0) atomicMax(&block_max, m);
    __syncthreads();
    if (threadIdx.x == 0) {
      const uint32_t mm = block_max;
      const float a = FP16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(mm)))
                           : __uint_as_float(mm << 16);
      unsigned* dst = reinterpret_cast<unsigned*>(sg.amax);
      if (__float_as_uint(a) > *static_cast<volatile unsigned*>(dst)) atomicMax(dst, __float_as_uint(a));
    }
  }
}

template <int G>
static cudaError_t launch_g(const NormRopeArgs& a, unsigned grid, bool pairs, bool fp16, cudaStream_t stream) {
  if (pairs && fp16) k_norm_rope<G, true, true><<<grid, 32 * ROPE_WARPS, 0, stream>>>(a);
  else if (pairs) k_norm_rope<G, true, false><<<grid, 32 * ROPE_WARPS, 0, stream>>>(a);
  else if (fp16) k_norm_rope<G, false, true><<<grid, 32 * ROPE_WARPS, 0, stream>>>(a);
  else k_norm_rope<G, false, false><<<grid, 32 * ROPE_WARPS, 0, stream>>>(a);
  return cudaGetLastError();
}

// The steps (of 32 / G heads) a warp takes for its token: all of them when the tokens alone give
// every SM plenty of warps, so that the table row is read and multiplied once; fewer when there are few
// tokens, down to one step, so that the heads of one token spread over the SMs.
bool plan_norm_rope(NormRopeArgs& a, int B, int num_sms, unsigned* grid) {
  const int lanes = a.D / 8;
  const int G = lanes <= 4 ? 4 : lanes <= 8 ? 8 : lanes <= 16 ? 16 : 32;
  const int heads = 32 / G;
  int most = 1;
  for (int i = 0; i < a.n; ++i) {
    const int st = (a.seg[i].H + heads - 1) / heads;
    if (st > most) most = st;
  }
  const int64_t want = static_cast<int64_t>(num_sms) * 32;      // warps
  int steps = most;
  for (;; steps = (steps + 1) / 2) {
    int64_t items = 0;
    for (int i = 0; i < a.n; ++i) {
      const int st = (a.seg[i].H + heads - 1) / heads;
      items += static_cast<int64_t>(B) * a.seg[i].L * ((st + steps - 1) / steps);
    }
    if (items >= want || steps == 1) break;
  }
  int64_t blocks = 0;
  for (int i = 0; i < a.n; ++i) {
    NormRopeSeg& s = a.seg[i];
    const int st = (s.H + heads - 1) / heads;
    s.steps = steps;
    s.chunks = (st + steps - 1) / steps;
    const int64_t items = static_cast<int64_t>(B) * s.L * s.chunks;
    if (items > 0xFFFFFFF0ll - ROPE_WARPS) return false;
    s.items = static_cast<uint32_t>(items);
    s.first_block = static_cast<unsigned>(blocks);
    blocks += (items + ROPE_WARPS - 1) / ROPE_WARPS;
    if (blocks > 0x7FFFFFFF) return false;
  }
  *grid = static_cast<unsigned>(blocks);
  return true;
}

cudaError_t launch_norm_rope(const NormRopeArgs& a, unsigned grid, int pairs, int fp16, cudaStream_t stream) {
  const int lanes = a.D / 8;
  if (lanes <= 4) return launch_g<4>(a, grid, pairs != 0, fp16 != 0, stream);
  if (lanes <= 8) return launch_g<8>(a, grid, pairs != 0, fp16 != 0, stream);
  if (lanes <= 16) return launch_g<16>(a, grid, pairs != 0, fp16 != 0, stream);
  return launch_g<32>(a, grid, pairs != 0, fp16 != 0, stream);
}

}  // namespace qattn
