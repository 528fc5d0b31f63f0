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
// rounding the rest moves the angle by at most 2^-28 turns (2.4e-8 rad).
// A thread keeps one pair (its frequency stays in registers) and steps over tokens; a block's
// stores are contiguous.
// -------------------------------------------------------------------------------------------
template <class P>
__global__ void __launch_bounds__(256) k_rope_table(const P* __restrict__ pos, int64_t pos_stride,
                                                    int tokens, int pairs,
                                                    const __grid_constant__ RopeFreqs f,
                                                    float2* __restrict__ table) {
  const int p = threadIdx.x % pairs, per_block = blockDim.x / pairs;
  const double turns = f.turns[p];
  const P* mine = pos + f.axis[p];
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * per_block + threadIdx.x / pairs; t < tokens;
       t += static_cast<int64_t>(gridDim.x) * per_block) {
    const double a = static_cast<double>(__ldg(mine + t * pos_stride)) * (4.0 * turns);   // quarter turns
    const double quarter = rint(a);
    float s, c;
    sincospif(0.5f * static_cast<float>(a - quarter), &s, &c);
    // quarter mod 4: exact in 64 bits, 0..3 after the shift
    const int q = static_cast<int>(quarter - 4.0 * floor(quarter * 0.25));
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

// E4M3 codes of four 16-bit values under scale s (r = RN(1 / s)).
template <bool FP16, bool FAST>
__device__ __forceinline__ uint32_t codes4(uint32_t w0, uint32_t w1, float s, float r) {
  float v[4];
  unpack2<FP16>(w0, v[0], v[1]);
  unpack2<FP16>(w1, v[2], v[3]);
  return cvt_e4m3x2(div_s<FAST>(v[0], s, r), div_s<FAST>(v[1], s, r)) |
         (cvt_e4m3x2(div_s<FAST>(v[2], s, r), div_s<FAST>(v[3], s, r)) << 16);
}

constexpr int ROPE_WARPS = 8;
constexpr int ROPE_UNROLL = 4;          // head steps whose loads are in flight together

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
  const int64_t item = static_cast<int64_t>(blockIdx.x - sg.first_block) * ROPE_WARPS + warp;
  const bool any = item < sg.items;     // warp-uniform
  uint32_t m2 = 0;                      // largest |y| bit patterns (two 16-bit halves)
  bool bad = false;
  if (any) {
    // token fastest, so that the warps of a block write neighbouring rows of the same heads
    const int t = static_cast<int>(item % sg.L);
    const int64_t rest = item / sg.L;
    const int chunk = static_cast<int>(rest % sg.chunks);
    const int b = static_cast<int>(rest / sg.chunks);
    const int c0 = gl * 8;
    const bool live = c0 < args.D;      // lanes past D in a group idle (D not a power of two)
    const bool norm = sg.weight != nullptr;
    const bool plain = !norm && sg.table == nullptr;

    float ca[8], cb[8];
    bool rot = false;
    int partner = lane;
    if (!plain) {
#pragma unroll
      for (int j = 0; j < 8; ++j) { ca[j] = 1.0f; cb[j] = 0.0f; }
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = 1.0f;
      if (norm && live) {
        const float4* wp = reinterpret_cast<const float4*>(sg.weight + c0);
        const float4 w0 = __ldg(wp), w1 = __ldg(wp + 1);
        w[0] = w0.x; w[1] = w0.y; w[2] = w0.z; w[3] = w0.w;
        w[4] = w1.x; w[5] = w1.y; w[6] = w1.z; w[7] = w1.w;
      }
      rot = sg.table != nullptr && c0 < args.R;
      const float* row = sg.table + b * sg.table_b + static_cast<int64_t>(t) * args.R;   // R/2 (cos, sin)
      if (PAIRS) {
        if (rot) {
          const float4* tp = reinterpret_cast<const float4*>(row + c0);
          const float4 t0 = __ldg(tp), t1 = __ldg(tp + 1);
          const float cs[8] = {t0.x, t0.y, t0.z, t0.w, t1.x, t1.y, t1.z, t1.w};
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            ca[2 * p] = w[2 * p] * cs[2 * p];
            cb[2 * p] = -w[2 * p + 1] * cs[2 * p + 1];
            ca[2 * p + 1] = w[2 * p + 1] * cs[2 * p];
            cb[2 * p + 1] = w[2 * p] * cs[2 * p + 1];
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) ca[j] = w[j];
        }
      } else {
        const int half = args.R / 2;
        const bool upper = c0 >= half;
        float wq[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) wq[j] = 1.0f;
        if (rot) {
          partner = upper ? lane - half / 8 : lane + half / 8;
          if (norm) {
            const float4* wp = reinterpret_cast<const float4*>(sg.weight + (upper ? c0 - half : c0 + half));
            const float4 w0 = __ldg(wp), w1 = __ldg(wp + 1);
            wq[0] = w0.x; wq[1] = w0.y; wq[2] = w0.z; wq[3] = w0.w;
            wq[4] = w1.x; wq[5] = w1.y; wq[6] = w1.z; wq[7] = w1.w;
          }
          const float4* tp = reinterpret_cast<const float4*>(row + 2 * (upper ? c0 - half : c0));
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const float4 v = __ldg(tp + p);
            ca[2 * p] = w[2 * p] * v.x;
            cb[2 * p] = (upper ? wq[2 * p] : -wq[2 * p]) * v.y;
            ca[2 * p + 1] = w[2 * p + 1] * v.z;
            cb[2 * p + 1] = (upper ? wq[2 * p + 1] : -wq[2 * p + 1]) * v.w;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) ca[j] = w[j];
        }
      }
    }

    // E4M3: scale of the given amax (a non-finite amax writes no code)
    float qs = 1.0f, qr = 1.0f;
    bool fast = true, write = true;
    if (sg.e4m3) {
      const float amax = __ldg(sg.amax);
      write = amax <= 3.402823466e38f;            // false for inf and NaN
      bad = !write;
      qs = amax == 0.0f ? 1.0f : __fdiv_rn(amax, 448.0f);
      qr = __frcp_rn(qs);
      fast = markstein_ok(qs);
      if (write && item == 0 && lane == 0) *sg.scale_out = qs;
    }

    const uint16_t* x = static_cast<const uint16_t*>(sg.x) + b * sg.x_b + t * sg.x_t + c0;
    const int64_t out0 = b * sg.o_b + t * sg.o_t + c0;
    const int h_end = min(sg.H, (chunk + 1) * sg.steps * HEADS);
    for (int h0 = chunk * sg.steps * HEADS; h0 < h_end; h0 += ROPE_UNROLL * HEADS) {
      uint4 v[ROPE_UNROLL];
#pragma unroll
      for (int u = 0; u < ROPE_UNROLL; ++u) {
        const int h = h0 + u * HEADS + hsub;
        v[u] = make_uint4(0u, 0u, 0u, 0u);
        if (live && h < h_end) v[u] = __ldcs(reinterpret_cast<const uint4*>(x + h * sg.x_h));
      }
#pragma unroll
      for (int u = 0; u < ROPE_UNROLL; ++u) {
        const int h = h0 + u * HEADS + hsub;
        uint32_t w4[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
        if (!plain) {
          float f[8], fp[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) unpack2<FP16>(w4[i], f[2 * i], f[2 * i + 1]);
          if (PAIRS) {
#pragma unroll
            for (int j = 0; j < 8; ++j) fp[j] = f[j ^ 1];
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              unpack2<FP16>(__shfl_sync(0xFFFFFFFFu, w4[i], partner), fp[2 * i], fp[2 * i + 1]);
          }
          float r = 1.0f;
          if (norm) {
            float ss = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
#pragma unroll
            for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
            bad |= !(ss <= 3.402823466e38f);      // a non-finite element, or squares past FP32
            r = rsqrtf(fmaf(ss, args.inv_d, args.eps));
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            f[j] *= ca[j] * r;
            if (rot) f[j] = fmaf(cb[j] * r, fp[j], f[j]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) w4[i] = pack2<FP16>(f[2 * i], f[2 * i + 1]);
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
            c.x = codes4<FP16, true>(w4[0], w4[1], qs, qr);
            c.y = codes4<FP16, true>(w4[2], w4[3], qs, qr);
          } else {
            c.x = codes4<FP16, false>(w4[0], w4[1], qs, qr);
            c.y = codes4<FP16, false>(w4[2], w4[3], qs, qr);
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
    s.items = static_cast<int64_t>(B) * s.L * s.chunks;
    s.first_block = static_cast<unsigned>(blocks);
    blocks += (s.items + ROPE_WARPS - 1) / ROPE_WARPS;
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
